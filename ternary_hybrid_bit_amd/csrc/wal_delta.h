// What the gated delta rule's kernels share (gfx950): their arguments and gates.
#pragma once

#include "wal_args.h"
#include "wal_device.h"
#include "wal_seq.h"

namespace wal {

constexpr uint32_t kSlice = 32;   // columns of a state that a workgroup takes
constexpr int kChunk = 64;        // tokens that meet in products
// What the scan over chunks reads, by the place of a chunk: of a key head K by rows and Q as operands, of a value head
// T in three parts and P in two as operands and the factors of the rows (all but the factors in bf16).
constexpr uint32_t kOperand = 1024, kTriangle = 6 * kOperand;   // 16 bytes a lane; a 64 x 64 lower triangle
constexpr uint32_t kTParts = 3, kPParts = 2;
constexpr uint32_t kPAt = kTParts * kTriangle, kVecAt = kPAt + kPParts * kTriangle, kItemBytes = kVecAt + 6 * 256;
constexpr uint32_t key_item_bytes(uint32_t key_dim) { return 2 * kChunk * 2 * key_dim; }
constexpr uint64_t place_bytes(uint32_t key_heads, uint32_t heads, uint32_t key_dim) {
  return (uint64_t)key_heads * key_item_bytes(key_dim) + (uint64_t)heads * kItemBytes;
}

struct Delta {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* a;
  const float* b;
  const float* decay;            // of each value head, NULL: a and b are the gates themselves
  const float* shift;
  const int32_t* starts;
  const int32_t* slots;
  float* state;                  // [n_slots][value head][key_dim][value_dim]
  uint16_t* out;
  uint64_t ldq, ldk, ldv, lda, ldb, ldo;
  uint32_t n_seqs, n, max_new, n_slots;
  uint32_t heads, group, value_dim, slices;   // value heads, those that share a key head
  float eps, scale;              // eps 0: q and k as they are
  uint32_t seq0;                 // token by token: sequences before the launch's
  int32_t few;                   // a call in both forms: sequences of at most so many rows go token by token, others on chunks
  // calls on chunks: sequence s has the places from starts[s] / 64 + s on, one for each chunk; a launch takes `places`
  // of them from place0, and a sequence that goes on leaves its state in carry[1] and finds it in carry[0]
  uint8_t* ws;                   // of value heads
  uint8_t* key_ws;               // of key heads
  float* carry[2];
  uint32_t place0, places, key_item;
  uint32_t seqs, together;       // sequences that a launch of the scan looks at, heads that it puts on one chiplet
};

// Launches (wal_status).  Token by token: of sequences with at most a.few rows; on chunks: of those with more.
int delta_step(const Delta& a, uint32_t key_dim, void* stream);
// In as many launches as a.places take of the call's `all` places.
int delta_chunks(Delta& a, uint32_t key_dim, uint32_t all, void* stream);

}  // namespace wal

namespace {

using namespace wal;

__device__ __forceinline__ Seq delta_seq(const Delta& a, uint32_t s) {
  return cut_seq(a.starts[s], a.starts[s + 1], 0, (int32_t)a.n, (int32_t)a.max_new, (int32_t)a.n, false);
}

// Where a sequence's state is kept; below 0: nowhere, it begins with zeros.
__device__ __forceinline__ int64_t kept_at(const Delta& a, uint32_t s) {
  const uint32_t slot = a.slots ? (uint32_t)a.slots[s] : 0xFFFFFFFFu;
  return a.state && slot < a.n_slots ? (int64_t)slot : -1;
}

struct Gates {
  float log_alpha, beta;   // the decay's logarithm, at most 0, and the step
};

__device__ __forceinline__ Gates gates_of(const Delta& a, uint64_t row, uint32_t head) {
  const float x = a.a[row * a.lda + head], y = a.b[row * a.ldb + head];
  if (!a.decay) return Gates{x > 0.f ? 0.f : x, y};
  const float z = x + a.shift[head], soft = fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
  const float g = -a.decay[head] * soft;
  return Gates{z != z ? z : g > 0.f ? 0.f : g, 1.f / (1.f + expf(-y))};
}

__device__ __forceinline__ float bf16_value(uint16_t w) { return __uint_as_float((uint32_t)w << 16); }

// 1 / sqrt(sum of squares + eps): what a row of q or k is multiplied by.  Squares past the range of fp32 would make it 0 and
// the row's part vanish without a sign of it: NaN, as on chunks.
__device__ __forceinline__ float unit(const Delta& a, float squares) {
  return !(squares < INFINITY) ? NAN : a.eps > 0.f ? 1.f / sqrtf(squares + a.eps) : 1.f;
}

}  // namespace
