// What the attention kernels share (gfx950): their arguments, the cutting of a
// call into sequences and rows, fragments of the matrix instructions.
#pragma once

#include "wal_args.h"
#include "wal_device.h"
#include "wal_seq.h"

namespace wal {

enum { kPacked = 0, kPagedBf16 = 1, kPagedInt8 = 2 };

struct Attn {
  const uint16_t* q;
  uint16_t* out;
  const int32_t* starts;
  uint64_t ldq, ldo;
  uint32_t n_seqs, n, q_heads, kv_heads, group;
  float scale;                   // of the scores, times log2(e): weights are powers of two; above 0,
  uint32_t q_sign;               // its sign goes to the queries (exclusive or on bf16 pairs)
  uint32_t causal, max_new, max_len;
  // paged
  const uint8_t* cache;
  const int32_t* tables;
  const int32_t* lens;
  uint64_t off_v, off_ks, off_vs;
  uint32_t ldt, n_pages, page_shift;
  // packed rows
  const uint16_t* k;
  const uint16_t* v;
  uint64_t ldk, ldv;
  // keys of one workgroup when the context is split, and the partial results
  uint32_t split, n_splits;
  float* part;                   // [split][kv head][n * group][dim] sums of w v
  float2* part_ml;               // [split][kv head][n * group] maximum, sum of w
  uint32_t* counters;            // [n_seqs][kv head] pieces done, 0 between calls: attn_stream joins itself (else NULL)
  uint32_t ones_done;            // contexts of one piece are not partial results
};

constexpr uint32_t kMaxSplit = 4096;   // keys of a workgroup of attn_stream: its pages' addresses fit in 2 KB of LDS
constexpr int kJoinHere = 16;          // pieces that attn_stream joins itself
constexpr uint32_t kCounters = 16384;  // sequences times key/value heads of such a call
// Query rows of a key/value head that attn_stream takes: two tiles of 16, one where two would not fit in registers.
constexpr uint32_t stream_rows(uint32_t dim) { return dim == 256 ? 16 : 32; }

// Few short sequences with one tile of rows: eight wavefronts to a workgroup instead of four, and no split.
constexpr bool stream_wide(uint32_t n_seqs, uint32_t kv_heads, uint32_t max_len) {
  return max_len <= 1024 && (uint64_t)n_seqs * kv_heads <= 256;
}

// Launches (wal_status).  attn_stream: rows of each key/value head <= 16 tiles, tiles 1 or 2;
// attn_join adds what it wrote when a.n_splits > 1 and a.counters is NULL.
int attn_stream(const Attn& a, bool int8, uint32_t dim, uint32_t tiles, void* stream);
int attn_join(const Attn& a, uint32_t dim, void* stream);
// Any number of rows; kind kPacked, kPagedBf16 or kPagedInt8.  attn_tiles: how many
// tiles of query rows (workgroups of each key/value head and split) it launches, attn_tile_rows: of how many rows.
int attn_tile(const Attn& a, int kind, uint32_t dim, void* stream);
uint32_t attn_tile_rows(uint32_t n_seqs, uint32_t n, uint32_t max_new, uint32_t group, uint32_t kv_heads, uint32_t dim);
uint64_t attn_tiles(uint32_t n_seqs, uint32_t n, uint32_t max_new, uint32_t group, uint32_t kv_heads, uint32_t dim);

}  // namespace wal

namespace {

using namespace wal;

constexpr float kNoMax = -3.0e38f;   // a running maximum before the first key: finite, so that nothing subtracts infinities

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// Place of a row's partial result: row (first row of the sequence + token) * group + query head of the group.
__device__ __forceinline__ uint64_t part_row(const Attn& a, uint32_t split, uint32_t kvh, uint64_t row) {
  return ((uint64_t)split * a.kv_heads + kvh) * ((uint64_t)a.n * a.group) + row;
}

__device__ __forceinline__ Seq seq_of(const Attn& a, uint32_t s, bool paged) {
  return cut_seq(a.starts[s], a.starts[s + 1], paged ? a.lens[s] : 0, (int32_t)a.n, (int32_t)a.max_new, (int32_t)a.max_len, paged);
}

// The sequence of query row t: the last s with starts[s] <= t.
__device__ __forceinline__ uint32_t find_seq(const int32_t* starts, uint32_t n_seqs, int32_t t) {
  uint32_t lo = 0, hi = n_seqs;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (starts[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ bf16x8_t as_bf16x8(u32x4_t v) { return __builtin_bit_cast(bf16x8_t, v); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// Four int8 codes to bf16, exactly: their floats' upper halves.
__device__ __forceinline__ u32x2_t codes_to_bf16(uint32_t w) {
  const float f0 = (float)(int8_t)w, f1 = (float)(int8_t)(w >> 8), f2 = (float)(int8_t)(w >> 16),
              f3 = (float)(int8_t)(w >> 24);
  return u32x2_t{__builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u),
                 __builtin_amdgcn_perm(__float_as_uint(f3), __float_as_uint(f2), 0x07060302u)};
}

// A pair of bf16 with infinities and NaN replaced by zero; odd: not 0 if there was one.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w, uint32_t& odd) {
  // 0xFFFF in the halves whose exponent is all ones
  const uint32_t e = ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u, f = (e >> 15) * 0xFFFFu;
  odd |= f;
  return w & ~f;
}

}  // namespace
