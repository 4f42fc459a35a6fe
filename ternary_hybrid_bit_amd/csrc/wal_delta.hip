// Entry points of the gated delta rule: checks of the arguments and the choice
// of kernel.
#include <hip/hip_runtime.h>

#include "wal_delta.h"

namespace {

constexpr uint32_t kMaxRows = 1u << 24;   // rows and sequences of a call
constexpr uint32_t kMaxPitch = 1u << 24;  // elements from a row to the next: 64 rows in 32 bits of bytes
// Tokens of a sequence up to which a call goes token by token, by its slices of states and tokens in all.  On chunks the time is the same up to
// 64 tokens and grows with the slices, token by token it grows with the tokens and little with the others before memory
// is busy.  Where the two meet (sequences of equal lengths in a graph, heads of 128 x 128 unless said; token by token and on
// chunks, us): 192 slices, 8 tokens 18.6 and 20.2, 10 tokens 21.6 and 20.2; 256 slices of heads of 64 x 32, 10 tokens 21.1 and 21.8; 384,
// 10 tokens 24.5 and 27.3, 12 tokens 27.9 and 27.4; 512 of 64 x 64, 12 tokens 26.4 and 27.8, 16 tokens 33.4 and 27.8; 768, 10 tokens 32.9
// and 36.4, 12 tokens 37.6 and 36.5; 1024, 16 tokens 41.8 and 41.7; 1280 of 64 x 64, 16 tokens 42.8 and 48.2, 24 tokens 60.4 and 48.3;
// 12288, 16 tokens 289 and 361, 24 tokens 412 and 367.  Uneven lengths, on average 0.4 of the largest: from 4096 slices on the sum
// of the tokens is what counts (6144, up to 24 tokens 131 and 178, 32 tokens 165 and 179, 48 tokens 235 and 181; 12288, 32 tokens 274 and
// 359, 48 tokens 388 and 365), below it is not quite (1280 of 64 x 64, 20 tokens 47.6 and 48.1; 1664, 24 tokens 53.5 and 59.8,
// 32 tokens 67.5 and 59.7).
constexpr uint32_t few_rows(uint64_t slices, uint32_t n_seqs, uint32_t n) {
  return slices < 384 ? 8 : slices < 1024 ? 12 : slices >= 4096 && n <= 16ull * n_seqs ? 32 : 16;
}
// The same for the sequences of a call that brings a prompt with them, each in its own form then, one after the other; 0: all
// on chunks (a prompt of 300 among others, us in both forms and on chunks: 512 slices, 7 of 4 tokens 41.9 and 36.0; 768, 3 of 4 tokens
// 49.8 and 47.9, of one 43.5 and 48.7; 1024, 15 of 4 tokens 46.8 and 49.3, of 12 62.4 and 49.3; 1536, 7 of 8 tokens 62.9 and
// 65.5; 2048, 31 of 4 tokens 55.4 and 76.3, of 12 78.8 and 76.6; 12288, 63 of 16 tokens and a prompt of 500 353 and 385, of one
// 151 and 369).
constexpr uint32_t few_beside_prompt(uint64_t slices) { return slices < 1024 ? 0 : slices < 4096 ? 8 : 16; }
constexpr uint64_t kMaxItems = 256ull << 20;   // bytes of a launch's chunks: what the last cache holds

// How a call is cut.
struct Plan {
  bool step, chunks;         // token by token, on chunks, or each sequence in one of both
  uint32_t few;              // rows of a sequence up to which it goes token by token
  uint32_t all, places;      // places of chunks, and those of one launch
  uint64_t carry, bytes;     // bytes of a carried state; of the workspace
};

Plan plan_of(const wal_delta_desc* d, uint32_t n_seqs, uint32_t n, uint32_t max_new) {
  Plan p{};
  const uint64_t slices = (uint64_t)n_seqs * d->value_heads * (d->value_dim / kSlice);
  p.few = few_rows(slices, n_seqs, n);
  p.chunks = n && n_seqs && max_new > p.few;
  p.step = !p.chunks;
  if (p.step) return p;
  // Both, if all but one sequence can bring that few rows on average (the host knows the sum and the largest).
  p.few = few_beside_prompt(slices);
  p.step = n_seqs > 1 && p.few && n <= max_new + (n_seqs - 1ull) * p.few;
  if (!p.step) p.few = 0;
  const uint64_t place = place_bytes(d->key_heads, d->value_heads, d->key_dim), most = kMaxItems / place;   // (four at least)
  p.all = n / kChunk + n_seqs;
  p.places = p.all <= most ? p.all : (uint32_t)most;
  p.carry = p.places < p.all ? 4ull * d->value_heads * d->key_dim * d->value_dim : 0;
  p.bytes = p.places * place + 2 * p.carry;
  return p;
}

int check_desc(const wal_delta_desc* d) {
  if (!d || !(fabsf(d->scale) < INFINITY) || !(d->norm_eps == 0.f || (d->norm_eps >= 0x1p-126f && d->norm_eps < INFINITY)))
    return WAL_ERR_ARG;
  if (!d->key_heads || !d->value_heads || d->value_heads > 1024 || d->value_heads % d->key_heads) return WAL_ERR_SHAPE;
  if ((d->key_dim != 64 && d->key_dim != 128) || !d->value_dim || d->value_dim % kSlice || d->value_dim > 256)
    return WAL_ERR_SHAPE;
  return WAL_OK;
}

}  // namespace

extern "C" int wal_delta_workspace_size(const wal_delta_desc* d, uint32_t n_seqs, uint32_t n, uint32_t max_new,
                                        size_t* bytes) {
  const int st = check_desc(d);
  if (st) return st;
  if (!bytes) return WAL_ERR_ARG;
  if (n_seqs > kMaxRows || n > kMaxRows || max_new > kMaxRows) return WAL_ERR_SHAPE;
  *bytes = plan_of(d, n_seqs, n, max_new).bytes;
  return WAL_OK;
}

extern "C" int wal_delta(const wal_delta_desc* d, const void* q_dev, uint32_t ldq, const void* k_dev, uint32_t ldk,
                         const void* v_dev, uint32_t ldv, const float* a_dev, uint32_t lda, const float* b_dev,
                         uint32_t ldb, const float* decay_dev, const float* shift_dev, const int32_t* starts_dev,
                         uint32_t n_seqs, uint32_t n, uint32_t max_new, float* state_dev, const int32_t* slots_dev,
                         uint32_t n_slots, void* out_dev, uint32_t ldo, void* ws_dev, size_t ws_bytes, void* stream) {
  size_t need = 0;
  int st = wal_delta_workspace_size(d, n_seqs, n, max_new, &need);
  if (st) return st;
  if (!a_dev || !b_dev || !starts_dev || !state_dev != !slots_dev || !decay_dev != !shift_dev || (need && !ws_dev))
    return WAL_ERR_ARG;
  if (n_slots > kMaxRows) return WAL_ERR_SHAPE;
  const uint64_t kw = (uint64_t)d->key_heads * d->key_dim, vw = (uint64_t)d->value_heads * d->value_dim, h = d->value_heads;
  if ((st = check_rows(q_dev, ldq, kw, WAL_X_BF16)) || (st = check_rows(k_dev, ldk, kw, WAL_X_BF16)) ||
      (st = check_rows(v_dev, ldv, vw, WAL_X_BF16)) || (st = check_rows(out_dev, ldo, vw, WAL_X_BF16)))
    return st;
  if (lda < h || ldb < h) return WAL_ERR_ARG;
  if (ldq > kMaxPitch || ldk > kMaxPitch || ldv > kMaxPitch || ldo > kMaxPitch) return WAL_ERR_SHAPE;
  if (!aligned(a_dev, 4) || !aligned(b_dev, 4) || !aligned(decay_dev, 4) || !aligned(shift_dev, 4) ||
      !aligned(starts_dev, 4) || !aligned(slots_dev, 4) || !aligned(state_dev, 16) || (need && !aligned(ws_dev, 256)))
    return WAL_ERR_ALIGN;
  if (ws_bytes < need) return WAL_ERR_BUFFER;
  const Rows out = rows(out_dev, n, ldo, vw, 2), ws = flat(ws_dev, need);
  const Rows state = state_dev ? flat(state_dev, 4ull * n_slots * h * d->key_dim * d->value_dim) : Rows{};
  const Rows in[9] = {rows(q_dev, n, ldq, kw, 2), rows(k_dev, n, ldk, kw, 2), rows(v_dev, n, ldv, vw, 2),
                      rows(a_dev, n, lda, h, 4), rows(b_dev, n, ldb, h, 4), flat(starts_dev, 4ull * (n_seqs + 1ull)),
                      slots_dev ? flat(slots_dev, 4ull * n_seqs) : Rows{},
                      decay_dev ? flat(decay_dev, 4 * h) : Rows{}, shift_dev ? flat(shift_dev, 4 * h) : Rows{}};
  for (const Rows& r : in)
    if (meet(r, out) || meet(r, state) || meet(r, ws)) return WAL_ERR_ARG;
  if (meet(out, state) || meet(out, ws) || meet(state, ws)) return WAL_ERR_ARG;
  if (!n || !n_seqs || !max_new) return WAL_OK;
  Delta a{};
  a.q = static_cast<const uint16_t*>(q_dev);
  a.k = static_cast<const uint16_t*>(k_dev);
  a.v = static_cast<const uint16_t*>(v_dev);
  a.a = a_dev;
  a.b = b_dev;
  a.decay = decay_dev;
  a.shift = shift_dev;
  a.starts = starts_dev;
  a.slots = slots_dev;
  a.state = state_dev;
  a.out = static_cast<uint16_t*>(out_dev);
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.lda = lda;
  a.ldb = ldb;
  a.ldo = ldo;
  a.n_seqs = n_seqs;
  a.n = n;
  a.max_new = max_new;
  a.n_slots = n_slots;
  a.heads = d->value_heads;
  a.group = d->value_heads / d->key_heads;
  a.value_dim = d->value_dim;
  a.slices = d->value_dim / kSlice;
  a.eps = d->norm_eps;
  a.scale = d->scale;
  const Plan p = plan_of(d, n_seqs, n, max_new);
  a.few = (int32_t)p.few;
  if (p.step && (st = delta_step(a, d->key_dim, stream))) return st;
  if (!p.chunks) return WAL_OK;
  a.ws = static_cast<uint8_t*>(ws_dev);
  a.key_ws = a.ws + (uint64_t)p.places * d->value_heads * kItemBytes;
  a.key_item = key_item_bytes(d->key_dim);
  a.places = p.places;
  a.carry[0] = reinterpret_cast<float*>(a.ws + p.places * place_bytes(d->key_heads, d->value_heads, d->key_dim));
  a.carry[1] = a.carry[0] + p.carry / 4;
  return delta_chunks(a, d->key_dim, p.all, stream);
}
