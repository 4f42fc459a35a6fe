// Entry points of the attention over the paged cache and over packed prompts:
// checks of the arguments, the choice of kernel and the cutting of the context.
#include <hip/hip_runtime.h>

#include "wal_attn.h"

namespace {

bool heads_ok(uint32_t q_heads, uint32_t kv_heads) {
  return q_heads && kv_heads && q_heads % kv_heads == 0 && q_heads / kv_heads <= 64;
}

constexpr uint32_t kMaxRows = 1u << 24;   // query rows and sequences of a call: times 64 heads of a group in 31 bits
constexpr uint32_t kMaxPitch = 1u << 26;  // elements from a row of keys to the next: 16 rows in 32 bits of bytes
constexpr uint64_t kMaxPartBytes = 1ull << 28;   // partial results of a call with many rows: fewer pieces beyond
constexpr float kLog2e = 1.4426950408889634f;

// The kernels multiply scores by a positive number only: masked ones are -infinity, so a
// scale of zero becomes one too small to tell weights apart.
bool scale_ok(float scale) { return fabsf(scale * kLog2e) < INFINITY; }
void set_scale(Attn& a, float scale) {
  a.scale = fmaxf(fabsf(scale * kLog2e), 1e-30f);
  a.q_sign = scale < 0.f ? 0x80008000u : 0u;
}

// How a call over the cache is cut.
struct Plan {
  bool stream;               // few rows for each key/value head: attn_stream, else attn_tile
  uint32_t split, n_splits;
  bool join_here;            // attn_stream joins the pieces itself
  uint64_t off_part, off_ml, bytes;   // of the workspace: counters, sums, maxima and sums of weights
};

// Keys of a piece of the context, max_len or more: whole.  The context is
// split when the workgroups of whole contexts leave compute units idle, or, over
// several sequences of lengths that the host does not know, would leave them
// waiting for the longest.
//  * Few rows, one sequence: two workgroups for each unit, not below 256 keys a
//    piece (131,001 bf16 tokens, 8 key/value heads: 97 us at 512 pieces, 100 at 1024, 109 at 4096).
//  * Few rows, several sequences: 6144 pieces in all, not below 256 keys, or 768 of
//    wide heads, whose workgroups have a compute unit to themselves (64 sequences up to
//    8192, int8: 102 us at 768 keys a piece, 108 at 2048 and at 512; 8 sequences up to 2048:
//    13.7 us at 256, 17.6 at 512; 4 sequences up to 16000, heads of 256: 34 us at 768, 46 at
//    512).  A piece of attn_stream is never above what a workgroup's page list holds.  Few
//    short contexts are not split at all (517 tokens: 9.3 us with eight wavefronts a workgroup,
//    6.5 + 3.0 us and a launch in pieces of 256 keys joined by k_attn_join; pieces joined by the
//    last workgroup were not timed at these lengths).
//  * Many rows, one sequence: into as many pieces as give the fewest rounds of
//    workgroups over the places for them, not below 512 keys, the joining counted as 1.5 % of
//    the products (2048 tokens over 32768, 256 workgroups: 1140 us whole, 1161 in two pieces).  At most
//    64 pieces: more were not timed, and few workgroups, as of one key/value head, leave places empty.
//  * Many rows, several sequences: pieces that fill the places once if all contexts were
//    the longest, from 128 to 1024 keys, unless there are workgroups enough for four rounds (13 sequences up to
//    4100, at most 260 workgroups: 63 us whole, 55 in pieces of 2048 keys, 49 of 1024, 52 of 512; 6
//    sequences up to 800, heads of 256: 42 us whole, 24 in pieces of 128 keys (23 with a later step), 35 of 512).
uint32_t piece(bool stream, uint32_t dim, uint32_t n_seqs, uint64_t items, uint32_t tile_rows, uint32_t max_len) {
  const auto up128 = [](uint64_t keys) { return (keys + 127) / 128 * 128; };
  if (stream) {
    const uint64_t target = n_seqs > 1 ? 6144 : 512, least = dim > 128 ? 768 : 256;
    const uint64_t want = (target + items - 1) / items, keys = up128((max_len + want - 1) / want);
    return (uint32_t)(keys < least ? least : keys > kMaxSplit ? kMaxSplit : keys);
  }
  const uint64_t places = tile_rows == 256 || dim > 128 ? 256 : 512;   // one workgroup on a compute unit, or two
  if (n_seqs > 1) {
    if (items >= 4 * places) return max_len;
    const uint64_t keys = up128(max_len * items / places);
    return (uint32_t)(keys < 128 ? 128 : keys > 1024 ? 1024 : keys);
  }
  uint32_t best = max_len;
  double least = 1e30;
  for (uint64_t n = 1; n <= 64; ++n) {
    const uint64_t keys = n == 1 ? max_len : up128((max_len + n - 1) / n);
    if (n > 1 && keys < 512) break;
    const double cost = (double)((items * n + places - 1) / places) / (double)n + (n > 1 ? 0.015 : 0.0);
    if (cost < least * 0.999) {
      least = cost;
      best = (uint32_t)keys;
    }
  }
  return best;
}

Plan plan_of(const wal_kv_desc* d, uint32_t q_heads, uint32_t n_seqs, uint32_t n, uint32_t max_new,
             uint32_t max_len) {
  Plan p{};
  const uint32_t group = q_heads / d->kv_heads, dim = d->head_dim;
  const uint64_t rows = (uint64_t)max_new * group;
  p.stream = rows <= stream_rows(dim);
  p.n_splits = 1;
  p.split = p.stream ? kMaxSplit : max_len;
  if (!rows || !n_seqs || !max_len || !n) return p;
  if (p.stream && rows <= 16 && stream_wide(n_seqs, d->kv_heads, max_len)) return p;
  const uint64_t items = (p.stream ? n_seqs : attn_tiles(n_seqs, n, max_new, group, d->kv_heads, dim)) * d->kv_heads;
  p.split = piece(p.stream, dim, n_seqs, items, attn_tile_rows(n_seqs, n, max_new, group, d->kv_heads, dim), max_len);
  const uint64_t all = (uint64_t)n * q_heads;   // rows of a split's partial results
  if (!p.stream) {
    const uint64_t most = kMaxPartBytes / (all * dim * 4), keys = most > 1 ? (max_len + most - 1) / most : max_len;
    if (p.split < keys) p.split = (uint32_t)((keys + 127) / 128 * 128);
  }
  p.n_splits = (max_len + p.split - 1) / p.split;
  if (p.n_splits == 1) return p;
  // Workgroups go to the shader engines in turn: with an even number of splits
  // to a sequence some engines would get the ends of the contexts again and again,
  // where shorter sequences have nothing to do.
  if (n_seqs > 1) p.n_splits |= 1;
  p.join_here = p.stream && p.n_splits <= (uint32_t)kJoinHere && (uint64_t)n_seqs * d->kv_heads <= kCounters;
  p.off_part = 4 * kCounters;
  p.off_ml = p.off_part + p.n_splits * all * dim * 4;
  p.bytes = p.off_ml + p.n_splits * all * 8;
  return p;
}

}  // namespace

extern "C" int wal_attn_paged_workspace_size(const wal_kv_desc* d, uint32_t q_heads, uint32_t n_seqs, uint32_t n,
                                             uint32_t max_new, uint32_t max_len, size_t* bytes) {
  wal_kv_info f;
  const int st = wal_kv_size(d, &f);
  if (st) return st;
  if (!bytes) return WAL_ERR_ARG;
  if (!heads_ok(q_heads, d->kv_heads) || n_seqs > kMaxRows || n > kMaxRows || max_new > kMaxRows ||
      max_len > (1u << 30) || (uint64_t)n * q_heads > 0x7FFFFFFFull)
    return WAL_ERR_SHAPE;
  *bytes = plan_of(d, q_heads, n_seqs, n, max_new, max_len).bytes;
  return WAL_OK;
}

extern "C" int wal_attn_paged(const wal_kv_desc* d, const void* cache_dev, const int32_t* tables_dev, uint32_t ldt,
                              const int32_t* lens_dev, const int32_t* starts_dev, uint32_t n_seqs, uint32_t n,
                              uint32_t max_new, uint32_t max_len, const void* q_dev, uint32_t q_heads, uint32_t ldq,
                              float scale, void* out_dev, uint32_t ldo, void* ws_dev, size_t ws_bytes,
                              void* stream) {
  wal_kv_info f;
  size_t need = 0;
  int st = wal_kv_size(d, &f);
  if (st) return st;
  if ((st = wal_attn_paged_workspace_size(d, q_heads, n_seqs, n, max_new, max_len, &need))) return st;
  if (!cache_dev || !tables_dev || !lens_dev || !starts_dev || (need && !ws_dev)) return WAL_ERR_ARG;
  if (!scale_ok(scale) || (uint64_t)ldt * d->page_size < max_len) return WAL_ERR_ARG;
  const uint64_t width = (uint64_t)q_heads * d->head_dim;
  if ((st = check_rows(q_dev, ldq, width, WAL_X_BF16)) || (st = check_rows(out_dev, ldo, width, WAL_X_BF16))) return st;
  if (!aligned(cache_dev, 256) || !aligned(tables_dev, 4) || !aligned(lens_dev, 4) || !aligned(starts_dev, 4) ||
      (need && !aligned(ws_dev, 256)))
    return WAL_ERR_ALIGN;
  if (ws_bytes < need) return WAL_ERR_BUFFER;
  const Rows out = rows(out_dev, n, ldo, width, 2), ws = flat(ws_dev, need);
  const Rows in[5] = {rows(q_dev, n, ldq, width, 2), flat(cache_dev, f.total_bytes),
                      flat(tables_dev, 4ull * n_seqs * ldt), flat(lens_dev, 4ull * n_seqs),
                      flat(starts_dev, 4ull * (n_seqs + 1))};
  for (const Rows& r : in)
    if (meet(r, out) || meet(r, ws)) return WAL_ERR_ARG;
  if (meet(out, ws)) return WAL_ERR_ARG;
  if (!n || !n_seqs || !max_new) return WAL_OK;
  Attn a{};
  a.q = static_cast<const uint16_t*>(q_dev);
  a.out = static_cast<uint16_t*>(out_dev);
  a.starts = starts_dev;
  a.ldq = ldq;
  a.ldo = ldo;
  a.n_seqs = n_seqs;
  a.n = n;
  a.q_heads = q_heads;
  a.group = q_heads / d->kv_heads;
  set_scale(a, scale);
  a.causal = 1;
  a.max_new = max_new;
  a.max_len = max_len;
  a.cache = static_cast<const uint8_t*>(cache_dev);
  a.tables = tables_dev;
  a.lens = lens_dev;
  a.off_v = f.off_v;
  a.off_ks = f.off_ks;
  a.off_vs = f.off_vs;
  a.ldt = ldt;
  a.n_pages = d->n_pages;
  a.page_shift = (uint32_t)__builtin_ctz(d->page_size);
  a.kv_heads = d->kv_heads;
  const Plan p = plan_of(d, q_heads, n_seqs, n, max_new, max_len);
  const bool int8 = d->fmt == WAL_KV_INT8, joined = p.n_splits > 1 && !p.join_here;
  if (joined && !launch_takes((uint64_t)n * q_heads / join_rows(d->head_dim) + 1, 256)) return WAL_ERR_SHAPE;
  a.split = p.split;
  a.n_splits = p.n_splits;
  uint8_t* ws_bytes_dev = static_cast<uint8_t*>(ws_dev);
  a.part = reinterpret_cast<float*>(ws_bytes_dev + p.off_part);
  a.part_ml = reinterpret_cast<float2*>(ws_bytes_dev + p.off_ml);
  a.counters = p.join_here ? static_cast<uint32_t*>(ws_dev) : nullptr;
  a.ones_done = p.stream;
  st = p.stream ? attn_stream(a, int8, d->head_dim, max_new * a.group <= 16 ? 1 : 2, stream)
                : attn_tile(a, int8 ? kPagedInt8 : kPagedBf16, d->head_dim, stream);
  return st || !joined ? st : attn_join(a, d->head_dim, stream);
}

extern "C" int wal_attn_prompt(const void* q_dev, uint32_t ldq, const void* k_dev, uint32_t ldk, const void* v_dev,
                               uint32_t ldv, const int32_t* starts_dev, uint32_t n_seqs, uint32_t n, uint32_t max_len,
                               uint32_t q_heads, uint32_t kv_heads, uint32_t head_dim, float scale, int causal,
                               void* out_dev, uint32_t ldo, void* stream) {
  if (!starts_dev || !scale_ok(scale)) return WAL_ERR_ARG;
  if (!heads_ok(q_heads, kv_heads) || kv_heads > 256 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      n_seqs > kMaxRows || n > kMaxRows || max_len > kMaxRows || ldk > kMaxPitch || ldv > kMaxPitch)
    return WAL_ERR_SHAPE;
  const uint64_t width = (uint64_t)q_heads * head_dim, kvw = (uint64_t)kv_heads * head_dim;
  int st;
  if ((st = check_rows(q_dev, ldq, width, WAL_X_BF16)) || (st = check_rows(k_dev, ldk, kvw, WAL_X_BF16)) ||
      (st = check_rows(v_dev, ldv, kvw, WAL_X_BF16)) || (st = check_rows(out_dev, ldo, width, WAL_X_BF16)))
    return st;
  if (!aligned(starts_dev, 4)) return WAL_ERR_ALIGN;
  const Rows out = rows(out_dev, n, ldo, width, 2);
  if (meet(out, rows(q_dev, n, ldq, width, 2)) || meet(out, rows(k_dev, n, ldk, kvw, 2)) ||
      meet(out, rows(v_dev, n, ldv, kvw, 2)) || meet(out, flat(starts_dev, 4ull * (n_seqs + 1))))
    return WAL_ERR_ARG;
  if (!n || !n_seqs || !max_len) return WAL_OK;
  Attn a{};
  a.q = static_cast<const uint16_t*>(q_dev);
  a.k = static_cast<const uint16_t*>(k_dev);
  a.v = static_cast<const uint16_t*>(v_dev);
  a.out = static_cast<uint16_t*>(out_dev);
  a.starts = starts_dev;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.ldo = ldo;
  a.n_seqs = n_seqs;
  a.n = n;
  a.q_heads = q_heads;
  a.group = q_heads / kv_heads;
  set_scale(a, scale);
  a.causal = causal ? 1 : 0;
  a.max_new = a.max_len = max_len;
  a.kv_heads = kv_heads;
  a.n_splits = 1;
  return attn_tile(a, kPacked, head_dim, stream);
}
