// Attention over the paged cache and over packed prompts for gfx950:
//     out[row][h] = sum_j w_j v_j,  w = softmax_j(scale * q[row][h] . k_j).
//
// One wavefront takes one query row of one head and runs over its keys 64 at
// a time, one lane per key for the scores and one lane per few elements of v
// for the sums, with the running maximum and sum of the softmax: one pass
// over the keys, nothing kept of the scores.
#include <hip/hip_runtime.h>

#include "wal_attn.h"

namespace {

template <int KIND, int D>
__device__ __forceinline__ float element(const Attn& a, bool v, int64_t row, uint32_t h, uint32_t e) {
  if constexpr (KIND == kPacked) {
    const uint16_t* p = v ? a.v + row * a.ldv : a.k + row * a.ldk;
    return __uint_as_float((uint32_t)p[h * D + e] << 16);
  } else if constexpr (KIND == kPagedBf16) {
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.cache + (v ? a.off_v : 0))[row * D + e] << 16);
  } else {
    return (float)reinterpret_cast<const int8_t*>(a.cache + (v ? a.off_v : 0))[row * D + e];
  }
}

template <int KIND, int D>
__global__ __launch_bounds__(64) void k_attn_row(Attn a) {
  __shared__ float qs[D], ps[64];
  __shared__ int64_t rs[64];
  const uint32_t t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, kvh = h / a.group;
  if (a.starts[0] > (int32_t)t || a.starts[a.n_seqs] <= (int32_t)t) return;
  const uint32_t s = find_seq(a.starts, a.n_seqs, (int32_t)t);
  const Seq q = seq_of(a, s, KIND != kPacked);
  const int32_t first = q.first, i = (int32_t)t - first;
  if (i < 0 || i >= q.rows) return;
  const int32_t last = a.causal ? q.old + i : q.len - 1;
  const int32_t keys = min(q.len, last + 1);
  for (uint32_t e = lane; e < D; e += 64) qs[e] = __uint_as_float((uint32_t)a.q[t * a.ldq + h * D + e] << 16);
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc[D / 64] = {};
  for (int32_t j0 = 0; j0 < keys; j0 += 64) {
    const int32_t j = j0 + (int32_t)lane;
    int64_t row = -1;
    if (j < keys) {
      if constexpr (KIND == kPacked) {
        row = first + j;
      } else {
        const uint32_t page = (uint32_t)a.tables[(uint64_t)s * a.ldt + (j >> a.page_shift)];
        if (page < a.n_pages)
          row = ((int64_t)((uint64_t)page * a.kv_heads + kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
      }
    }
    float x = -INFINITY, vs = 1.f;
    if (row >= 0) {
      x = 0.f;
      for (uint32_t e = 0; e < D; ++e) x += qs[e] * element<KIND, D>(a, false, row, kvh, e);
      x *= a.scale;
      if constexpr (KIND == kPagedInt8) {
        x *= reinterpret_cast<const float*>(a.cache + a.off_ks)[row];
        vs = reinterpret_cast<const float*>(a.cache + a.off_vs)[row];
      }
    }
    float top = x;
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float mn = fmaxf(m, top);
    const float c = mn == -INFINITY ? 1.f : exp2f(m - mn);
    const float p = row >= 0 ? exp2f(x - mn) : 0.f;
    float sum = p;
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    l = l * c + sum;
    m = mn;
    ps[lane] = p * vs;
    rs[lane] = row;
    __syncthreads();
    for (int u = 0; u < D / 64; ++u) acc[u] *= c;
    for (int r = 0; r < 64; ++r)
      if (rs[r] >= 0)
        for (int u = 0; u < D / 64; ++u) acc[u] += ps[r] * element<KIND, D>(a, true, rs[r], kvh, 64 * u + lane);
    __syncthreads();
  }
  for (int u = 0; u < D / 64; ++u)
    a.out[t * a.ldo + h * D + 64 * u + lane] = (uint16_t)bf16_rne(l > 0.f ? acc[u] / l : (l == 0.f ? 0.f : l));
}

template <int KIND>
int launch(const Attn& a, uint32_t dim, hipStream_t s) {
  const dim3 grid(a.n, a.q_heads);
  if (dim == 64) hipLaunchKernelGGL((k_attn_row<KIND, 64>), grid, dim3(64), 0, s, a);
  if (dim == 128) hipLaunchKernelGGL((k_attn_row<KIND, 128>), grid, dim3(64), 0, s, a);
  if (dim == 256) hipLaunchKernelGGL((k_attn_row<KIND, 256>), grid, dim3(64), 0, s, a);
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}

bool heads_ok(uint32_t q_heads, uint32_t kv_heads) {
  return q_heads && kv_heads && q_heads % kv_heads == 0 && q_heads / kv_heads <= 64;
}

constexpr uint32_t kMaxRows = 1u << 26;   // query rows, sequences and tokens of a call
constexpr float kLog2e = 1.4426950408889634f;

// How a call over the cache is cut.
struct Plan {
  bool stream;               // few rows for each key/value head
  uint32_t split, n_splits, part_rows;
  uint64_t off_ml, bytes;    // of the workspace
};

// The context is split when sequences times key/value heads leave compute units idle: into
// enough pieces for four workgroups on each, not below 256 keys a piece, not above what a workgroup's
// page list holds.
Plan plan_of(const wal_kv_desc* d, uint32_t q_heads, uint32_t n_seqs, uint32_t max_new, uint32_t max_len) {
  Plan p{};
  const uint32_t group = q_heads / d->kv_heads;
  const uint64_t rows = (uint64_t)max_new * group;
  p.stream = rows <= stream_rows(d->head_dim);
  p.n_splits = 1;
  p.split = kMaxSplit;
  if (!p.stream || !rows || !n_seqs || !max_len) return p;
  const uint64_t items = (uint64_t)n_seqs * d->kv_heads, want = (1024 + items - 1) / items;
  uint32_t split = (uint32_t)((max_len + want - 1) / want);
  split = split < 256 ? 256 : (split + 127) / 128 * 128;
  p.split = split > kMaxSplit ? kMaxSplit : split;
  p.n_splits = (max_len + p.split - 1) / p.split;
  if (p.n_splits == 1) return p;
  p.part_rows = (uint32_t)rows;
  const uint64_t slots = items * p.n_splits * rows;
  p.off_ml = slots * d->head_dim * 4;
  p.bytes = p.off_ml + slots * 8;
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
      max_len > (1u << 30))
    return WAL_ERR_SHAPE;
  *bytes = plan_of(d, q_heads, n_seqs, max_new, max_len).bytes;
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
  if (!(scale - scale == 0.f) || (uint64_t)ldt * d->page_size < max_len) return WAL_ERR_ARG;
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
  a.scale = scale * kLog2e;
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
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Plan p = plan_of(d, q_heads, n_seqs, max_new, max_len);
  if (p.stream) {
    a.split = p.split;
    a.n_splits = p.n_splits;
    a.part_rows = p.part_rows;
    a.part = static_cast<float*>(ws_dev);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws_dev) + p.off_ml);
    if ((uint64_t)n_seqs * d->kv_heads * p.n_splits > 0x7FFFFFFFull) return WAL_ERR_SHAPE;
    st = attn_stream(a, d->fmt == WAL_KV_INT8, d->head_dim, max_new * a.group <= 16 ? 1 : 2, stream);
    return st || p.n_splits == 1 ? st : attn_join(a, d->head_dim, stream);
  }
  return d->fmt == WAL_KV_INT8 ? launch<kPagedInt8>(a, d->head_dim, s) : launch<kPagedBf16>(a, d->head_dim, s);
}

extern "C" int wal_attn_prompt(const void* q_dev, uint32_t ldq, const void* k_dev, uint32_t ldk, const void* v_dev,
                               uint32_t ldv, const int32_t* starts_dev, uint32_t n_seqs, uint32_t n, uint32_t max_len,
                               uint32_t q_heads, uint32_t kv_heads, uint32_t head_dim, float scale, int causal,
                               void* out_dev, uint32_t ldo, void* stream) {
  if (!starts_dev || !(scale - scale == 0.f)) return WAL_ERR_ARG;
  if (!heads_ok(q_heads, kv_heads) || kv_heads > 256 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      n_seqs > kMaxRows || n > kMaxRows || max_len > kMaxRows)
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
  a.scale = scale * kLog2e;
  a.causal = causal ? 1 : 0;
  a.max_new = a.max_len = max_len;
  a.kv_heads = kv_heads;
  return launch<kPacked>(a, head_dim, static_cast<hipStream_t>(stream));
}
