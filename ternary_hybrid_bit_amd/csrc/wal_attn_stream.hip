// Attention of a few new tokens over the paged cache for gfx950 (decode): up
// to 32 query rows for each key/value head, a row being one token of one of
// the query heads that share it.
//
// Bound by the bytes of the cache, each read once.  A workgroup takes one
// key/value head of one sequence over `split` keys, its wavefronts taking tiles of 32
// keys in turn.  Everything is computed transposed, so that a lane's scores
// belong to one query row (lane & 15) and no value moves between lanes:
//   S^T = K Q^T   v_mfma_f32_16x16x32_bf16, A = 16 keys, B = the query rows.
//     The keys are dealt to the two A tiles of a tile of 32 so that lane
//     group c = lane >> 4 receives the scores of keys 8 c .. 8 c + 7.
//   O^T += V^T P^T  with exactly those keys as the B operand's K block, A = V^T:
//     lane m of a group loads dim / 16 neighbouring elements of each of its 8 keys
//     (whole rows across the 16 lanes), and one byte permutation per two
//     elements turns eight keys into the operand.  No LDS is touched.
// K and V tiles go from memory straight to registers, the next tile's loads
// issued as soon as the current one's registers are consumed.
//
// The softmax is the running one, with weights 2^(x - m): m follows the true
// maximum only when a score exceeds it by more than 8 (weights up to 2^8 lose
// nothing in fp32 or bf16), so most tiles exchange nothing between lanes and
// rescale nothing.  Weights become bf16, the operand type of the second product, once, for int8 times
// their value rows' scales; their sum is of the unrounded ones, in fp32.  Against 64 bits the outputs are
// off by 2.1e-3 to 2.4e-3 (relative 2-norm) where their own rounding to bf16 alone gives 1.7e-3; weights in
// two bf16 parts would keep to that at twice the products with V.
//
// Wavefronts join through LDS.  When the context is split over workgroups, each
// writes its sums in fp32; up to kJoinHere pieces are added up, in their order, by the
// workgroup that finishes last, more by k_attn_join.
//
// Measured (32 query, 8 key/value heads of 128): 131001 bf16 tokens 98 us with the join of
// 512 pieces, over three caches in turn (5.5 TB/s); 64 sequences up to 8192, int8,
// 104.5 us (4.7 TB/s); 517 tokens 9.3 us, a chain of dependent loads.
#include <hip/hip_runtime.h>

#include "wal_attn.h"

namespace {

constexpr float kSlack = 8.f;

template <int FMT, int D>
struct Tile {
  static constexpr bool kInt8 = FMT == kPagedInt8;
  static constexpr int E = D / 16;                     // elements of a v row in a lane
  u32x4_t k[2][kInt8 ? D / 64 : D / 32];
  uint32_t v[8][kInt8 ? E / 4 : E / 2];
  float ks[kInt8 ? 8 : 1], vs[kInt8 ? 8 : 1];
};

template <int BYTES>
__device__ __forceinline__ void load_bytes(uint32_t* d, const uint8_t* p) {
  if constexpr (BYTES >= 16) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const u32x4_t w = reinterpret_cast<const u32x4_t*>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) d[4 * i + j] = w[j];
    }
  } else if constexpr (BYTES == 8) {
    const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p);
    d[0] = w[0];
    d[1] = w[1];
  } else {
    d[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// groups: row index of the first key of each 16 keys of the workgroup (below
// 0: on no page of the cache).
template <int FMT, int D>
__device__ __forceinline__ void load_k(Tile<FMT, D>& t, const Attn& a, const int64_t* groups, uint32_t g, uint32_t lane) {
  constexpr uint32_t eb = FMT == kPagedInt8 ? 1 : 2;
  const uint32_t m = lane & 15, c = lane >> 4;
  const int64_t base = max(groups[g + (m >> 3)], (int64_t)0) + 8 * ((m >> 2) & 1) + (m & 3);
  const uint8_t* p = a.cache + (uint64_t)base * D * eb + 16 * c;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int u = 0; u < (int)(D * eb / 64); ++u)
      t.k[h][u] = *reinterpret_cast<const u32x4_t*>(p + 4 * h * D * eb + 64 * u);
  if constexpr (FMT == kPagedInt8) {
    const int64_t r = max(groups[g + (c >> 1)], (int64_t)0) + 8 * (c & 1);
    load_bytes<32>(reinterpret_cast<uint32_t*>(t.ks), a.cache + a.off_ks + 4 * r);
  }
}

template <int FMT, int D>
__device__ __forceinline__ void load_v(Tile<FMT, D>& t, const Attn& a, const int64_t* groups, uint32_t g, uint32_t lane) {
  constexpr uint32_t eb = FMT == kPagedInt8 ? 1 : 2, E = D / 16;
  const uint32_t m = lane & 15, c = lane >> 4;
  const int64_t r = max(groups[g + (c >> 1)], (int64_t)0) + 8 * (c & 1);
  const uint8_t* p = a.cache + a.off_v + (uint64_t)r * D * eb + E * eb * m;
#pragma unroll
  for (int i = 0; i < 8; ++i) load_bytes<E * eb>(t.v[i], p + i * D * eb);
  if constexpr (FMT == kPagedInt8) load_bytes<32>(reinterpret_cast<uint32_t*>(t.vs), a.cache + a.off_vs + 4 * r);
}

// Keeps what is computed from loaded registers behind this point: hoisted to
// just after the loads it would wait for them there.
template <int N>
__device__ __forceinline__ void here(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(r[i]));
}
template <int N>
__device__ __forceinline__ void here(u32x4_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(r[i]));
}

// V^T as the A operand of element e: keys 8 c .. 8 c + 7 of dim E (lane & 15) + e.
template <int FMT, int D>
__device__ __forceinline__ bf16x8_t v_operand(const Tile<FMT, D>& t, int e) {
  u32x4_t w;
  if constexpr (FMT == kPagedInt8) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float x = (float)(int8_t)(t.v[2 * p][e / 4] >> (8 * (e % 4)));
      const float y = (float)(int8_t)(t.v[2 * p + 1][e / 4] >> (8 * (e % 4)));
      w[p] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      w[p] = __builtin_amdgcn_perm(t.v[2 * p + 1][e / 2], t.v[2 * p][e / 2], e % 2 ? 0x07060302u : 0x05040100u);
  }
  return as_bf16x8(w);
}

// Cache policy of a load or store that every compute unit of the GPU sees.
constexpr int kAgent = 16;

// The partial results of a sequence's rows in a piece (the whole of them below 2^32 bytes).
template <int D>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t part_rsrc(const Attn& a, const Seq& q, uint32_t kvh, uint32_t piece, int32_t rows) {
  return rsrc(a.part + part_row(a, piece, kvh, (uint64_t)q.first * a.group) * D, 4u * D * (uint32_t)rows);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t ml_rsrc(const Attn& a, const Seq& q, uint32_t kvh, uint32_t piece, int32_t rows) {
  return rsrc(a.part_ml + part_row(a, piece, kvh, (uint64_t)q.first * a.group), 8u * (uint32_t)rows);
}

// Four elements of query row r of the sequence and head: the sums over the sum of the weights.
template <int D>
__device__ __forceinline__ void store_row(const Attn& a, const Seq& q, uint32_t kvh, int32_t r, uint32_t d, f32x4_t acc, float sum) {
  const int32_t tok = r / (int32_t)a.group;
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* p = a.out + (uint64_t)(q.first + tok) * a.ldo + (uint64_t)(kvh * a.group + r - tok * (int32_t)a.group) * D + d;
  *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16(acc[0] * f, acc[1] * f), pack_bf16(acc[2] * f, acc[3] * f)};
}

// Wavefronts a SIMD that the register allocator aims at.
constexpr int stream_waves(int fmt, int dim, int tiles) {
  return dim * tiles <= 128 ? 3 : dim == 256 && fmt == kPagedBf16 ? 1 : 2;
}

template <int FMT, int D, int NT, int NW>
__global__ __launch_bounds__(64 * NW, stream_waves(FMT, D, NT)) void k_attn_stream(Attn a) {
  constexpr int E = D / 16;
  constexpr bool kInt8 = FMT == kPagedInt8;
  __shared__ int64_t groups[kMaxSplit / 16 + 2];
  __shared__ float osh[NW][16][D + 4];
  __shared__ float msh[NW][16], lsh[NW][16];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, c = lane >> 4;
  const uint32_t kvh = blockIdx.x % a.kv_heads, rest = blockIdx.x / a.kv_heads;
  const uint32_t sp = rest % a.n_splits, s = rest / a.n_splits;
  const Seq q = seq_of(a, s, true);
  const int32_t k0 = (int32_t)(sp * a.split), k1 = min(k0 + (int32_t)a.split, q.len);
  const int32_t nrows = q.rows * (int32_t)a.group;
  const int32_t pieces = max((q.len + (int32_t)a.split - 1) / (int32_t)a.split, 1);   // that have keys (an empty context: one)
  if (!nrows || (int32_t)sp >= pieces) return;

  for (uint32_t i = threadIdx.x; i < (uint32_t)(max(k1 - k0, 0) + 31) / 32 * 2; i += 64 * NW) {
    const uint32_t key = (uint32_t)k0 + 16 * i;
    int64_t row = -1;
    if ((int32_t)key < k1) {
      const uint32_t page = (uint32_t)a.tables[(uint64_t)s * a.ldt + (key >> a.page_shift)];
      if (page < a.n_pages)
        row = (int64_t)(((uint64_t)page * a.kv_heads + kvh) << a.page_shift) + (key & ((1u << a.page_shift) - 1));
    }
    groups[i] = row;
  }

  // the query rows as B operands, in the order in which the keys' elements are loaded
  bf16x8_t qf[NT][D / 32];
  int32_t last[NT];   // the last key that the lane's row sees
  int64_t at[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int32_t r = 16 * t + (int32_t)n, i = r / (int32_t)a.group;
    const bool live = r < nrows;
    last[t] = live ? q.old + i : -1;
    at[t] = live ? (int64_t)(kvh * a.group + r - i * (int32_t)a.group) * D : -1;
    const uint16_t* p = a.q + (uint64_t)(q.first + (live ? i : 0)) * a.ldq + (live ? at[t] : 0);
#pragma unroll
    for (int st = 0; st < D / 32; ++st) {
      const uint32_t d = kInt8 ? 64 * (st / 2) + 16 * c + 8 * (st % 2) : 32 * st + 8 * c;
      u32x4_t w = *reinterpret_cast<const u32x4_t*>(p + d);
      w = live ? w ^ a.q_sign : u32x4_t{0, 0, 0, 0};
      qf[t][st] = as_bf16x8(w);
    }
  }
  f32x4_t o[NT][E];
  float m[NT], l[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = kNoMax;
    l[t] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[t][e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  __syncthreads();

  Tile<FMT, D> kv;
  uint32_t g = 2 * wave;   // the tile's first group
  const uint32_t g_end = (uint32_t)(max(k1 - k0, 0) + 31) / 32 * 2;
  if (g < g_end) {
    load_k<FMT, D>(kv, a, groups, g, lane);
    load_v<FMT, D>(kv, a, groups, g, lane);
  }
  for (; g < g_end; g += 2 * NW) {
    const int32_t kb = k0 + 16 * (int32_t)g;
    const bool there = groups[g + (c >> 1)] >= 0;
    const bool full = __builtin_amdgcn_readfirstlane(kb + 31 <= q.old && __all(there));
#pragma unroll
    for (int h = 0; h < 2; ++h) here(kv.k[h]);
    f32x4_t x[NT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int t = 0; t < NT; ++t) x[t][h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int st = 0; st < D / 32; ++st) {
        u32x4_t w;
        if constexpr (kInt8) {
          const u32x2_t lo = codes_to_bf16(kv.k[h][st / 2][2 * (st % 2)]), hi = codes_to_bf16(kv.k[h][st / 2][2 * (st % 2) + 1]);
          w = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
        } else {
          w = kv.k[h][st];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
          x[t][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), qf[t][st], x[t][h], 0, 0, 0);
      }
    }
    if constexpr (kInt8) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[t][i / 4][i % 4] *= kv.ks[i];
    }
    const bool more = g + 2 * NW < g_end;
    if (more) load_k<FMT, D>(kv, a, groups, g + 2 * NW, lane);

    uint32_t odd = 0;   // an infinity or NaN among the values of a tile that some row sees only in part
    int32_t upto[NT];   // the last of the lane's eight keys that its row sees
#pragma unroll
    for (int t = 0; t < NT; ++t) upto[t] = full ? 7 : there ? last[t] - kb - 8 * (int32_t)c : -1;
    if (!full) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[t][i / 4][i % 4] = i <= upto[t] ? x[t][i / 4][i % 4] : -INFINITY;
      if constexpr (!kInt8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < (int)(sizeof(kv.v[0]) / 4); ++e) kv.v[i][e] = finite_pair(kv.v[i][e], odd);
      }
    }
    bf16x8_t pf[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float y[8], top = kNoMax;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, x[t][i / 4][i % 4]);
      top *= a.scale;
      if (__any(top > m[t] + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m[t], top), f = __builtin_amdgcn_exp2f(m[t] - mn);
        m[t] = mn;
        l[t] *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[t][e] *= f;
      }
      u32x4_t w;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = __builtin_amdgcn_exp2f(fmaf(x[t][i / 4][i % 4], a.scale, -m[t]));
        l[t] += y[i];
      }
      if constexpr (kInt8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)   // a key that is not seen: 0 whatever its scale; one that is, NaN if that is, at a weight of 0 too
          y[i] = i <= upto[t] ? y[i] * kv.vs[i] : 0.f;
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) w[p] = pack_bf16(y[2 * p], y[2 * p + 1]);
      pf[t] = as_bf16x8(w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) here(kv.v[i]);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bf16x8_t vf = v_operand<FMT, D>(kv, e);
#pragma unroll
      for (int t = 0; t < NT; ++t) o[t][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[t], o[t][e], 0, 0, 0);
    }
    if (!kInt8 && !full && __any(odd != 0)) {
      // each row takes the infinities and NaN of the keys that it sees, and of those only
      for (int32_t j = 0; j < 32; ++j) {
        const int64_t row = groups[g + (j >> 4)];
        if (row < 0 || kb + j >= k1) continue;
        const uint16_t* p = reinterpret_cast<const uint16_t*>(a.cache + a.off_v) + (uint64_t)(row + (j & 15)) * D;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < E; ++e)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t b = p[E * (4 * c + r) + e];
              if ((b & 0x7F80u) == 0x7F80u && kb + j <= last[t]) o[t][e][r] += __uint_as_float(b << 16);
            }
      }
    }
    if (more) load_v<FMT, D>(kv, a, groups, g + 2 * NW, lane);
  }

  // the wavefronts' sums: common maximum, then one pass over rows and elements
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l[t] += __shfl_xor(l[t], 16);
    l[t] += __shfl_xor(l[t], 32);
    if (t) __syncthreads();
    if (c == 0) {
      msh[wave][n] = m[t];
      lsh[wave][n] = l[t];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) osh[wave][n][E * (4 * c + r) + e] = o[t][e][r];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < 16 * D / 4; i += 64 * NW) {
      const uint32_t row = i / (D / 4), d = 4 * (i % (D / 4));
      const int32_t r = 16 * t + (int32_t)row;
      if (r >= nrows) continue;
      float top = kNoMax, sum = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, msh[w][row]);
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = __builtin_amdgcn_exp2f(msh[w][row] - top);
        sum += f * lsh[w][row];
        acc += f * *reinterpret_cast<const f32x4_t*>(&osh[w][row][d]);
      }
      if (pieces == 1) {
        store_row<D>(a, q, kvh, r, d, acc, sum);
      } else if (a.counters) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc), part_rsrc<D>(a, q, kvh, sp, nrows), 4 * (r * D + d), 0, kAgent);
        if (d == 0)
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, make_float2(top, sum)), ml_rsrc(a, q, kvh, sp, nrows), 8 * r, 0, kAgent);
      } else {
        const uint64_t slot = part_row(a, sp, kvh, (uint64_t)q.first * a.group + r);
        *reinterpret_cast<f32x4_t*>(a.part + slot * D + d) = acc;
        if (d == 0) a.part_ml[slot] = make_float2(top, sum);
      }
    }
  }
  if (pieces == 1 || !a.counters) return;

  // The workgroup that counts itself last adds up the pieces, in their order.  Partial results go past the caches of one
  // chiplet (kAgent) both ways: a fence would write a whole cache back for every piece.
  __shared__ uint32_t before;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  uint32_t* counter = a.counters + (uint64_t)s * a.kv_heads + kvh;
  if (threadIdx.x == 0) before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (before != (uint32_t)pieces - 1) return;
  if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);   // for the next call
  for (uint32_t i = threadIdx.x; i < (uint32_t)nrows * (D / 4); i += 64 * NW) {
    const uint32_t r = i / (D / 4), d = 4 * (i % (D / 4));
    u32x2_t w[kJoinHere];
    u32x4_t v[kJoinHere];
#pragma unroll
    for (int p = 0; p < kJoinHere; ++p)
      if (p < pieces) {
        w[p] = __builtin_amdgcn_raw_buffer_load_b64(ml_rsrc(a, q, kvh, p, nrows), 8 * r, 0, kAgent);
        v[p] = __builtin_amdgcn_raw_buffer_load_b128(part_rsrc<D>(a, q, kvh, p, nrows), 4 * (r * D + d), 0, kAgent);
      }
    float top = kNoMax, sum = 0.f;
#pragma unroll
    for (int p = 0; p < kJoinHere; ++p)
      if (p < pieces) top = fmaxf(top, __uint_as_float(w[p][0]));
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < kJoinHere; ++p)
      if (p < pieces) {
        const float f = __builtin_amdgcn_exp2f(__uint_as_float(w[p][0]) - top);
        sum += f * __uint_as_float(w[p][1]);
        acc += f * __builtin_bit_cast(f32x4_t, v[p]);
      }
    store_row<D>(a, q, kvh, (int32_t)r, d, acc, sum);
  }
}

// The splits' sums of a row, added in the order of the splits (of kGroups strided parts of
// them, then of the parts): dim / 4 lanes to a row and part, 256 threads.  Many rows:
// one part, several rows to a workgroup; few rows: one row, several parts.
template <int D, int ROWS>
__global__ __launch_bounds__(256) void k_attn_join(Attn a) {
  constexpr uint32_t kLanes = D / 4, kGroups = 256 / kLanes / ROWS;
  __shared__ f32x4_t osh[ROWS][kGroups][kLanes];
  __shared__ float lsh[ROWS][kGroups], tsh[4];
  const uint32_t lane = threadIdx.x % kLanes, part = threadIdx.x / kLanes % kGroups, mine = threadIdx.x / kLanes / kGroups;
  const uint64_t row = (uint64_t)blockIdx.x * ROWS + mine;
  const uint32_t t = (uint32_t)(row / a.q_heads), h = (uint32_t)(row - (uint64_t)t * a.q_heads), kvh = h / a.group;
  const bool inside = t < a.n && a.starts[0] <= (int32_t)t && a.starts[a.n_seqs] > (int32_t)t;
  const uint32_t s = inside ? find_seq(a.starts, a.n_seqs, (int32_t)t) : 0;
  const Seq q = seq_of(a, s, true);
  const int32_t i = (int32_t)t - q.first;
  bool live = inside && i >= 0 && i < q.rows;
  uint32_t splits = ((uint32_t)q.len + a.split - 1) / a.split;
  if (a.ones_done && splits <= 1) live = false;   // attn_stream wrote the row itself
  if (!live) splits = 0;
  const uint64_t step = (uint64_t)a.n * a.q_heads;
  const uint64_t slot = live ? part_row(a, 0, kvh, (uint64_t)t * a.group + h - kvh * a.group) : 0;
  const float2* ml = a.part_ml + slot;
  // the row's maximum
  float top = kNoMax;
  if constexpr (ROWS == 1) {
    for (uint32_t p = threadIdx.x; p < splits; p += 256) top = fmaxf(top, ml[p * step].x);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    if ((threadIdx.x & 63) == 0) tsh[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tsh[0], tsh[1]), fmaxf(tsh[2], tsh[3]));
  } else {
    for (uint32_t p = lane; p < splits; p += kLanes) top = fmaxf(top, ml[p * step].x);
#pragma unroll
    for (int d = 1; d < (int)kLanes; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  }
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  const float* from = a.part + slot * D + 4 * lane;
  const uint64_t stride = step * D;
#pragma unroll 4
  for (uint32_t p = part; p < splits; p += kGroups) {
    const float2 w = ml[p * step];
    const f32x4_t x = *reinterpret_cast<const f32x4_t*>(from + p * stride);
    const float f = __builtin_amdgcn_exp2f(w.x - top);
    sum += f * w.y;
    acc += f * x;
  }
  if constexpr (kGroups > 1) {
    osh[mine][part][lane] = acc;
    if (!lane) lsh[mine][part] = sum;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (uint32_t w = 1; w < kGroups; ++w) {
      acc += osh[mine][w][lane];
      sum += lsh[mine][w];
    }
  }
  if (!live) return;
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<u32x2_t*>(a.out + (uint64_t)t * a.ldo + (uint64_t)h * D + 4 * lane) =
      u32x2_t{pack_bf16(acc[0] * f, acc[1] * f), pack_bf16(acc[2] * f, acc[3] * f)};
}

// Few rows up to twice the compute units' number.
template <int D>
void join(const Attn& a, hipStream_t s) {
  constexpr int kMany = (int)join_rows(D);
  const uint64_t n = (uint64_t)a.n * a.q_heads;
  if (n <= 512) hipLaunchKernelGGL((k_attn_join<D, 1>), dim3((uint32_t)n), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_attn_join<D, kMany>), dim3((uint32_t)((n + kMany - 1) / kMany)), dim3(256), 0, s, a);
}

template <int FMT, int D>
void launch(const Attn& a, uint32_t tiles, hipStream_t s) {
  const dim3 grid(a.n_splits * a.kv_heads * a.n_seqs);
  constexpr bool kRoom = D < 256 || FMT == kPagedInt8;   // for the registers of two wavefronts a SIMD
  if (kRoom && tiles == 1 && stream_wide(a.n_seqs, a.kv_heads, a.max_len))
    hipLaunchKernelGGL((k_attn_stream<FMT, D, 1, kRoom ? 8 : 4>), grid, dim3(512), 0, s, a);
  else if (tiles == 1)
    hipLaunchKernelGGL((k_attn_stream<FMT, D, 1, 4>), grid, dim3(256), 0, s, a);
  else if constexpr (stream_rows(D) > 16)
    hipLaunchKernelGGL((k_attn_stream<FMT, D, 2, 4>), grid, dim3(256), 0, s, a);
}

}  // namespace

namespace wal {

int attn_stream(const Attn& a, bool int8, uint32_t dim, uint32_t tiles, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!launch_takes((uint64_t)a.n_splits * a.kv_heads * a.n_seqs, 256)) return WAL_ERR_SHAPE;   // (512 threads: at most 256 of them)
  if (int8) {
    if (dim == 64) launch<kPagedInt8, 64>(a, tiles, s);
    if (dim == 128) launch<kPagedInt8, 128>(a, tiles, s);
    if (dim == 256) launch<kPagedInt8, 256>(a, tiles, s);
  } else {
    if (dim == 64) launch<kPagedBf16, 64>(a, tiles, s);
    if (dim == 128) launch<kPagedBf16, 128>(a, tiles, s);
    if (dim == 256) launch<kPagedBf16, 256>(a, tiles, s);
  }
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}

int attn_join(const Attn& a, uint32_t dim, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dim == 64) join<64>(a, s);
  if (dim == 128) join<128>(a, s);
  if (dim == 256) join<256>(a, s);
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}

}  // namespace wal
