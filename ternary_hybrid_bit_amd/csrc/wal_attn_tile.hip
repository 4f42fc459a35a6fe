// Attention of many query rows for gfx950: chunks of a prompt over the paged
// cache, and whole prompts packed one after another.
//
// Bound by the matrix cores.  A workgroup takes 32 QT NW query rows of one key/value
// head (a row is one token of one of the query heads that share the head, token by
// token, so that the rows of a workgroup see nearly the same keys) and runs over
// tiles of 64 keys, staged in LDS by all its wavefronts: from memory to registers
// while the tile before is computed, from there to the other of two LDS
// buffers (int8 codes become bf16, exactly, on the way).  As in the kernel
// for few rows everything is transposed, so that a lane's scores belong to one
// query row (lane & 31):
//   S^T = K Q^T     v_mfma_f32_32x32x16_bf16, A = keys from LDS, B = the query
//     rows, in registers throughout.  Bits 2 and 3 of the key index are exchanged in
//     the A rows, and lane half hh = lane >> 5 receives the scores of keys 16 s +
//     8 hh .. + 7 of each 16 keys s,
//   O^T += V^T P^T  which is the K block of the second product's B operand:
//     weights go from accumulators to operands inside a lane.  V^T comes from
//     the row-major tile with transposing LDS reads (ds_read_b64_tr_b16).
// LDS rows are whole and their 16-byte pieces are exchanged by an exclusive or with
// the row, chosen so that the 16 rows of a K read and the 4 rows of a V read
// fall on different banks.
//
// The softmax is the running one with a maximum that follows only rises above 8
// (a factor of 2^8); a lane adds up its own keys' weights and the two halves of a
// row meet once, at the end.
#include <hip/hip_runtime.h>

#include "wal_attn.h"

namespace {

constexpr float kSlack = 8.f;
constexpr int kKeys = 64;

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// Place of a row's 16-byte piece in its LDS row.
template <int D>
__device__ __forceinline__ uint32_t k_piece(uint32_t row, uint32_t piece) {
  return D == 64 ? piece ^ ((row >> 1) & 7) : piece ^ (row & 15);
}
template <int D>
__device__ __forceinline__ uint32_t v_piece(uint32_t row, uint32_t piece) {
  return D == 64 ? piece ^ (4 * ((row >> 1) & 1)) : piece ^ (4 * (row & 3));
}

template <int KIND, int D, int NW>
struct Stage {
  static constexpr bool kInt8 = KIND == kPagedInt8;
  static constexpr uint32_t kThreads = 64 * NW;
  static constexpr uint32_t kPieces = D * (kInt8 ? 1 : 2) / 16;   // 16-byte pieces of a row in memory
  static constexpr uint32_t kRows = kThreads / kPieces;           // rows of one pass
  static constexpr int kPasses = kKeys / kRows;
  static_assert(kKeys % kRows == 0, "whole passes");
  u32x4_t k[kPasses], v[kPasses];
  float scale;             // int8: key scale (threads 0..63) or value scale (64..127), 0 on no page
  int32_t page[kPasses];   // of the next tile
  int32_t page_scale;
};

template <int KIND, int D, int QT, int NW>
__global__ __launch_bounds__(64 * NW, QT == 1 && D <= 128 ? 2 : 1) void k_attn_tile(Attn a) {
  using St = Stage<KIND, D, NW>;
  constexpr bool kInt8 = KIND == kPagedInt8, kPaged = KIND != kPacked;
  constexpr int kRowBytes = 2 * D, kMT = D / 32;
  constexpr uint32_t kTileRows = 32 * QT * NW, kElem = kInt8 ? 1 : 2;
  __shared__ __attribute__((aligned(256))) uint8_t ksh[2][kKeys * kRowBytes], vsh[2][kKeys * kRowBytes];
  __shared__ __attribute__((aligned(16))) float ssh[2][2][kKeys];
  __shared__ int32_t there[2][4], odd[2];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t n = lane & 31, hh = lane >> 5;
  const uint32_t kvh = blockIdx.x % a.kv_heads, rest = blockIdx.x / a.kv_heads;
  const uint32_t sp = rest % a.n_splits;
  uint32_t tile = rest / a.n_splits, s = 0;

  // the sequence and the tile of its rows: tiles are counted over the sequences, 64 of them at a time
  {
    uint32_t base = 0;
    for (;; base += 64) {
      if (base >= a.n_seqs) return;
      uint32_t mine = 0;
      if (base + lane < a.n_seqs) mine = ((uint32_t)seq_of(a, base + lane, kPaged).rows * a.group + kTileRows - 1) / kTileRows;
      uint32_t sum = mine;   // inclusive over the lanes
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t x = (uint32_t)__shfl_up((int)sum, d);
        if (lane >= (uint32_t)d) sum += x;
      }
      const uint64_t past = __ballot(sum > tile);
      if (past) {
        const int l0 = __builtin_ctzll(past);
        s = base + l0;
        tile = (uint32_t)__builtin_amdgcn_readlane((int)mine, l0) - 1 -
               (tile - (uint32_t)(__builtin_amdgcn_readlane((int)sum, l0) - __builtin_amdgcn_readlane((int)mine, l0)));
        break;
      }
      tile -= (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
    }
  }
  const Seq q = seq_of(a, s, kPaged);
  const int32_t nrows = q.rows * (int32_t)a.group, row0 = (int32_t)(tile * kTileRows);
  const int32_t row_end = min(row0 + (int32_t)kTileRows, nrows);
  // keys that the workgroup's last row sees, this workgroup's part of them
  int32_t kend = a.causal ? min(q.len, q.old + (row_end - 1) / (int32_t)a.group + 1) : q.len;
  const int32_t k0 = (int32_t)(sp * a.split);
  if (a.n_splits > 1) {
    if (k0 >= q.len) return;
    kend = min(kend, k0 + (int32_t)a.split);
  }

  // query rows as B operands
  bf16x8_t qf[QT][D / 16];
  int32_t last[QT], rown[QT];
  int32_t wave_first = 0x7FFFFFFF, wave_last = -1;   // the keys that the wavefront's first row sees, and its last
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int32_t rb = row0 + 32 * (QT * (int32_t)wave + t), r = rb + (int32_t)n;
    const int32_t i = r / (int32_t)a.group;
    const bool live = r < nrows;
    rown[t] = live ? r : -1;
    last[t] = !live ? -1 : a.causal ? q.old + i : q.len - 1;
    if (rb < nrows) {
      wave_first = min(wave_first, a.causal ? q.old + rb / (int32_t)a.group : q.len - 1);
      wave_last = max(wave_last, a.causal ? q.old + (min(rb + 32, nrows) - 1) / (int32_t)a.group : q.len - 1);
    }
    const uint16_t* p = a.q + (uint64_t)(q.first + (live ? i : 0)) * a.ldq +
                        (uint64_t)(kvh * a.group + (live ? r - i * (int32_t)a.group : 0)) * D + 8 * hh;
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      u32x4_t w = *reinterpret_cast<const u32x4_t*>(p + 16 * st);
      w = live ? w ^ a.q_sign : u32x4_t{0, 0, 0, 0};
      qf[t][st] = as_bf16x8(w);
    }
  }
  wave_last = min(wave_last, q.len - 1);

  // Tiles from here on hold keys that some of the workgroup's rows do not see.
  // There infinities and NaN among the values are taken out of the product (a weight of zero would
  // make NaN of them) and given to the rows that do see them afterwards.
  const int32_t edge = a.causal ? q.old + row0 / (int32_t)a.group : q.len - 1;

  St st;
  const uint32_t prow = tid / St::kPieces, ppiece = tid % St::kPieces;
  const uint32_t pmask = (1u << a.page_shift) - 1;
  // bytes of a page of one plane, and from the plane's start to the head's rows of page 0
  const uint32_t page_bytes = (a.kv_heads << a.page_shift) * (D * kElem), head_bytes = (kvh << a.page_shift) * (D * kElem);
  const uint8_t* kbase = kPaged ? a.cache + head_bytes + 16 * ppiece
                                : reinterpret_cast<const uint8_t*>(a.k + (uint64_t)q.first * a.ldk + kvh * D) + 16 * ppiece;
  const uint8_t* vbase = kPaged ? kbase + a.off_v
                                : reinterpret_cast<const uint8_t*>(a.v + (uint64_t)q.first * a.ldv + kvh * D) + 16 * ppiece;
  auto key_of = [&](int32_t kb, uint32_t row) { return (uint32_t)min(kb + (int32_t)row, kend - 1); };
  const int32_t* tab = a.tables + (uint64_t)s * a.ldt;
  auto load_pages = [&](int32_t kb) {
    if constexpr (kPaged) {
#pragma unroll
      for (int p = 0; p < St::kPasses; ++p) st.page[p] = tab[key_of(kb, prow + p * St::kRows) >> a.page_shift];
      if constexpr (kInt8) st.page_scale = tab[key_of(kb, lane) >> a.page_shift];
    }
  };
  auto page_or_0 = [&](int32_t page) { return (uint32_t)page < a.n_pages ? (uint32_t)page : 0u; };   // (masked later)
  uint32_t here = 0;   // bit p: pass p's row lies on a page of the cache
  auto load_rows = [&](int32_t kb) {
    here = 0;
#pragma unroll
    for (int p = 0; p < St::kPasses; ++p) {
      const uint32_t key = key_of(kb, prow + p * St::kRows);
      if constexpr (kPaged) {
        here |= ((uint32_t)st.page[p] < a.n_pages ? 1u : 0u) << p;
        const uint64_t at = (uint64_t)page_or_0(st.page[p]) * page_bytes + (key & pmask) * (D * kElem);
        st.k[p] = *reinterpret_cast<const u32x4_t*>(kbase + at);
        st.v[p] = *reinterpret_cast<const u32x4_t*>(vbase + at);
      } else {
        st.k[p] = *reinterpret_cast<const u32x4_t*>(kbase + 2 * ((uint64_t)key * (uint32_t)a.ldk));
        st.v[p] = *reinterpret_cast<const u32x4_t*>(vbase + 2 * ((uint64_t)key * (uint32_t)a.ldv));
      }
    }
    if constexpr (kInt8) {
      if (wave < 2) {
        const uint64_t row = (uint64_t)page_or_0(st.page_scale) * (a.kv_heads << a.page_shift) + (kvh << a.page_shift) +
                             (key_of(kb, lane) & pmask);
        st.scale = reinterpret_cast<const float*>(a.cache + (wave ? a.off_vs : a.off_ks))[row];
        if ((uint32_t)st.page_scale >= a.n_pages) st.scale = 0.f;
      }
    }
  };
  auto store_rows = [&](int b, int32_t kb) {
    uint32_t any = 0;
    const bool at_edge = kb + kKeys - 1 > edge;
#pragma unroll
    for (int p = 0; p < St::kPasses; ++p) {
      const uint32_t row = prow + p * St::kRows;
      uint8_t* kd = &ksh[b][row * kRowBytes];
      uint8_t* vd = &vsh[b][row * kRowBytes];
      if constexpr (kInt8) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const u32x2_t k0_ = codes_to_bf16(st.k[p][2 * u]), k1_ = codes_to_bf16(st.k[p][2 * u + 1]);
          const u32x2_t v0_ = codes_to_bf16(st.v[p][2 * u]), v1_ = codes_to_bf16(st.v[p][2 * u + 1]);
          *reinterpret_cast<u32x4_t*>(kd + 16 * k_piece<D>(row, 2 * ppiece + u)) = u32x4_t{k0_[0], k0_[1], k1_[0], k1_[1]};
          *reinterpret_cast<u32x4_t*>(vd + 16 * v_piece<D>(row, 2 * ppiece + u)) = u32x4_t{v0_[0], v0_[1], v1_[0], v1_[1]};
        }
      } else {
        *reinterpret_cast<u32x4_t*>(kd + 16 * k_piece<D>(row, ppiece)) = st.k[p];
        if (at_edge) {
#pragma unroll
          for (int i = 0; i < 4; ++i) st.v[p][i] = finite_pair(st.v[p][i], any);
        }
        if (kPaged && !(here >> p & 1)) st.v[p] = u32x4_t{0, 0, 0, 0};
        *reinterpret_cast<u32x4_t*>(vd + 16 * v_piece<D>(row, ppiece)) = st.v[p];
      }
      if (kPaged && ppiece == 0 && (row & 15) == 0) there[b][row >> 4] = here >> p & 1;
    }
    if (kInt8 && wave < 2) {
      if (wave == 1 && !(fabsf(st.scale) < INFINITY) && at_edge) {
        any = 1;
        st.scale = 0.f;
      }
      ssh[b][wave][lane] = st.scale;
    }
    if (any) odd[b] = kb + 1;   // the tile's mark: nothing to clear
  };

  // LDS addresses of the wavefront's operands
  const uint32_t krow = 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);
  const uint32_t vi = lane & 15, vrow = 8 * hh + (vi >> 2);
  uint32_t kat[D / 16], vat[kMT];
#pragma unroll
  for (int x = 0; x < D / 16; ++x) kat[x] = krow * kRowBytes + 16 * k_piece<D>(krow, 2 * x + hh);
#pragma unroll
  for (int x = 0; x < kMT; ++x)
    vat[x] = vrow * kRowBytes + 16 * v_piece<D>(vrow, 4 * x + 2 * ((lane >> 4) & 1) + ((vi & 3) >> 1)) + 8 * (vi & 1);

  f32x16_t o[QT][kMT];
  float m[QT], l[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    m[t] = kNoMax;
    l[t] = 0.f;
#pragma unroll
    for (int x = 0; x < kMT; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][x][i] = 0.f;
  }

  auto compute = [&](int b, int32_t kb) {
    bool full = kb + kKeys - 1 <= wave_first;
    if constexpr (kPaged) full = full && there[b][0] && there[b][1] && there[b][2] && there[b][3];
    f32x16_t x[QT][2];
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[t][h][i] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bf16x8_t kf = as_bf16x8(*reinterpret_cast<const u32x4_t*>(&ksh[b][kat[d] + 32 * h * kRowBytes]));
#pragma unroll
        for (int t = 0; t < QT; ++t) x[t][h] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[t][d], x[t][h], 0, 0, 0);
      }
    // value i of x belongs to key 16 (i / 8) + 8 hh + i % 8 of the tile
    if constexpr (kInt8) {
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const f32x4_t ks = *reinterpret_cast<const f32x4_t*>(&ssh[b][0][16 * (i >> 3) + (i & 7) + 8 * hh]);
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int u = 0; u < 4; ++u) x[t][i >> 4][(i & 15) + u] *= ks[u];
      }
    }
    if (__builtin_amdgcn_readfirstlane(!full)) {
      uint32_t pages = 0xFu;
      if constexpr (kPaged) pages = (there[b][0] ? 1u : 0u) | (there[b][1] ? 2u : 0u) | (there[b][2] ? 4u : 0u) | (there[b][3] ? 8u : 0u);
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        const int32_t most = last[t] - kb - 8 * (int32_t)hh;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int32_t upto = pages >> g & 1 ? most - 16 * g : -1;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[t][g >> 1][8 * (g & 1) + i] = i <= upto ? x[t][g >> 1][8 * (g & 1) + i] : -INFINITY;
        }
      }
    }
    u32x4_t pf[QT][4];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      float top = kNoMax;
#pragma unroll
      for (int i = 0; i < 32; ++i) top = fmaxf(top, x[t][i >> 4][i & 15]);
      top *= a.scale;
      if (__any(top > m[t] + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m[t], top), f = __builtin_amdgcn_exp2f(m[t] - mn);
        m[t] = mn;
        l[t] *= f;
#pragma unroll
        for (int e = 0; e < kMT; ++e) o[t][e] *= f;
      }
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        float y[4];
        f32x4_t vs;
        if constexpr (kInt8) vs = *reinterpret_cast<const f32x4_t*>(&ssh[b][1][16 * (i >> 3) + (i & 7) + 8 * hh]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          y[u] = __builtin_amdgcn_exp2f(fmaf(x[t][i >> 4][(i & 15) + u], a.scale, -m[t]));
          l[t] += y[u];
          if constexpr (kInt8) y[u] *= vs[u];
        }
        pf[t][i >> 3][(i & 7) >> 1] = pack_bf16(y[0], y[1]);
        pf[t][i >> 3][((i & 7) >> 1) + 1] = pack_bf16(y[2], y[3]);
      }
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int e = 0; e < kMT; ++e) {
        union { s16x4_t h[2]; u32x4_t w; } vf;
#pragma unroll
        for (int u = 0; u < 2; ++u)
          vf.h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4_t*)(&vsh[b][vat[e] + (16 * ks + 4 * u) * kRowBytes]));
#pragma unroll
        for (int t = 0; t < QT; ++t)
          o[t][e] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(vf.w), as_bf16x8(pf[t][ks]), o[t][e], 0, 0, 0);
      }
    if (__builtin_amdgcn_readfirstlane(odd[b] == kb + 1)) {
      // each row takes the infinities and NaN of the keys that it sees, and of those only (from memory: it is rare)
      for (int32_t j = 0; j < kKeys && kb + j < kend; ++j) {
        if (kPaged && !there[b][j >> 4]) continue;
        const uint32_t key = (uint32_t)(kb + j);
        const uint8_t* p;
        uint64_t row = 0;
        if constexpr (kPaged) {
          row = (uint64_t)page_or_0(tab[key >> a.page_shift]) * (a.kv_heads << a.page_shift) + (kvh << a.page_shift) + (key & pmask);
          p = a.cache + a.off_v + row * (D * kElem);
        } else {
          p = reinterpret_cast<const uint8_t*>(a.v + (uint64_t)(q.first + (int32_t)key) * a.ldv + kvh * D);
        }
        float vs = 0.f;
        if constexpr (kInt8) vs = reinterpret_cast<const float*>(a.cache + a.off_vs)[row];
#pragma unroll
        for (int e = 0; e < kMT; ++e)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t d = 32 * e + 8 * (i >> 2) + 4 * hh + (i & 3);
            float y;
            if constexpr (kInt8) y = vs;
            else y = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[d] << 16);
            y = fabsf(y) < INFINITY ? 0.f : y;
#pragma unroll
            for (int t = 0; t < QT; ++t) o[t][e][i] += kb + j <= last[t] ? y : 0.f;
          }
      }
    }
  };

  if (tid < 2) odd[tid] = 0;
  __syncthreads();
  if (k0 < kend) {
    load_pages(k0);
    load_rows(k0);
    load_pages(k0 + kKeys);
    store_rows(0, k0);
    load_rows(k0 + kKeys);
    load_pages(k0 + 2 * kKeys);
  }
  __syncthreads();
  int b = 0;
  for (int32_t kb = k0; kb < kend; kb += kKeys, b ^= 1) {
    if (kb <= wave_last) compute(b, kb);
    if (kb + kKeys < kend) {
      store_rows(b ^ 1, kb + kKeys);
      if (kb + 2 * kKeys < kend) {
        load_rows(kb + 2 * kKeys);
        load_pages(kb + 3 * kKeys);
      }
    }
    __syncthreads();
  }

#pragma unroll
  for (int t = 0; t < QT; ++t) {
    l[t] += __shfl_xor(l[t], 32);
    if (rown[t] < 0) continue;
    if (a.n_splits == 1) {
      const int32_t i = rown[t] / (int32_t)a.group;
      const float f = l[t] == 0.f ? 0.f : 1.f / l[t];
      uint16_t* p = a.out + (uint64_t)(q.first + i) * a.ldo + (uint64_t)(kvh * a.group + rown[t] - i * (int32_t)a.group) * D + 4 * hh;
#pragma unroll
      for (int e = 0; e < kMT; ++e)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<u32x2_t*>(p + 32 * e + 8 * u) =
              u32x2_t{pack_bf16(o[t][e][4 * u] * f, o[t][e][4 * u + 1] * f), pack_bf16(o[t][e][4 * u + 2] * f, o[t][e][4 * u + 3] * f)};
    } else {
      const uint64_t slot = (((uint64_t)s * a.n_splits + sp) * a.kv_heads + kvh) * a.part_rows + rown[t];
      float* p = a.part + slot * D + 4 * hh;
#pragma unroll
      for (int e = 0; e < kMT; ++e)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<f32x4_t*>(p + 32 * e + 8 * u) =
              f32x4_t{o[t][e][4 * u], o[t][e][4 * u + 1], o[t][e][4 * u + 2], o[t][e][4 * u + 3]};
      if (hh == 0) a.part_ml[slot] = make_float2(m[t], l[t]);
    }
  }
}

template <int KIND, int D, int QT, int NW>
int launch(const Attn& a, hipStream_t s) {
  const uint64_t blocks = attn_tiles(a.n_seqs, a.n, a.max_new, a.group, D) * a.kv_heads * a.n_splits;
  if (blocks > 0x7FFFFFFFull) return WAL_ERR_SHAPE;
  hipLaunchKernelGGL((k_attn_tile<KIND, D, QT, NW>), dim3((uint32_t)blocks), dim3(64 * NW), 0, s, a);
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}

template <int KIND>
int launch(const Attn& a, uint32_t dim, hipStream_t s) {
  if (dim == 64) return launch<KIND, 64, 1, 4>(a, s);
  if (dim == 128) return launch<KIND, 128, 1, 4>(a, s);
  return launch<KIND, 256, 1, 4>(a, s);
}

}  // namespace

namespace wal {

uint64_t attn_tiles(uint32_t n_seqs, uint32_t n, uint32_t max_new, uint32_t group, uint32_t) {
  const uint64_t rows = 128, each = ((uint64_t)max_new * group + rows - 1) / rows;
  const uint64_t all = (uint64_t)n * group / rows + n_seqs;   // every sequence's last tile may be a part
  return each * n_seqs < all ? each * n_seqs : all;
}

int attn_tile(const Attn& a, int kind, uint32_t dim, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (kind == kPacked) return launch<kPacked>(a, dim, s);
  return kind == kPagedInt8 ? launch<kPagedInt8>(a, dim, s) : launch<kPagedBf16>(a, dim, s);
}

}  // namespace wal
