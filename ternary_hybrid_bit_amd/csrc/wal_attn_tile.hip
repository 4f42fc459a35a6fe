// Attention of many query rows for gfx950: chunks of a prompt over the paged
// cache, and whole prompts packed one after another.
//
// Bound by the matrix cores.  A workgroup takes 128 or 256 query rows of one key/value
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
// row meet once, at the end.  Weights become bf16, the operand type of the second product, once,
// for int8 times their value rows' scales (outputs 2.0e-3 to 2.4e-3 from 64 bits, relative
// 2-norm, where their own rounding to bf16 alone gives 1.5e-3 to 1.7e-3): a second part of them would
// add half of all products to kernels that the matrix cores bound.
//
// Measured: a prompt of 8192 (32 query, 8 key/value heads of 128) 532-540 us, 1.02 PFLOP/s;
// 2048 tokens over 32768 of the int8 cache 1149-1176 us, 0.92 PFLOP/s, its vector
// instructions 3.0 times the prompt's for 1.9 times the products (k_attn_pair); 9 packed
// prompts up to 777, heads of 256, 37 us; 13 chunks over up to 4100, heads of 64, 43 us and 8
// to join (k_attn_tile).
#include <hip/hip_runtime.h>

#include "wal_attn.h"

namespace {

constexpr float kSlack = 8.f;
constexpr int kKeys = 64;   // of a tile

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

// A workgroup's share of a call.
struct Work {
  uint32_t s, kvh, sp;          // sequence, key/value head, split
  Seq q;
  int32_t nrows, row0;          // query rows of the sequence and head; the workgroup's first
  int32_t k0, kend;             // its keys
  int32_t edge;                 // from here on some of its rows do not see every key
};

// Tiles of query rows are counted over the sequences, 64 of these at a time; the last tile
// of a sequence comes first, since its rows see the most keys.  False: nothing to do.
template <bool PAGED>
__device__ __forceinline__ bool find_work(const Attn& a, uint32_t tile_rows, uint32_t lane, Work& w) {
  w.kvh = blockIdx.x % a.kv_heads;
  const uint32_t rest = blockIdx.x / a.kv_heads;
  w.sp = rest % a.n_splits;
  uint32_t tile = rest / a.n_splits;
  const int32_t group = (int32_t)a.group;
  if (a.n_seqs == 1) {
    w.s = 0;
    w.q = seq_of(a, 0, PAGED);
    const uint32_t own = (uint32_t)(w.q.rows * group + (int32_t)tile_rows - 1) / tile_rows;
    if (tile >= own) return false;
    tile = own - 1 - tile;
  } else for (uint32_t base = 0;; base += 64) {
    if (base >= a.n_seqs) return false;
    uint32_t mine = 0;
    if (base + lane < a.n_seqs) mine = ((uint32_t)seq_of(a, base + lane, PAGED).rows * a.group + tile_rows - 1) / tile_rows;
    uint32_t sum = mine;   // inclusive over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t x = (uint32_t)__shfl_up((int)sum, d);
      if (lane >= (uint32_t)d) sum += x;
    }
    const uint64_t past = __ballot(sum > tile);
    if (past) {
      const int l0 = __builtin_ctzll(past);
      const uint32_t own = (uint32_t)__builtin_amdgcn_readlane((int)mine, l0);
      const uint32_t before = (uint32_t)__builtin_amdgcn_readlane((int)sum, l0) - own;
      w.s = base + l0;
      tile = own - 1 - (tile - before);
      break;
    }
    tile -= (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
  }
  if (a.n_seqs > 1) w.q = seq_of(a, w.s, PAGED);
  w.nrows = w.q.rows * group;
  w.row0 = (int32_t)(tile * tile_rows);
  const int32_t row_end = min(w.row0 + (int32_t)tile_rows, w.nrows);
  w.kend = a.causal ? min(w.q.len, w.q.old + (row_end - 1) / group + 1) : w.q.len;
  w.k0 = (int32_t)(w.sp * a.split);
  w.edge = a.causal ? w.q.old + w.row0 / group : w.q.len - 1;
  if (a.n_splits > 1) {
    if (w.k0 >= w.q.len) return false;
    w.kend = min(w.kend, w.k0 + (int32_t)a.split);
  }
  return true;
}

// The keys' way from memory to LDS.  A wavefront moves whole rows, kWaveRows
// neighbours in one instruction, a 16-byte piece a lane; a pass of all wavefronts moves kRows
// of a tile.  Neighbours lie on one page, so pages and addresses are scalars.
template <int KIND, int D, int NW>
struct Stage {
  static constexpr bool kInt8 = KIND == kPagedInt8, kPaged = KIND != kPacked;
  static constexpr uint32_t kElem = kInt8 ? 1 : 2;
  static constexpr uint32_t kPieces = D * kElem / 16;       // 16-byte pieces of a row in memory
  static constexpr uint32_t kWaveRows = 64 / kPieces, kRows = NW * kWaveRows;
  static constexpr bool kSpare = kRows > kKeys;             // more threads than pieces: the others store nothing
  static constexpr int kPasses = kSpare ? 1 : kKeys / (int)kRows;
  static constexpr int kRowBytes = 2 * D;                   // of a row in LDS
  static_assert(kWaveRows <= 16 && (kSpare || kKeys % kRows == 0), "rows of one page, whole passes");
  const Attn& a;
  const Work& w;
  const uint32_t lane, wave, pmask;
  const int32_t wrow;          // the wavefront's first row in pass 0
  const uint32_t page_bytes, head_bytes;   // of one plane: of a page, from a page to the head's rows
  const int32_t* tab;
  bool all_there;              // every key of the workgroup lies on a page of the cache

  __device__ __forceinline__ Stage(const Attn& a_, const Work& w_, uint32_t lane_, uint32_t wave_)
      : a(a_), w(w_), lane(lane_), wave(wave_), pmask((1u << a_.page_shift) - 1), wrow((int32_t)(wave_ * kWaveRows)),
        page_bytes((a_.kv_heads << a_.page_shift) * (D * kElem)), head_bytes((w_.kvh << a_.page_shift) * (D * kElem)),
        tab(kPaged ? a_.tables + (uint64_t)w_.s * a_.ldt : nullptr) {
    all_there = true;
  }
  // Looks through the workgroup's pages (with a barrier).
  __device__ __forceinline__ void look_at_pages() {
    if constexpr (kPaged) {
      int bad = 0;
      if (w.k0 < w.kend)
        for (int32_t p = (w.k0 >> a.page_shift) + (int32_t)threadIdx.x; p <= (w.kend - 1) >> a.page_shift; p += 64 * NW)
          bad |= !on_page(tab[p]);
      all_there = !__syncthreads_or(bad);
    }
  }
  __device__ __forceinline__ bool on_page(int32_t page) const { return (uint32_t)page < a.n_pages; }
  __device__ __forceinline__ uint32_t page_or_0(int32_t page) const { return on_page(page) ? (uint32_t)page : 0u; }
  __device__ __forceinline__ uint64_t row_index(uint32_t key) const {
    return (uint64_t)page_or_0(tab[key >> a.page_shift]) * (a.kv_heads << a.page_shift) + (w.kvh << a.page_shift) + (key & pmask);
  }
  // First key of the wavefront's rows in a pass; past the last key, rows of its group again (masked).
  __device__ __forceinline__ int32_t start(int32_t kb, int p) const {
    const int32_t key = kb + wrow + p * (int32_t)kRows;
    return key < w.kend ? key : (w.kend - 1) & ~(int32_t)(kWaveRows - 1);
  }

  __device__ __forceinline__ void load_pages(int32_t (&page)[kPasses], int32_t& page_scale, int32_t kb) const {
    if constexpr (kPaged) {
#pragma unroll
      for (int p = 0; p < kPasses; ++p) page[p] = tab[start(kb, p) >> a.page_shift];
      if (kInt8 && wave < 2) page_scale = tab[min(kb + (int32_t)lane, w.kend - 1) >> a.page_shift];
    }
  }
  // Bytes from a plane's (a packed tensor's) start to the wavefront's rows of a pass, the same for K and V of a cache.
  __device__ __forceinline__ uint64_t offset(int32_t page, int32_t kb, int p, uint32_t ld) const {
    const int32_t key = start(kb, p);
    if constexpr (kPaged)
      return (uint64_t)page_or_0(__builtin_amdgcn_readfirstlane(page)) * page_bytes + (head_bytes + ((uint32_t)key & pmask) * (D * kElem));
    else
      return 2 * ((uint64_t)(uint32_t)(w.q.first + key) * ld + w.kvh * D);
  }
  // The lane's piece of its row, from there; rows of ld elements.  Of a packed sequence nothing past the last key is
  // read: the last row again.
  __device__ __forceinline__ uint32_t lane_offset(uint32_t ld) const {
    return kPaged ? 16 * lane : lane / kPieces * (2 * ld) + 16 * (lane % kPieces);
  }
  __device__ __forceinline__ uint32_t last_lane_offset(uint32_t ld, int32_t kb, int p) const {
    if constexpr (kWaveRows == 2) {   // nor is a branch needed: the second row is a step of zero away
      const uint32_t step = start(kb, p) + 1 < w.kend ? 2 * ld : 0;
      return (lane < 32 ? 0 : step) + 16 * (lane % 32);
    }
    return min(lane / kPieces, (uint32_t)(w.kend - 1 - start(kb, p))) * (2 * ld) + 16 * (lane % kPieces);
  }
  __device__ __forceinline__ bool is_last(int32_t kb) const { return !kPaged && kb + kKeys > w.kend; }
  __device__ __forceinline__ u32x4_t fetch(const void* plane, uint64_t at, uint32_t lane_at) const {
    return *reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(plane) + at + lane_at);
  }
  // wavefront 0: the keys' scales, wavefront 1: the values'; 0 on no page
  __device__ __forceinline__ float load_scale(int32_t page, int32_t kb) const {
    const uint32_t key = (uint32_t)min(kb + (int32_t)lane, w.kend - 1);
    const uint64_t row = (uint64_t)page_or_0(page) * (a.kv_heads << a.page_shift) + (w.kvh << a.page_shift) + (key & pmask);
    const float s = reinterpret_cast<const float*>(a.cache + (wave ? a.off_vs : a.off_ks))[row];
    return on_page(page) ? s : 0.f;
  }
  // A lane's place in a tile in LDS in pass 0; in pass p the row is p kRows further, which changes the exchange of K's
  // pieces only if kRows is no multiple of 16.
  template <bool V>
  __device__ __forceinline__ uint32_t place() const {
    const uint32_t row = (uint32_t)wrow + lane / kPieces, piece = lane % kPieces * (kInt8 ? 2 : 1);
    return row * kRowBytes + 16 * (V ? v_piece<D>(row, piece) : k_piece<D>(row, piece));
  }
  template <bool V>
  __device__ __forceinline__ void put(uint8_t* tile, uint32_t at, const u32x4_t (&r)[kPasses]) const {
    static_assert(D != 64 || kRows % 16 == 0, "rows of 64 elements share their exchange in pairs");
    if (kSpare && wrow >= kKeys) return;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      uint8_t* d = tile + p * kRows * kRowBytes;
      const uint32_t to = V ? at ^ 16 * (4 * (p * kRows % 4)) : at ^ 16 * (p * kRows % 16);
      if constexpr (kInt8) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const u32x2_t x = codes_to_bf16(r[p][2 * u]), y = codes_to_bf16(r[p][2 * u + 1]);
          *reinterpret_cast<u32x4_t*>(d + (to ^ 16 * u)) = u32x4_t{x[0], x[1], y[0], y[1]};
        }
      } else {
        *reinterpret_cast<u32x4_t*>(d + to) = r[p];
      }
    }
  }
  __device__ __forceinline__ bool at_edge(int32_t kb) const { return kb + kKeys - 1 > w.edge || !all_there; }
  // Tiles with keys that some rows do not see: infinities and NaN are taken out of the product, where a weight of
  // zero would make NaN of them, and the tile is marked (odd = kb + 1: nothing to clear) so that the rows
  // that do see them get them afterwards.
  __device__ __forceinline__ void clean_v(int32_t* odd, u32x4_t (&r)[kPasses], const bool (&there)[kPasses], int32_t kb) const {
    if constexpr (!kInt8) {
      if (at_edge(kb)) {
        uint32_t any = 0;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
          const bool real = kb + wrow + p * (int32_t)kRows + (int32_t)(lane / kPieces) < w.kend && there[p];
#pragma unroll
          for (int i = 0; i < 4; ++i) r[p][i] = real ? finite_pair(r[p][i], any) : 0u;
        }
        if (any) *odd = kb + 1;
      }
    }
  }
  __device__ __forceinline__ void put_scale(float (*tile)[kKeys], int32_t* odd, float s, int32_t kb) const {
    if (wave == 1 && at_edge(kb) && !(fabsf(s) < INFINITY)) {
      s = 0.f;
      *odd = kb + 1;
    }
    tile[wave][lane] = s;
  }
};

// The order of a run of products: operands are read from LDS kAhead products before
// they are used, where the scheduler alone would read them just before.  FIRST products take two
// reads each, then SECOND products one.  LOADS loads from memory go among them.
constexpr int kAhead = 4;
template <int FIRST, int SECOND, int LOADS = 0>
__device__ __forceinline__ void ahead() {
  constexpr int kProduct = 0x008, kRead = 0x100, kLoad = 0x020;
  constexpr auto reads = [](int i) { return i < FIRST ? 2 : i < FIRST + SECOND ? 1 : 0; };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    if (reads(i) == 2) __builtin_amdgcn_sched_group_barrier(kRead, 2, 0);
    if (reads(i) == 1) __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
  }
#pragma unroll
  for (int i = 0; i < FIRST + SECOND; ++i) {
    __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
    if (reads(i + kAhead) == 2) __builtin_amdgcn_sched_group_barrier(kRead, 2, 0);
    if (reads(i + kAhead) == 1) __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
    if (i % 3 == 2 && i / 3 < LOADS) __builtin_amdgcn_sched_group_barrier(kLoad, 1, 0);
  }
}

// A wavefront's 32 query rows and its part of the products.
template <int KIND, int D>
struct Rows32 {
  static constexpr bool kInt8 = KIND == kPagedInt8, kPaged = KIND != kPacked;
  static constexpr int kMT = D / 32, kRowBytes = 2 * D;
  bf16x8_t qf[D / 16];          // B operands: the rows
  uint32_t pf[kKeys / 16][4];   // B operands: the weights of a tile
  f32x16_t x[kKeys / 32], o[kMT];
  float m, l;
  int32_t last, row;            // the last key that the lane's row sees; its row (below 0: none)
  int32_t first_sees, last_sees;   // the last keys that the first and the last of the 32 rows see
  uint32_t hh, kat, vat[kMT];   // LDS offsets of the operands

  __device__ __forceinline__ void begin(const Attn& a, const Work& w, uint32_t wave, uint32_t lane) {
    const uint32_t n = lane & 31;
    hh = lane >> 5;
    const int32_t group = (int32_t)a.group, rb = w.row0 + 32 * (int32_t)wave, r = rb + (int32_t)n, i = r / group;
    const bool live = r < w.nrows;
    row = live ? r : -1;
    last = !live ? -1 : a.causal ? w.q.old + i : w.q.len - 1;
    first_sees = 0x7FFFFFFF;
    last_sees = -1;
    if (rb < w.nrows) {
      first_sees = a.causal ? w.q.old + rb / group : w.q.len - 1;
      last_sees = min(a.causal ? w.q.old + (min(rb + 32, w.nrows) - 1) / group : w.q.len - 1, w.q.len - 1);
    }
    const uint16_t* p = a.q + (uint64_t)(w.q.first + (live ? i : 0)) * a.ldq +
                        (uint64_t)(w.kvh * a.group + (live ? r - i * group : 0)) * D + 8 * hh;
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      u32x4_t q = *reinterpret_cast<const u32x4_t*>(p + 16 * st);
      q = live ? q ^ a.q_sign : u32x4_t{0, 0, 0, 0};
      qf[st] = as_bf16x8(q);
    }
    const uint32_t krow = 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);
    const uint32_t vi = lane & 15, vrow = 8 * hh + (vi >> 2);
    kat = krow * kRowBytes + 16 * k_piece<D>(krow, hh);   // piece 2 d + hh: an exclusive or with 32 d
#pragma unroll
    for (int e = 0; e < kMT; ++e)
      vat[e] = vrow * kRowBytes + 16 * v_piece<D>(vrow, 4 * e + 2 * ((lane >> 4) & 1) + ((vi & 3) >> 1)) + 8 * (vi & 1);
    m = kNoMax;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < kMT; ++e)
#pragma unroll
      for (int i2 = 0; i2 < 16; ++i2) o[e][i2] = 0.f;
  }
  // Wide heads fill both halves of the register file: the sums stay in the accumulation registers, where the products
  // add to them, the rows in the others (left to itself the allocator moves the sums to and fro in every tile).
  __device__ __forceinline__ void keep_places() {
    if constexpr (D > 128) {
#pragma unroll
      for (int d = 0; d < D / 16; ++d) asm volatile("" : "+v"(qf[d]));
#pragma unroll
      for (int e = 0; e < kMT; ++e) asm volatile("" : "+a"(o[e]));
    }
  }
  __device__ __forceinline__ bf16x8_t k_operand(const uint8_t* tile, int d, int h) const {
    const uint32_t low = (D == 64 ? 112u : 240u) & (32 * d), high = 32 * d - low;   // the pieces' exchanged bits
    return as_bf16x8(*reinterpret_cast<const u32x4_t*>(tile + (kat ^ low) + high + 32 * h * kRowBytes));
  }
  __device__ __forceinline__ bf16x8_t v_operand(const uint8_t* tile, int ks, int e) const {
    union { s16x4_t h[2]; bf16x8_t w; } v;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      v.h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(tile + vat[e] + (16 * ks + 4 * u) * kRowBytes));
    return v.w;
  }
  __device__ __forceinline__ bf16x8_t p_operand(int ks) const { return as_bf16x8(u32x4_t{pf[ks][0], pf[ks][1], pf[ks][2], pf[ks][3]}); }

  // value i of x belongs to key 16 (i / 8) + 8 hh + i % 8 of the tile
  __device__ __forceinline__ void score_products(const uint8_t* tile) {
#pragma unroll
    for (int h = 0; h < kKeys / 32; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[h][i] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int h = 0; h < kKeys / 32; ++h) x[h] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k_operand(tile, d, h), qf[d], x[h], 0, 0, 0);
  }
  __device__ __forceinline__ void sum_products(const uint8_t* tile) {
#pragma unroll
    for (int ks = 0; ks < kKeys / 16; ++ks)
#pragma unroll
      for (int e = 0; e < kMT; ++e)
        o[e] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v_operand(tile, ks, e), p_operand(ks), o[e], 0, 0, 0);
  }
  __device__ __forceinline__ void scores(const uint8_t* tile) {
    score_products(tile);
    ahead<0, D / 16 * (kKeys / 32)>();
  }
  __device__ __forceinline__ void sums(const uint8_t* tile) {
    sum_products(tile);
    ahead<kKeys / 16 * kMT, 0>();
  }
  template <int NW>
  __device__ __forceinline__ void weights(const Attn& a, const float (*scales)[kKeys], const Stage<KIND, D, NW>& st, int32_t kb) {
    if constexpr (kInt8) {
#pragma unroll
      for (int i = 0; i < kKeys / 2; i += 4) {
        const f32x4_t ks = *reinterpret_cast<const f32x4_t*>(&scales[0][16 * (i >> 3) + (i & 7) + 8 * hh]);
#pragma unroll
        for (int u = 0; u < 4; ++u) x[i >> 4][(i & 15) + u] *= ks[u];
      }
    }
    if (__builtin_amdgcn_readfirstlane(kb + kKeys - 1 > first_sees || !st.all_there)) {
      const int32_t most = last - kb - 8 * (int32_t)hh;
#pragma unroll
      for (int g = 0; g < kKeys / 16; ++g) {
        int32_t upto = most - 16 * g;
        if constexpr (kPaged)
          if (!st.all_there && (kb + 16 * g >= st.w.kend || !st.on_page(st.tab[(uint32_t)(kb + 16 * g) >> a.page_shift]))) upto = -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[g >> 1][8 * (g & 1) + i] = i <= upto ? x[g >> 1][8 * (g & 1) + i] : -INFINITY;
      }
    }
    float top4[4] = {kNoMax, kNoMax, kNoMax, kNoMax};
#pragma unroll
    for (int i = 0; i < kKeys / 2; i += 2) top4[i / 2 & 3] = fmaxf(fmaxf(top4[i / 2 & 3], x[i >> 4][i & 15]), x[i >> 4][(i & 15) + 1]);
    float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * a.scale;
    if (__any(top > m + kSlack)) {
      top = fmaxf(top, __shfl_xor(top, 32));
      const float mn = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
      if (D <= 128 || kb != st.w.k0) {   // before the first tile they are 0, and wide ones costly to move to and fro
#pragma unroll
        for (int e = 0; e < kMT; ++e) o[e] *= f;
      }
      keep_places();
    }
    float sum[4] = {};
#pragma unroll
    for (int i = 0; i < kKeys / 2; i += 4) {
      float y[4];
      f32x4_t vs;
      if constexpr (kInt8) vs = *reinterpret_cast<const f32x4_t*>(&scales[1][16 * (i >> 3) + (i & 7) + 8 * hh]);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        y[u] = __builtin_amdgcn_exp2f(fmaf(x[i >> 4][(i & 15) + u], a.scale, -m));
        sum[u] += y[u];
        if constexpr (kInt8) y[u] *= vs[u];
      }
      pf[i >> 3][(i & 7) >> 1] = pack_bf16(y[0], y[1]);
      pf[i >> 3][((i & 7) >> 1) + 1] = pack_bf16(y[2], y[3]);
    }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  }
  // The infinities and NaN of a marked tile, to the rows that see their keys (from memory: it is rare).
  template <int NW>
  __device__ __forceinline__ void odd_values(const Attn& a, const Work& w, const Stage<KIND, D, NW>& st, int32_t kb) {
    for (int32_t j = kb; j < kb + kKeys && j < w.kend; ++j) {
      keep_places();
      const uint8_t* p;
      float vs = 0.f;
      if constexpr (kPaged) {
        if (!st.on_page(st.tab[(uint32_t)j >> a.page_shift])) continue;
        const uint64_t r = st.row_index((uint32_t)j);
        p = a.cache + a.off_v + r * (D * (kInt8 ? 1 : 2));
        if constexpr (kInt8) vs = reinterpret_cast<const float*>(a.cache + a.off_vs)[r];
      } else {
        p = reinterpret_cast<const uint8_t*>(a.v + (uint64_t)(w.q.first + j) * a.ldv + w.kvh * D);
      }
#pragma unroll
      for (int e = 0; e < kMT; ++e)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float y;
          if constexpr (kInt8) y = vs;
          else y = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[32 * e + 8 * (i >> 2) + 4 * hh + (i & 3)] << 16);
          o[e][i] += j <= last && !(fabsf(y) < INFINITY) ? y : 0.f;
        }
    }
    keep_places();
  }
  __device__ __forceinline__ void finish(const Attn& a, const Work& w) {
    l += __shfl_xor(l, 32);
    if (a.n_splits == 1) {
      const int32_t at = max(row, 0), i = at / (int32_t)a.group;
      const float f = l == 0.f ? 0.f : 1.f / l;
      uint16_t* p = a.out + (uint64_t)(w.q.first + i) * a.ldo + (uint64_t)(w.kvh * a.group + at - i * (int32_t)a.group) * D + 8 * hh;
#pragma unroll
      for (int e = 0; e < kMT; ++e)
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
          // the halves of a row exchange four elements: eight neighbours, 16 bytes, in each
          uint32_t x[2], y[2];
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            x[v] = pack_bf16(o[e][4 * u + 2 * v] * f, o[e][4 * u + 2 * v + 1] * f);
            y[v] = pack_bf16(o[e][4 * u + 4 + 2 * v] * f, o[e][4 * u + 4 + 2 * v + 1] * f);
            const auto z = __builtin_amdgcn_permlane32_swap(x[v], y[v], false, false);
            x[v] = z[0];
            y[v] = z[1];
          }
          if (row >= 0) *reinterpret_cast<u32x4_t*>(p + 32 * e + 8 * u) = u32x4_t{x[0], x[1], y[0], y[1]};
        }
    } else if (row >= 0) {
      const uint64_t slot = part_row(a, w.sp, w.kvh, (uint64_t)w.q.first * a.group + row);
      float* p = a.part + slot * D + 4 * hh;
#pragma unroll
      for (int e = 0; e < kMT; ++e)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<f32x4_t*>(p + 32 * e + 8 * u) = f32x4_t{o[e][4 * u], o[e][4 * u + 1], o[e][4 * u + 2], o[e][4 * u + 3]};
      if (hh == 0) a.part_ml[slot] = make_float2(m, l);
    }
  }
};

// Few workgroups, or heads too wide for two wavefronts a SIMD: four wavefronts that go through a tile
// together; two workgroups on a compute unit overlap each other's products and exponentials.
template <int KIND, int D>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_attn_tile(Attn a) {
  using St = Stage<KIND, D, 4>;
  constexpr bool kInt8 = KIND == kPagedInt8;
  __shared__ __attribute__((aligned(256))) uint8_t ksh[2][kKeys * 2 * D], vsh[2][kKeys * 2 * D];
  __shared__ __attribute__((aligned(16))) float ssh[2][2][kKeys];
  __shared__ int32_t odd[2];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Work w;
  if (!find_work<KIND != kPacked>(a, 128, lane, w)) return;
  Rows32<KIND, D> r;
  St st(a, w, lane, wave);
  u32x4_t kr[St::kPasses], vr[St::kPasses];
  int32_t next_page[St::kPasses] = {}, next_scale = 0;
  bool there[St::kPasses];
  float scale = 0.f;
  const uint32_t klane = st.lane_offset((uint32_t)a.ldk), vlane = st.lane_offset((uint32_t)a.ldv);
  const uint32_t kplace = st.template place<false>(), vplace = st.template place<true>();
  const void* kplane = St::kPaged ? static_cast<const void*>(a.cache) : a.k;
  const void* vplane = St::kPaged ? static_cast<const void*>(a.cache + a.off_v) : a.v;
  auto load = [&](int32_t kb) {
#pragma unroll
    for (int p = 0; p < St::kPasses; ++p) {
      there[p] = !St::kPaged || st.on_page(next_page[p]);
      const uint64_t kat = st.offset(next_page[p], kb, p, (uint32_t)a.ldk);
      const uint64_t vat = St::kPaged ? kat : st.offset(next_page[p], kb, p, (uint32_t)a.ldv);
      const bool cut = !St::kPaged && (St::kWaveRows == 2 || st.is_last(kb));
      kr[p] = st.fetch(kplane, kat, cut ? st.last_lane_offset((uint32_t)a.ldk, kb, p) : klane);
      vr[p] = st.fetch(vplane, vat, cut ? st.last_lane_offset((uint32_t)a.ldv, kb, p) : vlane);
    }
    if (kInt8 && wave < 2) scale = st.load_scale(next_scale, kb);
    st.load_pages(next_page, next_scale, kb + kKeys);
  };
  auto store = [&](int b, int32_t kb) {
    st.template put<false>(ksh[b], kplace, kr);
    st.clean_v(&odd[b], vr, there, kb);
    st.template put<true>(vsh[b], vplace, vr);
    if (kInt8 && wave < 2) st.put_scale(ssh[b], &odd[b], scale, kb);
  };
  if (tid < 2) odd[tid] = 0;
  if (w.k0 < w.kend) {
    st.load_pages(next_page, next_scale, w.k0);
    load(w.k0);
  }
  r.begin(a, w, wave, lane);   // with the first keys on their way
  st.look_at_pages();
  lds_barrier();
  if (w.k0 < w.kend) {
    store(0, w.k0);
    load(w.k0 + kKeys);
  }
  lds_barrier();
  int b = 0;
  for (int32_t kb = w.k0; kb < w.kend; kb += kKeys, b ^= 1) {
    if (kb <= r.last_sees) {
      r.scores(ksh[b]);
      r.keep_places();
      r.weights(a, ssh[b], st, kb);
      r.keep_places();
      r.sums(vsh[b]);
      r.keep_places();
      if (st.at_edge(kb) && __builtin_amdgcn_readfirstlane(odd[b] == kb + 1)) r.odd_values(a, w, st, kb);
    }
    if (kb + kKeys < w.kend) {
      store(b ^ 1, kb + kKeys);
      if (kb + 2 * kKeys < w.kend) load(kb + 2 * kKeys);
    }
    lds_barrier();
  }
  r.finish(a, w);
}

// Many workgroups: eight wavefronts, the second four a step behind the first, so that on every SIMD one
// wavefront is in its products while the other is in its exponentials.  A step between two
// barriers is, for tile j and in turn, the products (V^T P^T of tile j - 1 and K Q^T of tile j), with the staging of K of
// tile j + 1 and V of tile j among them, or the weights of tile j.  The first four are in
// the products of tile j in step 2 j, the others in step 2 j + 1: a tile is whole when the first four need it, in step
// 2 j + 2, and the buffer it goes to was last read in step 2 j - 1.
template <int KIND, int D>
__global__ __launch_bounds__(512, 2) void k_attn_pair(Attn a) {
  using St = Stage<KIND, D, 8>;
  constexpr bool kInt8 = KIND == kPagedInt8;
  __shared__ __attribute__((aligned(256))) uint8_t ksh[2][kKeys * 2 * D], vsh[2][kKeys * 2 * D];
  __shared__ __attribute__((aligned(16))) float ssh[4][2][kKeys];
  __shared__ int32_t odd[4];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool behind = wave >> 2;
  Work w;
  if (!find_work<KIND != kPacked>(a, 256, lane, w)) return;
  Rows32<KIND, D> r;
  St st(a, w, lane, wave);
  u32x4_t kr[St::kPasses], vr[St::kPasses];
  int32_t next_page[St::kPasses] = {}, next_scale = 0;
  bool kthere[St::kPasses] = {}, vthere[St::kPasses] = {};
  uint64_t kat[St::kPasses] = {}, vat[St::kPasses] = {};
  float scale = 0.f;
  const int32_t tiles = max(w.kend - w.k0 + kKeys - 1, 0) / kKeys;
  const uint32_t klane = st.lane_offset((uint32_t)a.ldk), vlane = st.lane_offset((uint32_t)a.ldv);
  const uint32_t kplace = st.template place<false>(), vplace = st.template place<true>();
  const void* kplane = St::kPaged ? static_cast<const void*>(a.cache) : a.k;
  const void* vplane = St::kPaged ? static_cast<const void*>(a.cache + a.off_v) : a.v;
  auto key0 = [&](int32_t tile) { return w.k0 + tile * kKeys; };
  // K of a tile and V of the one before
  uint32_t kl[St::kPasses], vl[St::kPasses];   // (the lanes' offsets for it, cut at the end: apart, a branch among the products would part them)
  auto cut = [&](int32_t tile) {
#pragma unroll
    for (int p = 0; p < St::kPasses; ++p) {
      kl[p] = klane;
      vl[p] = vlane;
    }
    if (st.is_last(key0(tile))) {
#pragma unroll
      for (int p = 0; p < St::kPasses; ++p) {
        kl[p] = st.last_lane_offset((uint32_t)a.ldk, key0(tile), p);
        if (st.is_last(key0(tile - 1))) vl[p] = st.last_lane_offset((uint32_t)a.ldv, key0(tile - 1), p);
      }
    }
  };
  auto load = [&](int32_t tile, bool v) {
#pragma unroll
    for (int p = 0; p < St::kPasses; ++p) {
      if constexpr (St::kPaged) {
        vat[p] = kat[p];
        vthere[p] = kthere[p];
        kthere[p] = st.on_page(next_page[p]);
      } else {
        vat[p] = st.offset(0, key0(tile - 1), p, (uint32_t)a.ldv);
        vthere[p] = true;
      }
      kat[p] = st.offset(next_page[p], key0(tile), p, (uint32_t)a.ldk);
      kr[p] = st.fetch(kplane, kat[p], kl[p]);
      if (v) vr[p] = st.fetch(vplane, vat[p], vl[p]);
    }
  };
  auto load_rest = [&](int32_t tile) {
    if (kInt8 && wave < 2) scale = st.load_scale(next_scale, key0(tile));
    st.load_pages(next_page, next_scale, key0(tile + 1));
  };
  auto odd_tile = [&](int32_t tile) {
    if (st.at_edge(key0(tile)) && __builtin_amdgcn_readfirstlane(odd[tile & 3] == key0(tile) + 1)) r.odd_values(a, w, st, key0(tile));
  };
  if (tid < 4) odd[tid] = 0;
  // before tile 0: no values, no weights
  for (uint32_t i = tid; i < kKeys * 2 * D / 16; i += 512) reinterpret_cast<u32x4_t*>(vsh[1])[i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) r.pf[i / 4][i % 4] = 0;
  if (tiles) {
    st.load_pages(next_page, next_scale, w.k0);
    cut(0);
    load(0, false);
    load_rest(0);
  }
  r.begin(a, w, wave, lane);   // with the first keys on their way
  st.look_at_pages();
  lds_barrier();
  if (tiles) {
    st.template put<false>(ksh[0], kplace, kr);
    if (kInt8 && wave < 2) st.put_scale(ssh[0], &odd[0], scale, w.k0);
    cut(1);
    load(1, true);
    load_rest(1);
  }
  lds_barrier();
  if (behind) lds_barrier();
  for (int32_t j = 0; j < tiles; ++j) {
    const int32_t kb = key0(j);
    st.clean_v(&odd[j & 3], vr, vthere, kb);
    if (kInt8 && wave < 2) st.put_scale(ssh[(j + 1) & 3], &odd[(j + 1) & 3], scale, kb + kKeys);
    cut(j + 2);
    st.template put<false>(ksh[(j + 1) & 1], kplace, kr);
    st.template put<true>(vsh[j & 1], vplace, vr);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    r.sum_products(vsh[(j + 1) & 1]);
    r.score_products(ksh[j & 1]);
    load(j + 2, true);   // past the last tile: its last keys again
    ahead<4 * (D / 32), D / 8, 2 * St::kPasses>();
    __builtin_amdgcn_s_setprio(0);
    load_rest(j + 2);
    if (j) odd_tile(j - 1);
    lds_barrier();
    r.weights(a, ssh[j & 3], st, kb);
    lds_barrier();
  }
  if (!behind) lds_barrier();
  if (tiles) {
    r.sums(vsh[(tiles - 1) & 1]);
    odd_tile(tiles - 1);
  }
  r.finish(a, w);
}

// Tiles of `rows` query rows: every sequence's last may be a part of one.
uint64_t tiles_of(uint32_t n_seqs, uint32_t n, uint32_t max_new, uint32_t group, uint32_t rows) {
  const uint64_t each = ((uint64_t)max_new * group + rows - 1) / rows, all = (uint64_t)n * group / rows + n_seqs;
  return each * n_seqs < all ? each * n_seqs : all;
}

template <int KIND, int D>
int launch(const Attn& a, hipStream_t s) {
  const uint32_t rows = attn_tile_rows(a.n_seqs, a.n, a.max_new, a.group, a.kv_heads, D);
  const uint64_t blocks = attn_tiles(a.n_seqs, a.n, a.max_new, a.group, a.kv_heads, D) * a.kv_heads * a.n_splits;
  if (!launch_takes(blocks, rows == 256 ? 512 : 256)) return WAL_ERR_SHAPE;
  if constexpr (D <= 128) {
    if (rows == 256) {
      hipLaunchKernelGGL((k_attn_pair<KIND, D>), dim3((uint32_t)blocks), dim3(512), 0, s, a);
      return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
    }
  }
  hipLaunchKernelGGL((k_attn_tile<KIND, D>), dim3((uint32_t)blocks), dim3(256), 0, s, a);
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}

template <int KIND>
int launch(const Attn& a, uint32_t dim, hipStream_t s) {
  if (dim == 64) return launch<KIND, 64>(a, s);
  if (dim == 128) return launch<KIND, 128>(a, s);
  return launch<KIND, 256>(a, s);
}

}  // namespace

namespace wal {

// Eight wavefronts of 32 rows when that gives every compute unit a workgroup (prompt of 8192 tokens, 32 query and 8
// key/value heads of 128: 515 us, and 590 with four), else four; wide heads have room for four only.
uint32_t attn_tile_rows(uint32_t n_seqs, uint32_t n, uint32_t max_new, uint32_t group, uint32_t kv_heads, uint32_t dim) {
  return dim <= 128 && tiles_of(n_seqs, n, max_new, group, 256) * kv_heads >= 256 ? 256 : 128;
}

uint64_t attn_tiles(uint32_t n_seqs, uint32_t n, uint32_t max_new, uint32_t group, uint32_t kv_heads, uint32_t dim) {
  return tiles_of(n_seqs, n, max_new, group, attn_tile_rows(n_seqs, n, max_new, group, kv_heads, dim));
}

int attn_tile(const Attn& a, int kind, uint32_t dim, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (kind == kPacked) return launch<kPacked>(a, dim, s);
  return kind == kPagedInt8 ? launch<kPagedInt8>(a, dim, s) : launch<kPagedBf16>(a, dim, s);
}

}  // namespace wal
