// The gated delta rule on chunks of 64 tokens for gfx950 (prompts).  With G_i the
// sum of the logarithms of the decays of a chunk's tokens up to i, S0 the state
// before it and u_i the rows that its tokens store,
//     u = T (diag(b) V - diag(b e^G) K S0),    T = (1 + A)^-1,
//         A_ij = b_i e^(G_i - G_j) k_i . k_j   (j < i)
//     O = diag(e^G) Q S0 + P u,    P_ij = e^(G_i - G_j) q_i . k_j   (j <= i)
//     S = e^G_end S0 + K^T diag(e^(G_end - G)) u
// so that tokens meet in products on the matrix cores and only states go from chunk
// to chunk.  k_delta_chunk makes T, P and the factors of the rows of every chunk and head, all of
// them at once; k_delta_scan walks the chunks of a sequence and head, a wavefront
// keeping 16 columns of the state in registers: everything that a column of the
// values meets belongs to that column alone.
//
// Numbers.  q, k and v are bf16 and go into the products as they are, the norms of q and k into
// the rows' factors.  What is fp32 (states, T, the rows b V - .., u) enters a product in
// parts of 8 bits, x = hi + mid + lo: three make a state's update as exact as fp32, two do for
// what only outputs in bf16 see.  G is added up in 64 bits, because e^(G_i - G_j) has to
// be exact also after a token that forgets everything.  Exponents are never above 0.
//
// Not finite.  A product with T would carry a NaN of row j into rows above j, as 0 * NaN.  From
// a chunk's first token on whose key or gates are not finite, rows are taken out of A and their
// factors are NaN; k_delta_scan looks at one row of u of each 32, and where it is not
// finite takes the rows that are not out of the product and puts NaN where they belong.
#include <hip/hip_runtime.h>

#include "wal_delta.h"

namespace {

constexpr int kC = kChunk;
constexpr uint32_t kLd = kC + 4;       // of T in LDS: four 16 x 16 blocks of the diagonal on different banks
constexpr uint32_t kBlockBytes = 1024; // an operand of a matrix instruction: 16 bytes a lane
constexpr uint32_t kBlocks = 6;        // of a 64 x 64 lower triangle, as (32-row block, half, 32-column block)
constexpr float kForget = -1000.f;     // logarithms of decays below this one are it: e^-1000 is 0

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// Rows 32 u + 8 (m / 4) + 4 h + m % 4 of operand (u, h): lane group c of a result holds rows 8 c + 4 h + i, and the two
// halves make the eight rows 8 c .. of a B operand.
__device__ __forceinline__ uint32_t dealt(uint32_t u, uint32_t h, uint32_t m) { return 32 * u + 8 * (m >> 2) + 4 * h + (m & 3); }

__device__ __forceinline__ bf16x8_t as_operand(u32x4_t w) { return __builtin_bit_cast(bf16x8_t, w); }

// Eight values as N parts of 8 bits: x = p[0] + p[1] + ..
template <int N>
__device__ __forceinline__ void split(const float (&x)[8], bf16x8_t (&p)[N]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x2_t b = {(__bf16)r[2 * i], (__bf16)r[2 * i + 1]};   // to nearest even
      w[i] = __builtin_bit_cast(uint32_t, b);
      if (k + 1 < N) {
        r[2 * i] -= __uint_as_float(w[i] << 16);
        r[2 * i + 1] -= __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    p[k] = as_operand(w);
  }
}
template <int N>
__device__ __forceinline__ void split(f32x4_t x, f32x4_t y, bf16x8_t (&p)[N]) {
  const float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  split(z, p);
}

// The sequence of a chunk's place: sequence s has those from starts[s] / 64 + s on.
__device__ __forceinline__ uint32_t seq_of_place(const Delta& a, uint32_t place, uint32_t lane) {
  uint32_t lo = 0, span = a.n_seqs;
  while (span > 1) {
    const uint32_t step = (span + 63) / 64, i = lane * step;
    const bool before = i < span && (uint32_t)between(a.starts[lo + i], 0, (int32_t)a.n) / kC + lo + i <= place;
    const uint32_t k = (uint32_t)max(__builtin_popcountll(__ballot(before)), 1) - 1;
    lo += k * step;
    span = min(step, span - k * step);
  }
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)lo);
}

// Place of a row's 16-byte piece in LDS, in k_delta_chunk (16 rows side by side are read together) ..
template <int DK>
__device__ __forceinline__ uint32_t row_piece(uint32_t r, uint32_t p) {
  return r * (2 * DK) + 16 * (DK == 128 ? p ^ (r & 15) : p ^ ((r >> 1) & 7));
}
// .. and in k_delta_scan, where it is the rows of dealt(), and by the transposing reads four neighbours.
template <int DK>
__device__ __forceinline__ uint32_t dealt_piece(uint32_t r, uint32_t p) {
  return r * (2 * DK) + 16 * (DK == 128 ? p ^ ((r & 3) << 2 | ((r >> 3) & 3)) : p ^ (((r >> 1) & 1) << 2 | ((r >> 3) & 3)));
}

// Four elements of a 16 x 16 tile (row 4 c + i, column n) of the product of 16 rows each.
template <int DK>
__device__ __forceinline__ f32x4_t tile_product(const uint8_t* x, const uint8_t* y, uint32_t it, uint32_t jt, uint32_t n, uint32_t c) {
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < DK / 32; ++s) {
    const u32x4_t xa = *reinterpret_cast<const u32x4_t*>(x + row_piece<DK>(16 * it + n, 4 * s + c));
    const u32x4_t yb = *reinterpret_cast<const u32x4_t*>(y + row_piece<DK>(16 * jt + n, 4 * s + c));
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_operand(xa), as_operand(yb), acc, 0, 0, 0);
  }
  return acc;
}

// acc += X Y of 16 x 16 blocks of LDS in fp32.
__device__ __forceinline__ f32x4_t block_product(const float (*t)[kLd], uint32_t xr, uint32_t xc, uint32_t yr, uint32_t yc, uint32_t n,
                                                 uint32_t c, f32x4_t acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(t[16 * xr + n][16 * xc + 4 * s + c], t[16 * yr + 4 * s + c][16 * yc + n], acc, 0, 0, 0);
  return acc;
}
// The same with Y such a result: the index added over is dealt as its rows are.
__device__ __forceinline__ f32x4_t block_product(const float (*t)[kLd], uint32_t xr, uint32_t xc, f32x4_t y, uint32_t n, uint32_t c,
                                                 f32x4_t acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(t[16 * xr + n][16 * xc + 4 * c + s], y[s], acc, 0, 0, 0);
  return acc;
}

// Eight values of a lower triangle in the order of operand block b.
__device__ __forceinline__ void operand_values(const float (*t)[kLd], uint32_t b, uint32_t l, float (&x)[8]) {
  const uint32_t u = b >> 1 > 0, s = b >> 1 > 1, row = dealt(u, b & 1, l & 15), col = 32 * s + 8 * (l >> 4);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4_t w = *reinterpret_cast<const f32x4_t*>(&t[row][col + 4 * i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[4 * i + j] = w[j];
  }
}

template <int DK>
__global__ __launch_bounds__(256) void k_delta_chunk(Delta a) {
  constexpr uint32_t kPieces = DK / 8, kRows = 256 / kPieces;
  constexpr uint32_t kRaw = 2 * kC * DK * 2, kMat = kC * kLd * 4;
  __shared__ __attribute__((aligned(256))) uint8_t raw[kRaw > kMat ? kRaw : kMat];
  __shared__ __attribute__((aligned(16))) float t[kC][kLd];
  __shared__ double far[kC];
  __shared__ float kk[kC], qq[kC], beta_sh[kC], rk_sh[kC], rq_sh[kC];
  __shared__ uint32_t first_bad;
  uint8_t *ks = raw, *qs = raw + kRaw / 2;
  float(*p)[kLd] = reinterpret_cast<float(*)[kLd]>(raw);
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, c = lane >> 4;
  const uint32_t h = blockIdx.x % a.heads, local = blockIdx.x / a.heads, place = a.place0 + local;
  const uint32_t s = seq_of_place(a, place, lane);
  const Seq q = delta_seq(a, s);
  const int32_t row0 = kC * (int32_t)(place - ((uint32_t)q.first / kC + s));   // of the sequence
  if (row0 < 0 || row0 >= q.rows) return;
  const int32_t count = min(q.rows - row0, kC);
  const uint64_t from = (uint64_t)(q.first + row0);
  const uint32_t kh = h / a.group;

  u32x4_t kr[kC / kRows], qr[kC / kRows];
#pragma unroll
  for (int i = 0; i < (int)(kC / kRows); ++i) {
    const int32_t r = (int32_t)(tid / kPieces + i * kRows);
    const uint64_t at = from + min(r, count - 1);
    kr[i] = *reinterpret_cast<const u32x4_t*>(a.k + at * a.ldk + kh * DK + 8 * (tid % kPieces));
    qr[i] = *reinterpret_cast<const u32x4_t*>(a.q + at * a.ldq + kh * DK + 8 * (tid % kPieces));
  }
  float beta = 0.f;
  if (wave == 0) {
    const bool there = (int32_t)lane < count;
    const Gates g = gates_of(a, from + min((int32_t)lane, count - 1), h);
    beta = there ? g.beta : 0.f;
    double x = !there ? 0.0 : g.log_alpha < kForget ? (double)kForget : (double)g.log_alpha;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double y = __shfl_up(x, d);
      if (lane >= (uint32_t)d) x += y;
    }
    far[lane] = x;
  }
#pragma unroll
  for (int i = 0; i < (int)(kC / kRows); ++i) {
    const uint32_t r = tid / kPieces + i * kRows, piece = tid % kPieces;
    if ((int32_t)r >= count) kr[i] = qr[i] = u32x4_t{0, 0, 0, 0};
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float k0 = __uint_as_float(kr[i][j] << 16), k1 = __uint_as_float(kr[i][j] & 0xFFFF0000u);
      const float q0 = __uint_as_float(qr[i][j] << 16), q1 = __uint_as_float(qr[i][j] & 0xFFFF0000u);
      x = fmaf(k1, k1, fmaf(k0, k0, x));
      y = fmaf(q1, q1, fmaf(q0, q0, y));
    }
#pragma unroll
    for (int d = 1; d < (int)kPieces; d *= 2) {
      x += __shfl_xor(x, d);
      y += __shfl_xor(y, d);
    }
    if (piece == 0) {
      kk[r] = x;
      qq[r] = y;
    }
    *reinterpret_cast<u32x4_t*>(ks + row_piece<DK>(r, piece)) = kr[i];
    *reinterpret_cast<u32x4_t*>(qs + row_piece<DK>(r, piece)) = qr[i];
  }
  __syncthreads();

  // the ten tiles of the lower triangle, of A and of P
  uint8_t* item = a.ws + (uint64_t)(local * a.heads + h) * kItemBytes;
  f32x4_t ak[3], pk[3];
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const uint32_t tile = wave + 4 * x, it = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0, jt = tile - it * (it + 1) / 2;
    if (tile >= 10) continue;
    ak[x] = tile_product<DK>(ks, ks, it, jt, n, c);
    pk[x] = tile_product<DK>(qs, ks, it, jt, n, c);
  }
  if (wave == 0) {
    const double g = far[lane], end = far[kC - 1];
    const bool there = (int32_t)lane < count;
    const float kn = kk[lane], rk = there ? unit(a, kn) : 0.f, rq = there ? unit(a, qq[lane]) * a.scale : 0.f;
    const bool bad = !(fabsf(kn) < INFINITY) || !(fabsf(beta) < INFINITY) || g != g;
    const uint64_t any = __ballot(bad);
    const uint32_t f = any ? (uint32_t)__builtin_ctzll(any) : (uint32_t)kC;
    const float lost = lane >= f ? NAN : 0.f, gone = any ? NAN : 0.f;
    const float decay = expf((float)g);
    float* vec = reinterpret_cast<float*>(item + kVecAt);
    vec[lane] = beta + lost;
    vec[kC + lane] = beta * decay * rk + lost;
    vec[2 * kC + lane] = expf((float)(end - g)) * rk + gone;
    vec[3 * kC + lane] = decay * rq + lost;
    if (lane == 0) {
      vec[4 * kC] = expf((float)end) + gone;
      first_bad = f;
    }
    beta_sh[lane] = beta;
    rk_sh[lane] = rk;
    rq_sh[lane] = rq;
  }
  __syncthreads();   // K and Q are read: P goes to their place
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const uint32_t tile = wave + 4 * x, it = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0, jt = tile - it * (it + 1) / 2;
    if (tile >= 10) continue;
    const uint32_t col = 16 * jt + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t row = 16 * it + 4 * c + i;
      const float e = expf((float)(far[row] - far[col])) * rk_sh[col];
      t[row][col] = col < row && row < first_bad ? beta_sh[row] * rk_sh[row] * e * ak[x][i] : 0.f;
      p[row][col] = col <= row ? rq_sh[row] * e * pk[x][i] : 0.f;
    }
  }
  if (wave >= 2) {   // tiles (0, 1) and (2, 3): nothing
    const uint32_t row = 32 * (wave - 2) + n, col = 32 * (wave - 2) + 16 + 4 * c;
    *reinterpret_cast<f32x4_t*>(&t[row][col]) = f32x4_t{0.f, 0.f, 0.f, 0.f};
    *reinterpret_cast<f32x4_t*>(&p[row][col]) = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  __syncthreads();

  if (wave == 0) {
    // the inverses of the four blocks of the diagonal, a column a lane, row after row
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float y[2] = {i == (int)n ? 1.f : 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const f32x4_t w = *reinterpret_cast<const f32x4_t*>(&t[16 * c + i][16 * c + j]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < i) y[e & 1] = fmaf(-w[e], x[j + e], y[e & 1]);
      }
      x[i] = y[0] + y[1];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) t[16 * c + i][16 * c + n] = x[i];
  } else {
    for (uint32_t i = tid - 64; i < kBlocks * 64; i += 192) {
      float x[8];
      bf16x8_t w[kPParts];
      operand_values(p, i >> 6, i & 63, x);
      split(x, w);
#pragma unroll
      for (int k = 0; k < kPParts; ++k)
        *reinterpret_cast<bf16x8_t*>(item + kPAt + k * (kBlocks * kBlockBytes) + 16 * i) = w[k];
    }
  }
  __syncthreads();
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  if (wave < 2) {   // blocks (1, 0) and (3, 2)
    const uint32_t r = 2 * wave + 1, b = 2 * wave;
    const f32x4_t y = block_product(t, r, b, b, b, n, c, zero), z = block_product(t, r, r, y, n, c, zero);
#pragma unroll
    for (int i = 0; i < 4; ++i) t[16 * r + 4 * c + i][16 * b + n] = -z[i];
  }
  __syncthreads();
  f32x4_t lower[2];
  if (wave < 2) {   // column `wave` of the lower left 32 x 32
    f32x4_t y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      y[i] = wave == 0 ? block_product(t, 2 + i, 0, 0, 0, n, c, zero) : zero;
      y[i] = block_product(t, 2 + i, 1, 1, wave, n, c, y[i]);
    }
    lower[0] = block_product(t, 2, 2, y[0], n, c, zero);
    lower[1] = block_product(t, 3, 3, y[1], n, c, block_product(t, 3, 2, y[0], n, c, zero));
  }
  __syncthreads();
  if (wave < 2)
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) t[16 * (2 + k) + 4 * c + i][16 * wave + n] = -lower[k][i];
  __syncthreads();
  for (uint32_t i = tid; i < kBlocks * 64; i += 256) {
    float x[8];
    bf16x8_t w[kTParts];
    operand_values(t, i >> 6, i & 63, x);
    split(x, w);
#pragma unroll
    for (int k = 0; k < kTParts; ++k) *reinterpret_cast<bf16x8_t*>(item + k * (kBlocks * kBlockBytes) + 16 * i) = w[k];
  }
}

constexpr int kScanGroups = 2;   // groups of 16 columns of a workgroup

// Rows of a chunk in memory: what lies behind the last one reads as zeros and is not written.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rows(const uint16_t* p, uint64_t ld, int32_t count, uint32_t width) {
  return rsrc(p, (uint32_t)(2 * ((uint64_t)(count - 1) * ld + width)));
}

// Two wavefronts share 16 columns, each on a SIMD of its own: the first takes the states from chunk to chunk, which is
// what a sequence waits for, the second, a chunk behind, makes the outputs from the states and rows that the first leaves in
// LDS as operands, and brings the next K.  (One wavefront for both: 559 us instead of @@ us for a prompt of 8192 tokens.)
template <int DK>
struct Scan {
  static constexpr int U = DK / 32;                       // 32-row blocks of the state
  static constexpr uint32_t kPieces = DK / 8, kRows = 64 * kScanGroups / kPieces;
  static constexpr int kPasses = kC / (int)kRows;
  struct Shared {
    __attribute__((aligned(256))) uint8_t k[2][kC * DK * 2];
    u32x4_t parts[2][kScanGroups][U][2][64];              // of the states before a chunk
    f32x4_t u[2][kScanGroups][2][2][64];
    __attribute__((aligned(16))) float vec[2][4 * kC];
    int32_t bad[2][kScanGroups][16];                      // the first of a column's rows that is not finite
  };
  const Delta& a;
  Shared& sh;
  const Seq q;
  const uint32_t base, h, kh, col, lane, n, c, group;
  const int32_t j0, j1;

  __device__ __forceinline__ const uint8_t* item_of(int32_t j) const {
    return a.ws + ((uint64_t)(base + (uint32_t)j - a.place0) * a.heads + h) * kItemBytes;
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const uint16_t* p, uint64_t ld, int32_t j, uint32_t at, uint32_t width) const {
    return chunk_rows(p + (uint64_t)(q.first + j * kC) * ld + at, ld, min(q.rows - j * kC, kC), width);
  }

  // The first wavefront: u and the state after each chunk.  What a chunk needs is loaded a chunk ahead, each part when
  // the one before is used.  Runs of products go over their tiles first, so that none waits for the one before.
  __device__ __forceinline__ void states(const float* before, float* after) {
    const uint32_t dv = a.value_dim, ldv = (uint32_t)a.ldv, vlane = 2 * (8 * c * ldv + col);
    f32x4_t st[U][2];   // element i: row 32 u + 8 c + 4 h + i
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < 4; ++i) st[u][hf][i] = before ? before[(uint64_t)(32 * u + 4 * hf + i) * dv] : 0.f;
    // Lanes' places in K: of rows dealt(0, 0, n), and for the transposing reads; a 32-column block further is an exclusive
    // or with 64 bytes, and rows 4 hf and 32 w further change no bits that the pieces' exchange looks at.
    const uint32_t kat = dealt_piece<DK>(dealt(0, 0, n), c), tat = dealt_piece<DK>(8 * c + (n >> 2), n & 3);
    u32x4_t tw[kTParts][kBlocks];
    uint16_t v[2][2][4];
    const auto load_t = [&](int32_t j) {
#pragma unroll
      for (int e = 0; e < kTParts; ++e)
#pragma unroll
        for (int i = 0; i < (int)kBlocks; ++i) tw[e][i] = *reinterpret_cast<const u32x4_t*>(item_of(j) + (e * kBlocks + i) * kBlockBytes + 16 * lane);
    };
    const auto load_v = [&](int32_t j) {
      const __amdgpu_buffer_rsrc_t r = rows_of(a.v, a.ldv, j, h * dv, dv);
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[w][hf][i] = __builtin_amdgcn_raw_buffer_load_b16(r, vlane + (32 * w + 4 * hf + i) * 2 * ldv, 0, 0);
    };
    load_v(j0);
    load_t(j0);
    lds_barrier();
    for (int32_t j = j0; j < j1; ++j) {
      const float decay = *reinterpret_cast<const __attribute__((address_space(4))) float*>(
          reinterpret_cast<uintptr_t>(item_of(j) + kVecAt + 16 * kC));
      const uint8_t* k = sh.k[j & 1];
      const float* vec = sh.vec[j & 1];
      const int32_t next = min(j + 1, j1 - 1);
      // the state in parts, and K S
      f32x4_t ks[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) ks[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        bf16x8_t part[3], kw[4];
        split(st[u][0], st[u][1], part);
#pragma unroll
        for (int e = 0; e < 2; ++e) sh.parts[j & 1][group][u][e][lane] = __builtin_bit_cast(u32x4_t, part[e]);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          kw[t] = as_operand(*reinterpret_cast<const u32x4_t*>(k + (kat ^ 64 * u) + (16 * (t & 2) + 4 * (t & 1)) * 2 * DK));
#pragma unroll
        for (int e = 2; e >= 0; --e)
#pragma unroll
          for (int t = 0; t < 4; ++t) ks[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kw[t], part[e], ks[t], 0, 0, 0);
      }
      // the rows b V - b e^G K S0
      f32x4_t rows[2][2];
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t r = 32 * w + 8 * c + 4 * hf;
          const f32x4_t c1 = *reinterpret_cast<const f32x4_t*>(vec + r), c2 = *reinterpret_cast<const f32x4_t*>(vec + kC + r);
#pragma unroll
          for (int i = 0; i < 4; ++i) rows[w][hf][i] = fmaf(-c2[i], ks[2 * w + hf][i], c1[i] * bf16_value(v[w][hf][i]));
        }
      load_v(next);
      f32x4_t u[2][2];
      const auto solve = [&] {
        bf16x8_t part[2][3];
#pragma unroll
        for (int w = 0; w < 2; ++w) split(rows[w][0], rows[w][1], part[w]);
#pragma unroll
        for (int t = 0; t < 4; ++t) u[t / 2][t % 2] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 2; e >= 0; --e)   // parts whose product is 2^-16, 2^-8 and 1 of the whole
#pragma unroll
          for (int f = 0; f <= e; ++f)
#pragma unroll
            for (int b = 0; b < (int)kBlocks; ++b) {
              const int w = b > 1, sb = b > 3, hf = b & 1;
              u[w][hf] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_operand(tw[f][b]), part[sb][e - f], u[w][hf], 0, 0, 0);
            }
      };
      solve();
      int32_t bad = kC;
      if (__any(!(fabsf(u[0][0][0]) < INFINITY) || !(fabsf(u[1][0][0]) < INFINITY))) {
#pragma unroll
        for (int w = 1; w >= 0; --w)
#pragma unroll
          for (int hf = 1; hf >= 0; --hf)
#pragma unroll
            for (int i = 3; i >= 0; --i)
              if (!(fabsf(rows[w][hf][i]) < INFINITY)) {
                bad = 32 * w + 8 * (int32_t)c + 4 * hf + i;
                rows[w][hf][i] = 0.f;
              }
        bad = min(bad, __shfl_xor(bad, 16));
        bad = min(bad, __shfl_xor(bad, 32));
        solve();
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (32 * w + 8 * (int32_t)c + 4 * hf + i >= bad) u[w][hf][i] = 0.f;
      }
      load_t(next);
      if (c == 0) sh.bad[j & 1][group][n] = bad;
      // S = decay S + K^T diag(e^(G_end - G)) u
      bf16x8_t up[2][3];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        f32x4_t y[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          sh.u[j & 1][group][w][hf][lane] = u[w][hf];
          y[hf] = *reinterpret_cast<const f32x4_t*>(vec + 2 * kC + 32 * w + 8 * c + 4 * hf) * u[w][hf];
        }
        split(y[0], y[1], up[w]);
      }
#pragma unroll
      for (int ub = 0; ub < U; ++ub)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) st[ub][hf] *= decay;
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int ub = 0; ub < U; ub += 2) {
          union { s16x4_t half[2]; bf16x8_t all; } kt[4];   // four tokens of the lane's row of K^T each
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int z = 0; z < 2; ++z)
              kt[t].half[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (lds_s16x4_t*)(k + (tat ^ 64 * (ub + t / 2)) + (32 * w + 4 * z) * 2 * DK + 8 * (t % 2)));
#pragma unroll
          for (int e = 2; e >= 0; --e)
#pragma unroll
            for (int t = 0; t < 4; ++t)
              st[ub + t / 2][t % 2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kt[t].all, up[w][e], st[ub + t / 2][t % 2], 0, 0, 0);
        }
      if (__any(bad < kC)) {
#pragma unroll
        for (int ub = 0; ub < U; ++ub)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int i = 0; i < 4; ++i) st[ub][hf][i] = bad < kC ? NAN : st[ub][hf][i];
      }
      lds_barrier();
    }
    if (after)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int i = 0; i < 4; ++i) after[(uint64_t)(32 * u + 4 * hf + i) * dv] = st[u][hf][i];
  }

  // The second wavefront: K of the chunk after, and the outputs of the chunk before, O = diag(e^G) Q S0 + P u.
  __device__ __forceinline__ void outputs() {
    const uint32_t dv = a.value_dim, ldq = (uint32_t)a.ldq, ldk = (uint32_t)a.ldk, ldo = (uint32_t)a.ldo, tid = 64 * group + lane;
    const uint32_t klane = 2 * (tid / kPieces * ldk + 8 * (tid % kPieces)), olane = 2 * (8 * c * ldo + col), qlane = 2 * (dealt(0, 0, n) * ldq + 8 * c);
    u32x4_t kr[kPasses], pw[kPParts][kBlocks], qw[4][U];
    f32x4_t c4[4];
    float2 vr;
    const auto load_k = [&](int32_t j) {
      const __amdgpu_buffer_rsrc_t r = rows_of(a.k, a.ldk, j, kh * DK, DK);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) kr[i] = __builtin_amdgcn_raw_buffer_load_b128(r, klane + i * kRows * 2 * ldk, 0, 0);
      vr = *reinterpret_cast<const float2*>(item_of(j) + kVecAt + 8 * tid);
    };
    const auto store_k = [&](int b) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        *reinterpret_cast<u32x4_t*>(sh.k[b] + dealt_piece<DK>(tid / kPieces + i * kRows, tid % kPieces)) = kr[i];
      *reinterpret_cast<float2*>(&sh.vec[b][2 * tid]) = vr;
    };
    const auto load_q = [&](int32_t j) {
      const __amdgpu_buffer_rsrc_t r = rows_of(a.q, a.ldq, j, kh * DK, DK);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int u = 0; u < U; ++u) qw[t][u] = __builtin_amdgcn_raw_buffer_load_b128(r, qlane + (16 * (t & 2) + 4 * (t & 1)) * 2 * ldq + 64 * u, 0, 0);
        c4[t] = *reinterpret_cast<const f32x4_t*>(item_of(j) + kVecAt + 4 * (3 * kC + 16 * (t & 2) + 8 * c + 4 * (t & 1)));
      }
    };
    const auto load_p = [&](int32_t j) {
#pragma unroll
      for (int e = 0; e < kPParts; ++e)
#pragma unroll
        for (int i = 0; i < (int)kBlocks; ++i)
          pw[e][i] = *reinterpret_cast<const u32x4_t*>(item_of(j) + kPAt + (e * kBlocks + i) * kBlockBytes + 16 * lane);
    };
    load_k(j0);
    store_k(j0 & 1);
    lds_barrier();
    load_k(min(j0 + 1, j1 - 1));
    load_p(j0);
    load_q(j0);
    store_k((j0 + 1) & 1);
    load_k(min(j0 + 2, j1 - 1));
    lds_barrier();
    for (int32_t j = j0; j < j1; ++j) {
      // the states' wavefront is at chunk j + 1, whose K is there
      f32x4_t o[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      store_k(j & 1);   // of chunk j + 2: all are done with chunk j's
      load_k(min(j + 3, j1 - 1));
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 1; e >= 0; --e) {
          const bf16x8_t part = as_operand(sh.parts[j & 1][group][u][e][lane]);
#pragma unroll
          for (int t = 0; t < 4; ++t) o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_operand(qw[t][u]), part, o[t], 0, 0, 0);
        }
      bf16x8_t part[2][2];
#pragma unroll
      for (int w = 0; w < 2; ++w) split(sh.u[j & 1][group][w][0][lane], sh.u[j & 1][group][w][1][lane], part[w]);
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] *= c4[t];
      load_q(min(j + 1, j1 - 1));
#pragma unroll
      for (int e = 1; e >= 0; --e)
#pragma unroll
        for (int f = 0; f <= e; ++f)
#pragma unroll
          for (int i = 0; i < (int)kBlocks; ++i) {
            const int t = 2 * (i > 1) + (i & 1);
            o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_operand(pw[f][i]), part[i > 3][e - f], o[t], 0, 0, 0);
          }
      load_p(min(j + 1, j1 - 1));
      const int32_t bad = sh.bad[j & 1][group][n];
      const __amdgpu_buffer_rsrc_t r = rows_of(a.out, a.ldo, j, h * dv, dv);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t row = 16 * (t & 2) + 4 * (t & 1) + i;
          __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)((int32_t)(row + 8 * c) >= bad ? NAN : o[t][i])), r,
                                                olane + row * 2 * ldo, 0, 0);
        }
      if (j + 1 < j1) lds_barrier();   // (the other wavefronts have met here once less)
    }
  }
};

template <int DK>
__global__ __launch_bounds__(128 * kScanGroups, 1) void k_delta_scan(Delta a) {
  __shared__ typename Scan<DK>::Shared sh;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, c = lane >> 4;
  const uint32_t group = wave % kScanGroups;
  // The workgroups of a head sit on one chiplet, so that its cache serves what they share: blocks go to the eight
  // chiplets in turn.
  const uint32_t x = blockIdx.x % 8, g = blockIdx.x / 8, pair = g / a.slices * 8 + x;
  if (pair >= a.n_seqs * a.heads) return;
  const uint32_t s = pair / a.heads, h = pair % a.heads, col = kSlice * (g % a.slices) + 16 * group + n;
  const Seq q = delta_seq(a, s);
  const uint32_t base = (uint32_t)q.first / kC + s;
  const int32_t chunks = (q.rows + kC - 1) / kC;
  const int32_t j0 = max(0, (int32_t)a.place0 - (int32_t)base), j1 = min(chunks, (int32_t)(a.place0 + a.places) - (int32_t)base);
  if (j0 >= j1) return;
  const int64_t slot = kept_at(a, s);
  const uint64_t head_at = ((uint64_t)h * DK + 8 * c) * a.value_dim + col;
  float* kept = slot < 0 ? nullptr : a.state + (uint64_t)slot * a.heads * DK * a.value_dim + head_at;
  Scan<DK> scan{a, sh, q, base, h, h / a.group, col, lane, n, c, group, j0, j1};
  if (wave < kScanGroups) scan.states(j0 ? a.carry[0] + head_at : kept, j1 < chunks ? a.carry[1] + head_at : kept);
  else scan.outputs();
}

template <int DK>
int launch(Delta& a, uint32_t all, hipStream_t s) {
  float* carry[2] = {a.carry[0], a.carry[1]};
  for (uint32_t first = 0, i = 0; first < all; first += a.places, ++i) {
    a.place0 = first;
    a.carry[0] = carry[i % 2];
    a.carry[1] = carry[(i + 1) % 2];
    const uint64_t items = (uint64_t)(all - first < a.places ? all - first : a.places) * a.heads;
    const uint64_t blocks = ((uint64_t)a.n_seqs * a.heads + 7) / 8 * 8 * a.slices;
    if (items > 0x7FFFFFFFull || blocks > 0x7FFFFFFFull) return WAL_ERR_SHAPE;
    hipLaunchKernelGGL((k_delta_chunk<DK>), dim3((uint32_t)items), dim3(256), 0, s, a);
    hipLaunchKernelGGL((k_delta_scan<DK>), dim3((uint32_t)blocks), dim3(128 * kScanGroups), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}

}  // namespace

namespace wal {

int delta_chunks(Delta& a, uint32_t key_dim, uint32_t all, void* stream) {
  static_assert(kScanGroups * 16 == kSlice, "a workgroup takes a slice");
  hipStream_t s = static_cast<hipStream_t>(stream);
  return key_dim == 64 ? launch<64>(a, all, s) : launch<128>(a, all, s);
}

}  // namespace wal
