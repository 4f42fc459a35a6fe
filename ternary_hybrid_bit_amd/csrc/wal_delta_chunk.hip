// The gated delta rule on chunks of 64 tokens for gfx950 (prompts).  With G_i the
// sum of the logarithms of the decays of a chunk's tokens up to i, S0 the state
// before it and u_i the rows that its tokens store,
//     u = T (diag(b) V - diag(b e^G) K S0),    T = (1 + A)^-1,
//         A_ij = b_i e^(G_i - G_j) k_i . k_j   (j < i)
//     O = diag(e^G) Q S0 + P u,    P_ij = e^(G_i - G_j) q_i . k_j   (j <= i)
//     S = e^G_end S0 + K^T diag(e^(G_end - G)) u
// so that tokens meet in products on the matrix cores and only states go from chunk
// to chunk.  k_delta_chunk makes T, P and the factors of the rows of every chunk and head, all of
// them at once; k_delta_scan walks the chunks of a sequence and head, two wavefronts
// keeping 16 columns of the state in registers, half of the rows each: everything that a
// column of the values meets belongs to that column alone.
//
// Numbers.  Values enter the products as sums of parts in bf16, which has fp32's range: what an update of a state sees (the
// state, T, the rows b V - .., u) as three, 24 bits, and what only outputs in bf16 see (P, u and the state there) as two, 16
// bits; K and Q hold bf16 to begin with.  So a value keeps its bits whatever lies beside it: a row a billion times its
// neighbours takes nothing from the rows before it, nor from those behind a token that forgets it.  Two parts in half precision
// hold 22 bits and lose them as soon as rows of a column that share a scale differ by 2^9 (that way 8192 tokens of 48 heads took
// 320 us for 364, of 32 heads 271 for 322); outputs of one part in half precision were off by up to 3.2e-3 where keys are alike and stored rows
// cancel, for the 1.66e-3 of their rounding to bf16.  Rows of K and Q are brought to
// lengths of 1 to 2 by powers of two.  Keys and queries are taken as unit vectors and lengths, the lengths into the
// factors of the rows.  G is added up in 64 bits, because e^(G_i - G_j) has to be exact also after a token that
// forgets everything.  Exponents are never above 0.
//
// Not finite.  A product with T would carry a NaN of row j into rows above j, as 0 * NaN.  From
// a chunk's first token on whose key or gates are not finite, rows are taken out of A and their
// factors are NaN; k_delta_scan looks at one row of u of each 32, and where it is not
// finite takes the rows that are not out of the product and puts NaN where they belong.
//
// What bounds it.  k_delta_chunk: instructions and latencies (its stores hide behind them).  k_delta_scan: the
// chain of a chunk, K S, the sum of its halves, T, K^T u: 5200 cycles of which a SIMD's matrix cores are busy 1800 (1340 with
// the states, the rest with outputs); what else there is are the parts' roundings and latencies, of LDS too.  With
// 192 workgroups of 16 + 16 columns the clock falls besides (2.1 GHz).
// Measured (graph): 8192 tokens, 48 heads of 128 on 16 364 us, about 82 of them k_delta_chunk; 32 heads 322; 4096 tokens, 32 heads
// 168; 9 sequences up to 1111, 8 heads of 64 x 96 on 4, 53 (49 call by call, where a call's inputs are warmer).
#include <hip/hip_runtime.h>

#include "wal_delta.h"
#include "wal_find.h"

namespace {

constexpr int kC = kChunk;
constexpr uint32_t kLd = kC + 4;       // of T in LDS: four 16 x 16 blocks of the diagonal on different banks
constexpr uint32_t kBlocks = kTriangle / kOperand;   // (32-row block, half, 32-column block) of a lower triangle
constexpr int kPair = 2;               // value heads of a workgroup of k_delta_chunk
// The rows of u are taken times 2^-8: T's values are at most 2 as long as b |k|^2 is, so that 64 of them with a row at the end
// of fp32's range stay inside it.
constexpr float kRow = 0x1p-8f, kRowBack = 0x1p8f;
constexpr float kForget = -1000.f;     // logarithms of decays below this one are it: e^-1000 is 0

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// Rows 32 u + 8 (m / 4) + 4 h + m % 4 of operand (u, h): lane group c of a result holds rows 8 c + 4 h + i, and the two
// halves make the eight rows 8 c .. of a B operand.
__device__ __forceinline__ uint32_t dealt(uint32_t u, uint32_t h, uint32_t m) { return 32 * u + 8 * (m >> 2) + 4 * h + (m & 3); }

__device__ __forceinline__ f32x4_t product(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Eight values as the sum of N parts in bf16, each the nearest to what the ones before leave: 8 bits more apiece.
template <int N>
__device__ __forceinline__ void split(f32x4_t x, f32x4_t y, u32x4_t (&p)[N]) {
  static_assert(N >= 1 && N <= 3, "three parts hold what fp32 does");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float r0 = i < 2 ? x[2 * i] : y[2 * i - 4], r1 = i < 2 ? x[2 * i + 1] : y[2 * i - 3];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const uint32_t w = __builtin_bit_cast(uint32_t, (bf16x2_t{(__bf16)r0, (__bf16)r1}));
      p[e][i] = w;
      if (e + 1 < N) {
        r0 -= __uint_as_float(w << 16);
        r1 -= __uint_as_float(w & 0xFFFF0000u);
      }
    }
  }
}

// 2^-e and 2^e of a row's length, rounded down to 2^e, by its sum of squares; e is at least -107.
struct Scale {
  float up, down;
};
__device__ __forceinline__ Scale row_scale(float squares) {
  const uint32_t e = max(((__float_as_uint(squares) >> 23 & 0xFFu) + 127u) >> 1, 20u);
  return Scale{__uint_as_float((254u - e) << 23), __uint_as_float(e << 23)};
}

// The sum over 8 or 16 lanes side by side, in each of them.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
  x += dpp<0xB1>(x);    // quad_perm [1, 0, 3, 2]
  x += dpp<0x4E>(x);    // quad_perm [2, 3, 0, 1]
  x += dpp<0x141>(x);   // row_half_mirror
  if constexpr (LANES == 16) x += dpp<0x140>(x);   // row_mirror
  return x;
}

// 2^(x - y) of sums kept as high and low halves, exact to fp32 however long they are.
__device__ __forceinline__ float power(float2 x, float2 y) { return __builtin_amdgcn_exp2f((x.x - y.x) + (x.y - y.y)); }

// The sequence of a chunk's place: sequence s has those from starts[s] / 64 + s on.
__device__ __forceinline__ uint32_t seq_of_place(const Delta& a, uint32_t place, uint32_t lane) {
  return last_begun(a.n_seqs, lane, [&](uint32_t s) { return (uint32_t)between(a.starts[s], 0, (int32_t)a.n) / kC + s <= place; });
}

// What a launch's place holds of a value head and of a key head: a head's places side by side, since they are read one
// after another.
__device__ __forceinline__ uint8_t* item_of(const Delta& a, uint32_t local, uint32_t head) {
  return a.ws + ((uint64_t)head * a.places + local) * kItemBytes;
}
__device__ __forceinline__ uint8_t* key_item_of(const Delta& a, uint32_t local, uint32_t kh) {
  return a.key_ws + ((uint64_t)kh * a.places + local) * a.key_item;
}

// Place of a row's 16-byte piece in LDS: 16 neighbours that are read together, the rows of dealt(), and in the transposing
// reads four neighbours fall on different banks.
template <int DK>
__device__ __forceinline__ uint32_t row_piece(uint32_t r, uint32_t p) {
  return r * (2 * DK) + 16 * (DK == 128 ? p ^ (r & 15) : p ^ ((r >> 1) & 7));
}
template <int DK>
__device__ __forceinline__ uint32_t dealt_piece(uint32_t r, uint32_t p) {
  return r * (2 * DK) + 16 * (DK == 128 ? p ^ ((r & 3) << 2 | ((r >> 3) & 3)) : p ^ (((r >> 1) & 1) << 2 | ((r >> 3) & 3)));
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

// Rows I .. 15 of the inverse of 1 + a, a 16 x 16 block whose rows the 16 lanes of a group hold: x is the lane's column.
template <int I>
__device__ __forceinline__ void invert_rows(const float (&a)[16], float (&x)[16], uint32_t n) {
  if constexpr (I < 16) {
    float y[2] = {I == n ? 1.f : 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < I; ++j) y[j & 1] = fmaf(-dpp<0x150 + I>(a[j]), x[j], y[j & 1]);   // lane I's, in every lane
    x[I] = y[0] + y[1];
    invert_rows<I + 1>(a, x, n);
  }
}

// T, P and the rows' factors of a chunk of up to two value heads that share a key head, and (the first of them) K and Q.
template <int DK>
__global__ __launch_bounds__(256) void k_delta_chunk(Delta a) {
  constexpr uint32_t kPieces = DK / 8, kRows = 256 / kPieces, U = DK / 32;
  constexpr uint32_t kRaw = 2 * kC * DK * 2, kMat = kPair * kC * kLd * 4;
  __shared__ __attribute__((aligned(256))) uint8_t raw[kRaw > kMat ? kRaw : kMat];
  __shared__ __attribute__((aligned(16))) float2 far[kPair][kC];   // sums of the decays' logarithms to base 2, high and low halves
  __shared__ __attribute__((aligned(16))) float kk[kC], qq[kC], left[kPair][kC], unit_k[kC], unit_q[kC];
  __shared__ uint32_t first_bad[kPair];
  uint8_t *ks = raw, *qs = raw + kRaw / 2;
  float(*t)[kC][kLd] = reinterpret_cast<float(*)[kC][kLd]>(raw);
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, c = lane >> 4;
  const uint32_t pairs = (a.group + kPair - 1) / kPair, key_heads = a.heads / a.group;
  const uint32_t pair = blockIdx.x % pairs, kh = blockIdx.x / pairs % key_heads, local = blockIdx.x / pairs / key_heads;
  const uint32_t h0 = kh * a.group + kPair * pair, heads = min(a.group - kPair * pair, (uint32_t)kPair);
  const uint32_t s = seq_of_place(a, a.place0 + local, lane);
  const Seq q = delta_seq(a, s);
  const int32_t row0 = kC * (int32_t)(a.place0 + local - ((uint32_t)q.first / kC + s));   // of the sequence
  if (row0 < 0 || row0 >= q.rows || q.rows <= a.few) return;
  const int32_t count = min(q.rows - row0, kC);
  const uint64_t from = (uint64_t)(q.first + row0);

  u32x4_t kr[kC / kRows], qr[kC / kRows];
#pragma unroll
  for (int i = 0; i < (int)(kC / kRows); ++i) {
    const int32_t r = (int32_t)(tid / kPieces + i * kRows);
    const uint64_t at = from + min(r, count - 1);
    kr[i] = *reinterpret_cast<const u32x4_t*>(a.k + at * a.ldk + kh * DK + 8 * (tid % kPieces));
    qr[i] = *reinterpret_cast<const u32x4_t*>(a.q + at * a.ldq + kh * DK + 8 * (tid % kPieces));
  }
  float beta = 0.f;
  if (wave < heads) {
    const bool there = (int32_t)lane < count;
    const Gates g = gates_of(a, from + min((int32_t)lane, count - 1), h0 + wave);
    beta = there ? g.beta : 0.f;
    double x = !there ? 0.0 : g.log_alpha < kForget ? (double)kForget : (double)g.log_alpha;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double y = __shfl_up(x, d);
      if (lane >= (uint32_t)d) x += y;
    }
    x *= 1.4426950408889634074;
    far[wave][lane] = make_float2((float)x, (float)(x - (double)(float)x));
  }
  uint8_t* key_item = key_item_of(a, local, kh);
#pragma unroll
  for (int i = 0; i < (int)(kC / kRows); ++i) {
    const uint32_t r = tid / kPieces + i * kRows, piece = tid % kPieces;
    if ((int32_t)r >= count) kr[i] = qr[i] = u32x4_t{0, 0, 0, 0};
    f32x4_t k4[2], q4[2];
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      k4[j / 2][2 * (j % 2)] = __uint_as_float(kr[i][j] << 16);
      k4[j / 2][2 * (j % 2) + 1] = __uint_as_float(kr[i][j] & 0xFFFF0000u);
      q4[j / 2][2 * (j % 2)] = __uint_as_float(qr[i][j] << 16);
      q4[j / 2][2 * (j % 2) + 1] = __uint_as_float(qr[i][j] & 0xFFFF0000u);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x = fmaf(k4[j / 4][j % 4], k4[j / 4][j % 4], x);
      y = fmaf(q4[j / 4][j % 4], q4[j / 4][j % 4], y);
    }
    x = lanes_sum<kPieces>(x);
    y = lanes_sum<kPieces>(y);
    if (piece == 0) {
      kk[r] = x;
      qq[r] = y;
    }
    u32x4_t kw[1], qw[1];
    const float ks2 = row_scale(x).up, qs2 = row_scale(y).up;   // powers of two: bf16 holds the rows as before
    split(k4[0] * ks2, k4[1] * ks2, kw);
    split(q4[0] * qs2, q4[1] * qs2, qw);
    *reinterpret_cast<u32x4_t*>(ks + row_piece<DK>(r, piece)) = kw[0];
    *reinterpret_cast<u32x4_t*>(qs + row_piece<DK>(r, piece)) = qw[0];
    if (pair == 0) {
      *reinterpret_cast<u32x4_t*>(key_item + r * (2 * DK) + 16 * piece) = kw[0];
      // operand (tile of dealt rows, 32 columns), lane (row, eight columns)
      const uint32_t tile = 2 * (r >> 5) + ((r >> 2) & 1), m = (r >> 3 & 3) * 4 + (r & 3);
      *reinterpret_cast<u32x4_t*>(key_item + kC * 2 * DK + (tile * U + piece / 4) * kOperand + 16 * (16 * (piece % 4) + m)) = qw[0];
    }
  }
  lds_barrier();

  // The ten 16 x 16 tiles of A's lower triangle by rows; P's six operands: transposed tiles of K Q^T with dealt rows, whose
  // results are what a lane of the operand holds.  Wavefronts 0 and 1 take two tiles and two operands, the others three and one.
  const uint32_t tiles = wave < 2 ? 2 : 3, ops = wave < 2 ? 2 : 1;
  const uint32_t tile0 = wave < 2 ? 2 * wave : 3 * wave - 2, op0 = wave < 2 ? 2 * wave : wave + 2;
  f32x4_t ak[3], pk[2][2];
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const uint32_t tile = min(tile0 + x, 9u), it = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0, jt = tile - it * (it + 1) / 2;
    ak[x] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (x < (int)tiles)
#pragma unroll
      for (uint32_t u = 0; u < U; ++u)
        ak[x] = product(*reinterpret_cast<const u32x4_t*>(ks + row_piece<DK>(16 * it + n, 4 * u + c)),
                        *reinterpret_cast<const u32x4_t*>(ks + row_piece<DK>(16 * jt + n, 4 * u + c)), ak[x]);
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint32_t b = min(op0 + x, 5u), w = b > 1, sb = b > 3, hf = b & 1;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      pk[x][z] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (x < (int)ops)
#pragma unroll
        for (uint32_t u = 0; u < U; ++u)
          pk[x][z] = product(*reinterpret_cast<const u32x4_t*>(ks + row_piece<DK>(dealt(sb, z, n), 4 * u + c)),
                             *reinterpret_cast<const u32x4_t*>(qs + row_piece<DK>(dealt(w, hf, n), 4 * u + c)), pk[x][z]);
    }
  }
  if (wave < heads) {
    const float2 g = far[wave][lane], end = far[wave][kC - 1], none = make_float2(0.f, 0.f);
    // keys are unit vectors times lengths: K holds k 2^e, that is unit vectors times 1 / uk
    const float k2 = kk[lane], q2 = qq[lane], kn = sqrtf(k2), qn = sqrtf(q2);
    const Scale ek = row_scale(k2), eq = row_scale(q2);
    const float uk = kn > 0.f ? ek.down / kn : 0.f, uq = qn > 0.f ? eq.down / qn : 0.f;
    const float to_k = unit(a, k2), to_q = unit(a, q2);
    const bool bad = !(fabsf(k2) < INFINITY) || !(fabsf(beta) < INFINITY) || g.x != g.x;
    const uint64_t any = __ballot(bad);
    const uint32_t f = any ? (uint32_t)__builtin_ctzll(any) : (uint32_t)kC;
    const float lost = lane >= f ? NAN : 0.f, gone = any ? NAN : 0.f;
    const float decay = power(g, none), len = kn * to_k;
    float* vec = reinterpret_cast<float*>(item_of(a, local, h0 + wave) + kVecAt);
    vec[lane] = kRow * beta * len + lost;
    vec[kC + lane] = kRow * beta * len * len * decay * uk + lost;
    vec[2 * kC + lane] = power(end, g) * uk + gone;
    vec[4 * kC + lane] = decay * uq;
    vec[5 * kC + lane] = qn * to_q * a.scale;
    if (lane == 0) {
      vec[3 * kC] = power(end, none) + gone;
      first_bad[wave] = f;
    }
    left[wave][lane] = beta * len * len * uk;
    if (wave == 0) {
      unit_k[lane] = uk;
      unit_q[lane] = uq;
    }
  }
  lds_barrier();   // K and Q are read: A goes to their place
  for (uint32_t b = 0; b < heads; ++b) {
    const float2* g = far[b];
    const uint32_t bad = first_bad[b];
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      const uint32_t tile = tile0 + x, it = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0, jt = tile - it * (it + 1) / 2;
      if (x >= (int)tiles) continue;
      const uint32_t col = 16 * jt + n, row = 16 * it + 4 * c;
      const f32x4_t l = *reinterpret_cast<const f32x4_t*>(&left[b][row]), g0 = *reinterpret_cast<const f32x4_t*>(&g[row]),
                    g1 = *reinterpret_cast<const f32x4_t*>(&g[row + 2]);
      const float2 gc = g[col];
      const float uk = unit_k[col];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 gr = i < 2 ? make_float2(g0[2 * i], g0[2 * i + 1]) : make_float2(g1[2 * i - 4], g1[2 * i - 3]);
        t[b][row + i][col] = col < row + i && row + i < bad ? l[i] * uk * power(gr, gc) * ak[x][i] : 0.f;
      }
    }
    if (wave >= 2) {   // tiles (0, 1) and (2, 3): nothing
      const uint32_t row = 32 * (wave - 2) + n, col = 32 * (wave - 2) + 16 + 4 * c;
      *reinterpret_cast<f32x4_t*>(&t[b][row][col]) = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t o = op0 + x, w = o > 1, sb = o > 3, hf = o & 1, row = dealt(w, hf, n);
      if (x >= (int)ops) continue;
      f32x4_t y[2];
      const float2 gr = g[row];
      const float uq = unit_q[row];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t col = 32 * sb + 8 * c + 4 * z;
        const f32x4_t uk = *reinterpret_cast<const f32x4_t*>(&unit_k[col]), g0 = *reinterpret_cast<const f32x4_t*>(&g[col]),
                      g1 = *reinterpret_cast<const f32x4_t*>(&g[col + 2]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 gc = i < 2 ? make_float2(g0[2 * i], g0[2 * i + 1]) : make_float2(g1[2 * i - 4], g1[2 * i - 3]);
          y[z][i] = col + i <= row ? uq * uk[i] * power(gr, gc) * pk[x][z][i] : 0.f;
        }
      }
      u32x4_t p[kPParts];
      split(y[0], y[1], p);
#pragma unroll
      for (int e = 0; e < (int)kPParts; ++e)
        *reinterpret_cast<u32x4_t*>(item_of(a, local, h0 + b) + kPAt + e * kTriangle + o * kOperand + 16 * lane) = p[e];
    }
  }
  lds_barrier();

  if (wave < heads) {   // the inverses of the four blocks of the diagonal
    float(*tb)[kLd] = t[wave];
    float x[16], d[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4_t w = *reinterpret_cast<const f32x4_t*>(&tb[16 * c + n][16 * c + 4 * i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[4 * i + j] = w[j];
    }
    invert_rows<0>(d, x, n);
#pragma unroll
    for (int i = 0; i < 16; ++i) tb[16 * c + i][16 * c + n] = x[i];
  }
  lds_barrier();
  // two wavefronts a head: blocks (1, 0) and (3, 2), then the columns of the lower left 32 x 32
  const uint32_t hb = wave >> 1, half = wave & 1;
  float(*tb)[kLd] = t[hb];
  const bool mine = hb < heads;
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  if (mine) {
    const uint32_t r = 2 * half + 1, b = 2 * half;
    const f32x4_t y = block_product(tb, r, b, b, b, n, c, zero), z = block_product(tb, r, r, y, n, c, zero);
#pragma unroll
    for (int i = 0; i < 4; ++i) tb[16 * r + 4 * c + i][16 * b + n] = -z[i];
  }
  lds_barrier();
  f32x4_t lower[2];
  if (mine) {
    f32x4_t y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      y[i] = half == 0 ? block_product(tb, 2 + i, 0, 0, 0, n, c, zero) : zero;
      y[i] = block_product(tb, 2 + i, 1, 1, half, n, c, y[i]);
    }
    lower[0] = block_product(tb, 2, 2, y[0], n, c, zero);
    lower[1] = block_product(tb, 3, 3, y[1], n, c, block_product(tb, 3, 2, y[0], n, c, zero));
  }
  lds_barrier();
  if (mine)
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) tb[16 * (2 + k) + 4 * c + i][16 * half + n] = -lower[k][i];
  lds_barrier();
  for (uint32_t i = tid; i < heads * kBlocks * 64; i += 256) {
    const uint32_t b = i / (kBlocks * 64), e = i - b * (kBlocks * 64), o = e >> 6, l = e & 63;
    const uint32_t row = dealt(o > 1, o & 1, l & 15), col = 32 * (o > 3) + 8 * (l >> 4);
    u32x4_t w[kTParts];
    split(*reinterpret_cast<const f32x4_t*>(&t[b][row][col]), *reinterpret_cast<const f32x4_t*>(&t[b][row][col + 4]), w);
    uint8_t* item = item_of(a, local, h0 + b);
#pragma unroll
    for (int k = 0; k < (int)kTParts; ++k) *reinterpret_cast<u32x4_t*>(item + k * kTriangle + 16 * e) = w[k];
  }
}

constexpr int kScanGroups = 2;   // groups of 16 columns of a workgroup

// Rows of a chunk in memory: what lies behind the last one reads as zeros and is not written.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rows(const uint16_t* p, uint64_t ld, int32_t count, uint32_t width) {
  return rsrc(p, (uint32_t)(2 * ((uint64_t)(count - 1) * ld + width)));
}

// Four wavefronts share 16 columns.  Two take the state from chunk to chunk, half of its rows each, which is what a
// sequence waits for; they add up K S between them and make u both.  The others, behind them, make the outputs, of 32 of a
// chunk's tokens each, from the states and rows that the first leave in LDS as operands, and bring the next chunks' K, V, T
// and factors there.
//
// One barrier a chunk, between a chunk's K S and its u:
//   states   .. | u of j, S, K S of j + 1 | u of j + 1, ..
//   outputs  .. | out of j - 1, Q S of j, stores K of j + 2 and V, T of j + 1 | ..
// Everything is kept twice.
template <int DK>
struct Scan {
  static constexpr int U = DK / 32, UH = U / 2;           // 32-row blocks of the state, of a half
  static constexpr uint32_t kPieces = DK / 8, kThreads = 128 * kScanGroups, kRows = kThreads / kPieces;   // that stage
  static constexpr int kPasses = kC / (int)kRows;
  static constexpr uint32_t kTPieces = kTParts * kTriangle / 16;
  static constexpr int kTPasses = (kTPieces + kThreads - 1) / kThreads;
  static_assert(kThreads == 256 && kC * kSlice * 2 == 16 * kThreads && 4 * kC == kThreads, "V and the factors in one pass");
  struct Shared {
    __attribute__((aligned(256))) uint8_t k[2][kC * DK * 2];
    __attribute__((aligned(16))) uint8_t v[2][kC * kSlice * 2];
    u32x4_t t[2][kTParts * kBlocks][64];
    u32x4_t state[2][kScanGroups][U][2][64];              // before a chunk, its first two parts
    u32x4_t u[2][kScanGroups][2][2][64];                  // of 32 tokens each, two parts
    f32x4_t ks[2][kScanGroups][2][4][64];                 // the halves' K S
    __attribute__((aligned(16))) float vec[2][4 * kC];
    int32_t bad[2][kScanGroups][16];                      // the first of a column's rows that is not finite
  };
  const Delta& a;
  Shared& sh;
  const Seq q;
  const uint32_t base, h, kh, col, lane, n, c, group;
  const int32_t j0, j1;

  __device__ __forceinline__ uint32_t local(int32_t j) const { return base + (uint32_t)j - a.place0; }
  __device__ __forceinline__ const uint8_t* item(int32_t j) const { return item_of(a, local(j), h); }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const uint16_t* p, uint64_t ld, int32_t j, uint32_t at, uint32_t width) const {
    return chunk_rows(p + (uint64_t)(q.first + j * kC) * ld + at, ld, min(q.rows - j * kC, kC), width);
  }

  // Rows DK / 2 half .. of the state; element i of st[u][hf]: row 32 u + 8 c + 4 hf + i of them.  Runs of products go
  // over their tiles first, so that none waits for the one before.
  __device__ __forceinline__ void states(uint32_t half, const float* before, float* after) {
    const uint32_t dv = a.value_dim, at0 = DK / 2 * half;
    f32x4_t st[UH][2];
#pragma unroll
    for (int u = 0; u < UH; ++u)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < 4; ++i) st[u][hf][i] = before ? before[(uint64_t)(at0 + 32 * u + 4 * hf + i) * dv] : 0.f;
    // Lanes' places in K: of rows dealt(0, 0, n), and for the transposing reads; a 32-column block further is an exclusive
    // or with 64 bytes, and rows 4 hf and 32 w further change no bits that the pieces' exchange looks at.
    const uint32_t kat = dealt_piece<DK>(dealt(0, 0, n), c) ^ 64 * UH * half, tat = dealt_piece<DK>(8 * c + (n >> 2), n & 3) ^ 64 * UH * half;
    f32x4_t ks[4];
    union { s16x4_t half[2]; u32x4_t all; } kt[2][2 * UH];   // four tokens of the lane's row of K^T each
    // the state in parts, and its half of K S of chunk j; what the chunk needs of K^T besides
    const auto take = [&](int32_t j) {
      const uint8_t* k = sh.k[j & 1];
      u32x4_t kw[UH][4];
#pragma unroll
      for (int u = 0; u < UH; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) kw[u][t] = *reinterpret_cast<const u32x4_t*>(k + (kat ^ 64 * u) + (16 * (t & 2) + 4 * (t & 1)) * 2 * DK);
#pragma unroll
      for (int t = 0; t < 4; ++t) ks[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < UH; ++u) {
        u32x4_t part[3];
        split(st[u][0], st[u][1], part);
#pragma unroll
        for (int e = 0; e < 2; ++e) sh.state[j & 1][group][UH * half + u][e][lane] = part[e];
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll
          for (int t = 0; t < 4; ++t) ks[t] = product(kw[u][t], part[e], ks[t]);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int t = 0; t < 2 * UH; ++t)
#pragma unroll
          for (int z = 0; z < 2; ++z)
            kt[w][t].half[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4_t*)(k + (tat ^ 64 * (t / 2)) + (32 * w + 4 * z) * 2 * DK + 8 * (t % 2)));
#pragma unroll
      for (int t = 0; t < 4; ++t) sh.ks[j & 1][group][half][t][lane] = ks[t];
    };
    lds_barrier();
    take(j0);
    lds_barrier();
    for (int32_t j = j0; j < j1; ++j) {
      const float* vec = sh.vec[j & 1];
      const float decay = vec[3 * kC];
      // the rows b V - b e^G K S0; the lane's rows of V are four tokens of its column each
      f32x4_t rows[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t r = 16 * (t & 2) + 8 * c + 4 * (t & 1);
        const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(sh.v[j & 1] + 2 * kSlice * (r + (n >> 2)) + 32 * group + 8 * (n & 3)));
        const f32x4_t c1 = *reinterpret_cast<const f32x4_t*>(vec + r), c2 = *reinterpret_cast<const f32x4_t*>(vec + kC + r);
        const f32x4_t both = ks[t] + sh.ks[j & 1][group][1 - half][t][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[t][i] = fmaf(-c2[i], both[i], c1[i] * bf16_value((uint16_t)v[i]));
      }
      f32x4_t c3[4];   // read here, where nothing waits for them yet
#pragma unroll
      for (int t = 0; t < 4; ++t) c3[t] = *reinterpret_cast<const f32x4_t*>(vec + 2 * kC + 16 * (t & 2) + 8 * c + 4 * (t & 1));
      f32x4_t u[4];   // times 2^-8
      const auto solve = [&] {
        u32x4_t part[2][3];
#pragma unroll
        for (int w = 0; w < 2; ++w) split(rows[2 * w], rows[2 * w + 1], part[w]);
#pragma unroll
        for (int t = 0; t < 4; ++t) u[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 3; ++e)   // by size, so that they begin before the small parts are there; those below 2^-24 are left out
#pragma unroll
          for (int f = 0; f <= e; ++f)
#pragma unroll
            for (int b = 0; b < (int)kBlocks; ++b) {
              const int t = 2 * (b > 1) + (b & 1), sb = b > 3;
              u[t] = product(sh.t[j & 1][(e - f) * kBlocks + b][lane], part[sb][f], u[t]);
            }
      };
      solve();
      int32_t bad = kC;
      if (__any(!(fabsf(u[0][0]) < INFINITY) || !(fabsf(u[2][0]) < INFINITY))) {
#pragma unroll
        for (int t = 3; t >= 0; --t)
#pragma unroll
          for (int i = 3; i >= 0; --i)
            if (!(fabsf(rows[t][i]) < INFINITY)) {
              bad = 16 * (t & 2) + 8 * (int32_t)c + 4 * (t & 1) + i;
              rows[t][i] = 0.f;
            }
        bad = min(bad, __shfl_xor(bad, 16));
        bad = min(bad, __shfl_xor(bad, 32));
        solve();
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * (t & 2) + 8 * (int32_t)c + 4 * (t & 1) + i >= bad) u[t][i] = 0.f;
      }
      // S = decay S + K^T diag(e^(G_end - G)) u
      u32x4_t up[2][3], own[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) split(c3[2 * w] * u[2 * w], c3[2 * w + 1] * u[2 * w + 1], up[w]);
      split(half ? u[2] : u[0], half ? u[3] : u[1], own);
#pragma unroll
      for (int e = 0; e < 2; ++e) sh.u[j & 1][group][half][e][lane] = own[e];
      // every lane that holds a value writes it: a branch here would keep what is around it apart
      sh.bad[j & 1][group][n] = bad;
      float back = bad < kC ? NAN : kRowBack;
      asm("" : "+v"(back));   // chosen once, not after each of the sums below
      f32x4_t add[2 * UH];
#pragma unroll
      for (int t = 0; t < 2 * UH; ++t) add[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 3; ++e)
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int t = 0; t < 2 * UH; ++t) add[t] = product(kt[w][t].all, up[w][e], add[t]);
#pragma unroll
      for (int t = 0; t < 2 * UH; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) st[t / 2][t % 2][i] = fmaf(add[t][i], back, decay * st[t / 2][t % 2][i]);
      take(j + 1);   // behind the last chunk: of some chunk's K, and not read
      lds_barrier();
    }
    if (after)
#pragma unroll
      for (int u = 0; u < UH; ++u)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int i = 0; i < 4; ++i) after[(uint64_t)(at0 + 32 * u + 4 * hf + i) * dv] = st[u][hf][i];
  }

  // O = diag(e^G) Q S0 + P u, of tokens 32 w ..  What is stored to LDS was loaded a chunk before, operands when the ones
  // before are used.
  __device__ __forceinline__ void outputs(uint32_t w) {
    const uint32_t dv = a.value_dim, ldo = (uint32_t)a.ldo, ldv = (uint32_t)a.ldv, tid = 64 * (kScanGroups * w + group) + lane;
    const uint32_t olane = 2 * ((32 * w + 8 * c) * ldo + col), vlane = 2 * (tid / 4 * ldv + (col & ~(kSlice - 1)) + 8 * (tid % 4));
    u32x4_t kr[kPasses], vr, tr[kTPasses], pw[2][kPParts][2], qw[2][U];   // P: of 32 tokens before (zeros for the first), of its own
    f32x4_t c4[2], c6[2], o[2];
    float fr;
    const int32_t last = j1 - 1;
    const auto load_k = [&](int32_t j) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) kr[i] = *reinterpret_cast<const u32x4_t*>(key_item_of(a, local(min(j, last)), kh) + 16 * (tid + i * kThreads));
    };
    const auto store_k = [&](int32_t j) {
      uint8_t* k = sh.k[j & 1];
#pragma unroll
      for (int i = 0; i < kPasses; ++i) *reinterpret_cast<u32x4_t*>(k + dealt_piece<DK>(tid / kPieces + i * kRows, tid % kPieces)) = kr[i];
    };
    const auto load_rest = [&](int32_t j) {
      const uint8_t* p = item(min(j, last));
#pragma unroll
      for (int i = 0; i < kTPasses; ++i) tr[i] = *reinterpret_cast<const u32x4_t*>(p + 16 * (tid + i * kThreads));   // and some of P behind it
      fr = *reinterpret_cast<const float*>(p + kVecAt + 4 * tid);
      vr = __builtin_amdgcn_raw_buffer_load_b128(rows_of(a.v, a.ldv, min(j, last), h * dv, dv), vlane, 0, 0);
    };
    const auto store_rest = [&](int32_t j) {
#pragma unroll
      for (int i = 0; i < kTPasses; ++i)
        if ((i + 1) * kThreads <= kTPieces || 64 * kScanGroups * w + i * kThreads < kTPieces) (&sh.t[j & 1][0][0])[tid + i * kThreads] = tr[i];
      sh.vec[j & 1][tid] = fr;
      *reinterpret_cast<u32x4_t*>(sh.v[j & 1] + 16 * tid) = vr;
    };
    const auto load_q = [&](int32_t j) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < U; ++u)
          qw[t][u] = *reinterpret_cast<const u32x4_t*>(key_item_of(a, local(min(j, last)), kh) + kC * 2 * DK + ((2 * w + t) * U + u) * kOperand + 16 * lane);
    };
    const auto load_p = [&](int32_t j) {
      const uint8_t* p = item(min(j, last));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int e = 0; e < (int)kPParts; ++e) {
          const uint8_t* part = p + kPAt + e * kTriangle + 16 * lane;
          pw[0][e][t] = w ? *reinterpret_cast<const u32x4_t*>(part + (2 + t) * kOperand) : u32x4_t{0, 0, 0, 0};
          pw[1][e][t] = *reinterpret_cast<const u32x4_t*>(part + (4 * w + t) * kOperand);
        }
        const uint8_t* f = p + kVecAt + 4 * (4 * kC + 32 * w + 8 * c + 4 * t);
        c4[t] = *reinterpret_cast<const f32x4_t*>(f);
        c6[t] = *reinterpret_cast<const f32x4_t*>(f + 4 * kC);
      }
    };
    const auto from_state = [&](int32_t j) {   // Q S of chunk j, by the state's parts
      f32x4_t x[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int t = 0; t < 2; ++t) x[e][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const u32x4_t part = sh.state[j & 1][group][u][e][lane];
#pragma unroll
          for (int t = 0; t < 2; ++t) x[e][t] = product(qw[t][u], part, x[e][t]);
        }
#pragma unroll
      for (int t = 0; t < 2; ++t) o[t] = x[0][t] + x[1][t];
    };
    const auto finish = [&](int32_t j) {
      f32x4_t p[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int e = 1; e >= 0; --e)   // the product of the second parts, below 2^-16, is left out
#pragma unroll
        for (int f = 0; f <= e; ++f)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const u32x4_t u = sh.u[j & 1][group][b ? w : 0][f][lane];
#pragma unroll
            for (int t = 0; t < 2; ++t) p[t] = product(pw[b][e - f][t], u, p[t]);
          }
      const int32_t bad = sh.bad[j & 1][group][n] - 32 * (int32_t)w;
      const __amdgpu_buffer_rsrc_t r = rows_of(a.out, a.ldo, j, h * dv, dv);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = c6[t][i] * fmaf(c4[t][i], o[t][i], kRowBack * p[t][i]);
          __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)((int32_t)(4 * t + i + 8 * c) >= bad ? NAN : y)), r,
                                                olane + (4 * t + i) * 2 * ldo, 0, 0);
        }
    };
    load_k(j0);
    load_rest(j0);
    store_k(j0);
    load_k(j0 + 1);
    store_rest(j0);
    store_k(j0 + 1);
    load_k(j0 + 2);
    load_rest(j0 + 1);
    load_q(j0);
    load_p(j0);
    lds_barrier();
    lds_barrier();   // the states' first K S
    const auto step = [&](int32_t j) {
      store_k(j + 2);
      load_k(j + 3);
      store_rest(j + 1);
      load_rest(j + 2);
      from_state(j);
      load_q(j + 1);
      lds_barrier();
    };
    step(j0);   // (before the loop and at its end: what is in flight is the same both ways in, and no wait covers more than it has to)
    for (int32_t j = j0; j < last; ++j) {
      finish(j);
      load_p(j + 1);
      step(j + 1);
    }
    finish(last);
  }
};

template <int DK>
__global__ __launch_bounds__(256 * kScanGroups, 1) void k_delta_scan(Delta a) {
  __shared__ typename Scan<DK>::Shared sh;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, c = lane >> 4;
  const uint32_t group = wave % kScanGroups;
  // The workgroups of a head sit on one chiplet, or those of all heads of a key head, so that its cache serves what they
  // share: blocks go to the eight chiplets in turn.
  const uint32_t per = a.together * a.slices, g = blockIdx.x / 8, slice = g % per % a.slices;
  const uint32_t pair = (g / per * 8 + blockIdx.x % 8) * a.together + g % per / a.slices;
  if (pair >= a.seqs * a.heads) return;
  // from the sequence of the launch's first place on
  const uint32_t s = (a.place0 ? seq_of_place(a, a.place0, lane) : 0) + pair / a.heads, h = pair % a.heads;
  if (s >= a.n_seqs) return;
  const uint32_t col = kSlice * slice + 16 * group + n;
  const Seq q = delta_seq(a, s);
  const uint32_t base = (uint32_t)q.first / kC + s;
  const int32_t chunks = (q.rows + kC - 1) / kC;
  const int32_t j0 = max(0, (int32_t)a.place0 - (int32_t)base), j1 = min(chunks, (int32_t)(a.place0 + a.places) - (int32_t)base);
  if (j0 >= j1 || q.rows <= a.few) return;
  const int64_t slot = kept_at(a, s);
  const uint64_t head_at = ((uint64_t)h * DK + 8 * c) * a.value_dim + col;
  float* kept = slot < 0 ? nullptr : a.state + (uint64_t)slot * a.heads * DK * a.value_dim + head_at;
  Scan<DK> scan{a, sh, q, base, h, h / a.group, col, lane, n, c, group, j0, j1};
  const uint32_t role = wave / kScanGroups;
  if (role < 2) scan.states(role, j0 ? a.carry[0] + head_at : kept, j1 < chunks ? a.carry[1] + head_at : kept);
  else scan.outputs(role - 2);
}

template <int DK>
int launch(Delta& a, uint32_t all, hipStream_t s) {
  float* carry[2] = {a.carry[0], a.carry[1]};
  for (uint32_t first = 0, i = 0; first < all; first += a.places, ++i) {
    a.place0 = first;
    a.carry[0] = carry[i % 2];
    a.carry[1] = carry[(i + 1) % 2];
    const uint64_t items = (uint64_t)(all - first < a.places ? all - first : a.places) * (a.heads / a.group) * ((a.group + kPair - 1) / kPair);
    a.seqs = a.n_seqs < a.places ? a.n_seqs : a.places;   // a sequence has a place at least
    // heads of a key head together where no chiplet's 32 compute units get more workgroups than otherwise, or all at once (us
    // in a graph, together and each head by itself: 5 sequences of 300 tokens, 16 heads of 128 on 8 45.5 and 49.9; 9 up to 1111, 8
    // heads on 4 52.7 and 54.9; one of 8192, 48 heads on 16 363 and 365; nine key heads, each chiplet by turns: one of 2048, 54 heads
    // 161 and 104, one of 1024, 108 heads of 64 x 128 113 and 86)
    const uint64_t units = (uint64_t)a.seqs * (a.heads / a.group), each = (units + 7) / 8 * a.group * a.slices;
    a.together = units % 8 == 0 || each <= 32 ? a.group : 1;
    const uint64_t blocks = a.together > 1 ? each * 8 : ((uint64_t)a.seqs * a.heads + 7) / 8 * 8 * a.slices;
    // (at most 256 MB of places, 32 KB a head: both are far below what a launch takes)
    hipLaunchKernelGGL((k_delta_chunk<DK>), dim3((uint32_t)items), dim3(256), 0, s, a);
    hipLaunchKernelGGL((k_delta_scan<DK>), dim3((uint32_t)blocks), dim3(256 * kScanGroups), 0, s, a);
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
