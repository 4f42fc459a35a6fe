// The gated delta rule token by token for gfx950 (decode): for each value head a
// state S [key_dim][value_dim] in fp32,
//     u = b (v - a S^T k),  S <- a S + k u^T,  o = S^T q
// with S^T k and S^T q of the old state in one pass over it, since the new one's
// S^T q is a S^T q + (k . q) u.
//
// Bound by the bytes of the states, each read and written once however many tokens
// a sequence has in the call.  A workgroup takes 32 columns of one head of one
// sequence, or 64: a wavefront's load covers whole 128-byte lines, a thread keeps some rows of
// four columns in registers, and sums over rows meet by lane exchange in a
// wavefront and once in LDS, summed in one order by every wavefront.
//
// Measured (16 key and 48 value heads of 128): 64 sequences 85 us, 4.8 TB/s (a copy reaches 5.0); one sequence 5.8 us.
#include <hip/hip_runtime.h>

#include "wal_delta.h"

namespace {

constexpr uint32_t kThreads = 256, kWaves = kThreads / 64;

// A token's rows as a thread needs them.
template <int J>
struct Token {
  float q[J], k[J];
  f32x4_t v;
  Gates g;
};

template <int J>
__device__ __forceinline__ void load_row(const uint16_t* p, float (&x)[J]) {
  uint32_t w[J / 2];
  if constexpr (J >= 8) {
#pragma unroll
    for (int i = 0; i < J / 8; ++i) {
      const u32x4_t r = reinterpret_cast<const u32x4_t*>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = r[j];
    }
  } else if constexpr (J == 4) {
    const u32x2_t r = *reinterpret_cast<const u32x2_t*>(p);
    w[0] = r[0];
    w[1] = r[1];
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
#pragma unroll
  for (int i = 0; i < J / 2; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <int DK, int NV>
__global__ __launch_bounds__(kThreads) void k_delta_step(Delta a) {
  constexpr uint32_t kCols = NV / 4;               // threads side by side
  constexpr int J = DK / (int)(kThreads / kCols);  // rows of a thread
  constexpr int kSums = 11;             // S^T k and S^T q of four columns, k . k, q . q, k . q
  __shared__ float sums[2][kWaves][kCols][kSums + 1];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = threadIdx.x % kCols, r = threadIdx.x / kCols;
  const uint32_t slices = a.value_dim / NV, slice = blockIdx.x % slices, rest = blockIdx.x / slices, h = rest % a.heads, s = a.seq0 + rest / a.heads;
  const Seq seq = delta_seq(a, s);
  if (!seq.rows || seq.rows > a.few) return;
  const int64_t slot = kept_at(a, s);
  const uint32_t kh = h / a.group, col = NV * slice + 4 * c;
  float* state = a.state + ((uint64_t)max(slot, (int64_t)0) * a.heads + h) * DK * a.value_dim + (uint64_t)(J * r) * a.value_dim + col;
  const auto token = [&](int32_t i) {
    Token<J> t;
    const uint64_t row = (uint64_t)(seq.first + i);
    load_row<J>(a.q + row * a.ldq + kh * DK + J * r, t.q);
    load_row<J>(a.k + row * a.ldk + kh * DK + J * r, t.k);
    float v[4];
    load_row<4>(a.v + row * a.ldv + h * a.value_dim + col, v);
    t.v = f32x4_t{v[0], v[1], v[2], v[3]};
    t.g = gates_of(a, row, h);
    return t;
  };
  Token<J> t = token(0);
  f32x4_t m[J];
#pragma unroll
  for (int j = 0; j < J; ++j)
    m[j] = slot < 0 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : *reinterpret_cast<const f32x4_t*>(state + (uint64_t)j * a.value_dim);
  for (int32_t i = 0; i < seq.rows; ++i) {
    const Token<J> next = token(min(i + 1, seq.rows - 1));
    float x[kSums] = {};
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = fmaf(t.k[j], m[j][e], x[e]);
        x[4 + e] = fmaf(t.q[j], m[j][e], x[4 + e]);
      }
      x[8] = fmaf(t.k[j], t.k[j], x[8]);
      x[9] = fmaf(t.q[j], t.q[j], x[9]);
      x[10] = fmaf(t.k[j], t.q[j], x[10]);
    }
#pragma unroll
    for (int e = 0; e < kSums; ++e)
#pragma unroll
      for (int d = kCols; d < 64; d *= 2) x[e] += __shfl_xor(x[e], d);
    if (lane < kCols)
#pragma unroll
      for (int e = 0; e < kSums; ++e) sums[i & 1][wave][c][e] = x[e];
    __syncthreads();   // (two buffers: the next token's sums go to the other one)
#pragma unroll
    for (int e = 0; e < kSums; ++e) {
      x[e] = sums[i & 1][0][c][e];
#pragma unroll
      for (int w = 1; w < (int)kWaves; ++w) x[e] += sums[i & 1][w][c][e];
    }
    const float rk = unit(a, x[8]), rq = unit(a, x[9]) * a.scale, alpha = expf(t.g.log_alpha), kq = x[10] * rk;
    f32x4_t u, o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[e] = t.g.beta * fmaf(-alpha * rk, x[e], t.v[e]);
      o[e] = rq * fmaf(alpha, x[4 + e], kq * u[e]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float k = rk * t.k[j];
#pragma unroll
      for (int e = 0; e < 4; ++e) m[j][e] = fmaf(k, u[e], alpha * m[j][e]);
    }
    if (r == 0) {
      const bf16x2_t lo = {(__bf16)o[0], (__bf16)o[1]}, hi = {(__bf16)o[2], (__bf16)o[3]};
      *reinterpret_cast<u32x2_t*>(a.out + (uint64_t)(seq.first + i) * a.ldo + h * a.value_dim + col) =
          u32x2_t{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    }
    t = next;
  }
  if (slot >= 0)
#pragma unroll
    for (int j = 0; j < J; ++j) *reinterpret_cast<f32x4_t*>(state + (uint64_t)j * a.value_dim) = m[j];
}

// A launch has fewer than 2^32 threads along an axis: of more sequences than that allows, several.
template <int DK, int NV>
void launch(Delta a, hipStream_t s) {
  const uint32_t each = a.heads * (a.value_dim / NV), most = 0xFFFFFFFFu / kThreads / each;
  for (a.seq0 = 0; a.seq0 < a.n_seqs; a.seq0 += most)
    hipLaunchKernelGGL((k_delta_step<DK, NV>), dim3((a.n_seqs - a.seq0 < most ? a.n_seqs - a.seq0 : most) * each), dim3(kThreads), 0, s, a);
}

// Columns of a workgroup: 64 where that makes two workgroups for each compute unit, else 32 (key heads of 128, 64 sequences
// of 48 heads 85 us and 92 with 32; 13 sequences of up to 5 tokens, 32 heads 20 and 27; one sequence of 48 heads 6.1 and
// 5.8).  128 are no faster (86, 20 and 7.0 us).
template <int DK>
void launch(const Delta& a, hipStream_t s) {
  if (a.value_dim % 64 == 0 && (uint64_t)a.n_seqs * a.heads * (a.value_dim / 64) >= 512) launch<DK, 64>(a, s);
  else launch<DK, 32>(a, s);
}

}  // namespace

namespace wal {

int delta_step(const Delta& a, uint32_t key_dim, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (key_dim == 64) launch<64>(a, s);
  else launch<128>(a, s);
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}

}  // namespace wal
