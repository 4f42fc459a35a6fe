// Causal convolution of a few taps for each channel, over rows packed by
// sequence, with the rows before a call kept in a state (gfx950):
//     y[t][c] = f(bias[c] + sum_j w[c][j] x[t - taps + 1 + j][c])
//
// One pass over memory, bound by its bandwidth for many rows and by a few round
// trips for few.  A thread takes four channels and walks down a tile of rows
// with the window in registers, so that a row is read once but for the taps - 1 rows
// above each tile.  Rows that need the state, a sequence's first taps - 1, belong to
// the tile of the sequence's first row, whichever tile they lie in: the thread
// that reads a state is then the only one that does, and writes the new one after.
//
// Measured (4 taps, in a graph): fp32 to bf16, 17 000 tokens of 8192 channels in 7 prompts 141 us, 4.8 TB/s (a copy
// reaches 5.0); one token of 10240 channels 4.5 us, 64 sequences of one 7.6 us.
#include <hip/hip_runtime.h>

#include "wal_args.h"
#include "wal_device.h"
#include "wal_find.h"
#include "wal_seq.h"

namespace {

constexpr uint32_t kConvThreads = 64;   // (256 are as fast, and slower where channels are few)
constexpr uint32_t kAhead = 4;      // rows loaded at once
constexpr int V = 4;                // channels of a thread (8 of bf16, 16 bytes, take twice the registers: 64 sequences of one
                                    // token 8.4 us for 7.3, 8000 rows within 2 %)

struct Conv {
  const char* x;
  const char* weight;
  const char* bias;
  const int32_t* starts;
  const int32_t* slots;
  char* state;
  char* out;
  uint64_t ldx, ldo;
  uint32_t n, channels, n_seqs, n_slots, tile, w_bf16, out_bf16, silu;
};

// V values at element e of p as floats.
template <bool BF16>
__device__ __forceinline__ void load(const char* p, uint64_t e, float (&v)[V]) {
  if constexpr (BF16) {
    const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p + 2 * e);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const f32x4_t w = *reinterpret_cast<const f32x4_t*>(p + 4 * e);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = w[i];
  }
}

__device__ __forceinline__ void store(char* p, uint64_t e, const float (&v)[V], bool bf16) {
  if (bf16) {
    const bf16x2_t lo = {(__bf16)v[0], (__bf16)v[1]}, hi = {(__bf16)v[2], (__bf16)v[3]};   // to nearest even, NaN kept
    *reinterpret_cast<u32x2_t*>(p + 2 * e) = u32x2_t{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
  } else {
    *reinterpret_cast<f32x4_t*>(p + 4 * e) = f32x4_t{v[0], v[1], v[2], v[3]};
  }
}

// Rows of BF16 or fp32 x, V channels to a thread.
template <bool BF16, int TAPS>
__global__ __launch_bounds__(kConvThreads) void k_conv(Conv a) {
  constexpr int H = TAPS - 1;   // rows of history
  const uint32_t lane = threadIdx.x, c = (blockIdx.x * kConvThreads + lane) * V;
  const bool mine = c < a.channels;
  const int32_t t0 = (int32_t)(blockIdx.y * a.tile), t1 = (int32_t)min(t0 + a.tile, a.n);
  float w[TAPS][V], bias[V];
  if (mine) {
    // V * TAPS weights side by side, in pieces of V
    float all[TAPS * V];
#pragma unroll
    for (int i = 0; i < TAPS; ++i) {
      float part[V];
      if (a.w_bf16) load<true>(a.weight, (uint64_t)c * TAPS + i * V, part);
      else load<false>(a.weight, (uint64_t)c * TAPS + i * V, part);
#pragma unroll
      for (int j = 0; j < V; ++j) all[i * V + j] = part[j];
    }
#pragma unroll
    for (int j = 0; j < TAPS; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) w[j][i] = all[i * TAPS + j];
    if (!a.bias) {
#pragma unroll
      for (int i = 0; i < V; ++i) bias[i] = 0.f;
    } else if (a.w_bf16) {
      load<true>(a.bias, c, bias);
    } else {
      load<false>(a.bias, c, bias);
    }
  }
  for (int32_t t = t0; t < t1;) {
    const uint32_t s = seq_at(a.starts, a.n_seqs, t, lane);
    const Seq q = cut_seq(a.starts[s], a.starts[s + 1], 0, (int32_t)a.n, (int32_t)a.n, (int32_t)a.n, false);
    const int32_t end = q.first + q.rows;
    if (t < q.first) {   // before the first sequence
      t = q.first;
      continue;
    }
    if (t >= end) return;   // behind the last one
    if (q.first < t0 && t - q.first < H) {   // rows of the tile before
      t = min(q.first + H, end);
      continue;
    }
    const int32_t stop = min(max(t1, q.first >= t0 ? q.first + H : 0), end);
    if (mine) {
      const uint32_t slot = a.slots ? (uint32_t)a.slots[s] : 0xFFFFFFFFu;
      const bool kept = a.state && slot < a.n_slots;
      const uint64_t kept_at = (uint64_t)slot * H * a.channels + c;
      float win[H][V];
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const int32_t p = t - H + j;
        if (p >= q.first) {
          load<BF16>(a.x, (uint64_t)p * a.ldx + c, win[j]);
        } else if (kept) {
          load<BF16>(a.state, kept_at + (uint64_t)(H + p - q.first) * a.channels, win[j]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) win[j][i] = 0.f;
        }
      }
      if (kept && t == q.first) {
        // the last H rows: at the sequence's first row the window is the old state
        float last[H][V];
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const int32_t p = end - H + j;
          if (p >= q.first) load<BF16>(a.x, (uint64_t)p * a.ldx + c, last[j]);
          else
#pragma unroll
            for (int k = j; k < H; ++k)
              if (k == H + p - q.first)
#pragma unroll
                for (int i = 0; i < V; ++i) last[j][i] = win[k][i];
        }
#pragma unroll
        for (int j = 0; j < H; ++j) store(a.state, kept_at + (uint64_t)j * a.channels, last[j], BF16);
      }
      for (int32_t r = t; r < stop; r += kAhead) {
        float row[kAhead][V];
#pragma unroll
        for (int u = 0; u < (int)kAhead; ++u) load<BF16>(a.x, (uint64_t)min(r + u, stop - 1) * a.ldx + c, row[u]);
#pragma unroll
        for (int u = 0; u < (int)kAhead; ++u) {
          float y[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            y[i] = bias[i];
#pragma unroll
            for (int j = 0; j < TAPS; ++j) {
              const int at = u + j - H;   // of the rows loaded here, below 0: of the window
              y[i] = fmaf(w[j][i], at < 0 ? win[(H + at) % H][i] : row[at < 0 ? 0 : at][i], y[i]);
            }
            if (a.silu) y[i] = y[i] / (1.f + expf(-y[i]));
          }
          if (r + u < stop) store(a.out, (uint64_t)(r + u) * a.ldo + c, y, a.out_bf16);
        }
#pragma unroll
        for (int j = 0; j < H; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) win[j][i] = row[kAhead - H + j][i];
      }
    }
    t = stop;
  }
}

template <bool BF16>
void launch(const Conv& a, uint32_t taps, dim3 grid, hipStream_t s) {
  if (taps == 2) hipLaunchKernelGGL((k_conv<BF16, 2>), grid, dim3(kConvThreads), 0, s, a);
  if (taps == 3) hipLaunchKernelGGL((k_conv<BF16, 3>), grid, dim3(kConvThreads), 0, s, a);
  if (taps == 4) hipLaunchKernelGGL((k_conv<BF16, 4>), grid, dim3(kConvThreads), 0, s, a);
}

}  // namespace

extern "C" int wal_conv(const void* x_dev, int x_dtype, uint32_t n, uint32_t channels, uint32_t ldx,
                        const void* weight_dev, int w_dtype, uint32_t taps, const void* bias_dev, int silu,
                        const int32_t* starts_dev, uint32_t n_seqs, void* state_dev, const int32_t* slots_dev,
                        uint32_t n_slots, void* out_dev, int out_dtype, uint32_t ldo, void* stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype) || !dtype_ok(w_dtype)) return WAL_ERR_ARG;
  if (!weight_dev || !starts_dev || !state_dev != !slots_dev) return WAL_ERR_ARG;
  if (!channels || channels % 8 || channels > (1u << 24) || taps < 2 || taps > 4 || n > (1u << 24) ||
      n_seqs > (1u << 24) || n_slots > (1u << 24))
    return WAL_ERR_SHAPE;
  int st;
  if ((st = check_rows(x_dev, ldx, channels, x_dtype)) || (st = check_rows(out_dev, ldo, channels, out_dtype))) return st;
  if (!aligned(weight_dev, 16) || !aligned(bias_dev, 16) || !aligned(state_dev, 16) || !aligned(starts_dev, 4) ||
      !aligned(slots_dev, 4))
    return WAL_ERR_ALIGN;
  const uint64_t xb = elem_bytes(x_dtype), wb = elem_bytes(w_dtype);
  const Rows out = rows(out_dev, n, ldo, channels, elem_bytes(out_dtype));
  const Rows state = state_dev ? flat(state_dev, (uint64_t)n_slots * (taps - 1) * channels * xb) : Rows{};
  const Rows in[5] = {rows(x_dev, n, ldx, channels, xb), flat(weight_dev, wb * channels * taps),
                      bias_dev ? flat(bias_dev, wb * channels) : Rows{}, flat(starts_dev, 4ull * (n_seqs + 1ull)),
                      slots_dev ? flat(slots_dev, 4ull * n_seqs) : Rows{}};
  for (const Rows& r : in)
    if (meet(r, out) || meet(r, state)) return WAL_ERR_ARG;
  if (meet(out, state)) return WAL_ERR_ARG;
  if (!n || !n_seqs) return WAL_OK;
  Conv a{};
  a.x = static_cast<const char*>(x_dev);
  a.weight = static_cast<const char*>(weight_dev);
  a.bias = static_cast<const char*>(bias_dev);
  a.starts = starts_dev;
  a.slots = slots_dev;
  a.state = static_cast<char*>(state_dev);
  a.out = static_cast<char*>(out_dev);
  a.ldx = ldx;
  a.ldo = ldo;
  a.n = n;
  a.channels = channels;
  a.n_seqs = n_seqs;
  a.n_slots = n_slots;
  a.w_bf16 = w_dtype == WAL_X_BF16;
  a.out_bf16 = out_dtype == WAL_X_BF16;
  a.silu = silu ? 1 : 0;
  const uint32_t groups = channels / 4;
  // Rows of a tile.  As many sequences as rows, or half as many where there is little work: one each, since a tile walks its
  // sequences one after another, and there is little above a row to read again (fp32, tiles of one row and those below:
  // 64 of one token, 10240 channels 8.2 and 15.2 us, 1000 of them 77 and 79; 63 of one token and one of 64, 10240 channels 10.5 and
  // 16.6; 999 of one and one of 1000, 1024 channels 14 and 18.5, 8192 channels 95 and 79; 255 of one and one of 256, 8192
  // channels 23 and 22; 2000 of two, 1024 channels 25 and 17.5; one of 1000 and 999 without rows, 8192 channels 36 and 15, which
  // the host cannot tell from 1000 of one, 64 and 70).  Else long tiles read little above them twice and short ones fill the
  // GPU (fp32, 8192 channels, tiles of 4, 8 and 16: 1000 rows 13.9, 14.6 and 16.6 us, 4000 rows 51, 46 and 51, 16000 rows 189,
  // 156 and 160; bf16: 1000 rows 14, 14 and 15, 4000 rows 51, 42 and 41, 8000 rows 98, 75 and 68, with tiles of 32 73).
  const bool bf16 = x_dtype == WAL_X_BF16;
  const uint64_t work = (uint64_t)n * groups;
  a.tile = n <= n_seqs || (n <= 2ull * n_seqs && work < (1ull << 19)) ? 1 : work < (8ull << 18) ? 4 : bf16 && work >= (32ull << 18) ? 16 : 8;
  while (((uint64_t)n + a.tile - 1) / a.tile > 65535) a.tile *= 2;
  const dim3 grid((groups + kConvThreads - 1) / kConvThreads, (n + a.tile - 1) / a.tile);
  if (bf16) launch<true>(a, taps, grid, static_cast<hipStream_t>(stream));
  else launch<false>(a, taps, grid, static_cast<hipStream_t>(stream));
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}
