// Causal convolution of a few taps for each channel, over rows packed by
// sequence, with the rows before a call kept in a state (gfx950):
//     y[t][c] = f(bias[c] + sum_j w[c][j] x[t - taps + 1 + j][c])
//
// One pass over memory, bound by its bandwidth for many rows and by a few round
// trips for few.  A thread takes 16 bytes of channels and walks down a tile of rows
// with the window in registers, so that a row is read once but for the taps - 1 rows
// above each tile.  Rows that need the state, a sequence's first taps - 1, belong to
// the tile of the sequence's first row, whichever tile they lie in: the thread
// that reads a state is then the only one that does, and writes the new one after.
#include <hip/hip_runtime.h>

#include "wal_args.h"
#include "wal_device.h"
#include "wal_find.h"
#include "wal_seq.h"

namespace {

constexpr uint32_t kAhead = 4;   // rows loaded at once

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
template <bool BF16, int V>
__device__ __forceinline__ void load(const char* p, uint64_t e, float (&v)[V]) {
  if constexpr (BF16) {
    uint32_t w[V / 2];
    if constexpr (V == 8) {
      const u32x4_t r = *reinterpret_cast<const u32x4_t*>(p + 2 * e);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = r[i];
    } else {
      const u32x2_t r = *reinterpret_cast<const u32x2_t*>(p + 2 * e);
      w[0] = r[0];
      w[1] = r[1];
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const f32x4_t r = reinterpret_cast<const f32x4_t*>(p + 4 * e)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = r[j];
    }
  }
}

template <int V>
__device__ __forceinline__ void store(char* p, uint64_t e, const float (&v)[V], bool bf16) {
  if (bf16) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const bf16x2_t b = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};   // to nearest even, NaN kept
      w[i] = __builtin_bit_cast(uint32_t, b);
    }
    if constexpr (V == 8) *reinterpret_cast<u32x4_t*>(p + 2 * e) = u32x4_t{w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<u32x2_t*>(p + 2 * e) = u32x2_t{w[0], w[1]};
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      reinterpret_cast<f32x4_t*>(p + 4 * e)[i] = f32x4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
  }
}

// Rows of BF16 or fp32 x, V channels of 16 bytes to a thread.
template <bool BF16, int TAPS>
__global__ __launch_bounds__(256) void k_conv(Conv a) {
  constexpr int V = BF16 ? 8 : 4, H = TAPS - 1;   // H rows of history
  const uint32_t lane = threadIdx.x & 63, c = (blockIdx.x * blockDim.x + threadIdx.x) * V;
  const bool mine = c < a.channels;
  const int32_t t0 = (int32_t)(blockIdx.y * a.tile), t1 = (int32_t)min(t0 + a.tile, a.n);
  float w[TAPS][V], bias[V];
  if (mine) {
    // V * TAPS weights side by side, in pieces of V
    float all[TAPS * V];
#pragma unroll
    for (int i = 0; i < TAPS; ++i) {
      float part[V];
      if (a.w_bf16) load<true, V>(a.weight, (uint64_t)c * TAPS + i * V, part);
      else load<false, V>(a.weight, (uint64_t)c * TAPS + i * V, part);
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
      load<true, V>(a.bias, c, bias);
    } else {
      load<false, V>(a.bias, c, bias);
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
          load<BF16, V>(a.x, (uint64_t)p * a.ldx + c, win[j]);
        } else if (kept) {
          load<BF16, V>(a.state, kept_at + (uint64_t)(H + p - q.first) * a.channels, win[j]);
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
          if (p >= q.first) load<BF16, V>(a.x, (uint64_t)p * a.ldx + c, last[j]);
          else
#pragma unroll
            for (int k = j; k < H; ++k)
              if (k == H + p - q.first)
#pragma unroll
                for (int i = 0; i < V; ++i) last[j][i] = win[k][i];
        }
#pragma unroll
        for (int j = 0; j < H; ++j) store<V>(a.state, kept_at + (uint64_t)j * a.channels, last[j], BF16);
      }
      for (int32_t r = t; r < stop; r += kAhead) {
        float row[kAhead][V];
#pragma unroll
        for (int u = 0; u < (int)kAhead; ++u) load<BF16, V>(a.x, (uint64_t)min(r + u, stop - 1) * a.ldx + c, row[u]);
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
          if (r + u < stop) store<V>(a.out, (uint64_t)(r + u) * a.ldo + c, y, a.out_bf16);
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
void launch(const Conv& a, uint32_t taps, dim3 grid, dim3 block, hipStream_t s) {
  if (taps == 2) hipLaunchKernelGGL((k_conv<BF16, 2>), grid, block, 0, s, a);
  if (taps == 3) hipLaunchKernelGGL((k_conv<BF16, 3>), grid, block, 0, s, a);
  if (taps == 4) hipLaunchKernelGGL((k_conv<BF16, 4>), grid, block, 0, s, a);
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
  const uint32_t groups = channels / (x_dtype == WAL_X_BF16 ? 8 : 4);
  // Long tiles read little above them twice, short ones fill the GPU with few rows.
  const uint64_t work = (uint64_t)n * groups;
  a.tile = work >= (32ull << 18) ? 32 : work >= (8ull << 18) ? 8 : 4;
  while (((uint64_t)n + a.tile - 1) / a.tile > 65535) a.tile *= 2;
  const uint32_t threads = groups >= 16384 || work >= (1u << 18) ? 256 : 64;
  const dim3 grid((groups + threads - 1) / threads, (n + a.tile - 1) / a.tile), block(threads);
  if (x_dtype == WAL_X_BF16) launch<true>(a, taps, grid, block, static_cast<hipStream_t>(stream));
  else launch<false>(a, taps, grid, block, static_cast<hipStream_t>(stream));
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}
