// Rotary positions and the rows of the paged key/value cache for gfx950:
//     (a, b) -> m (a cos p f - b sin p f, b cos p f + a sin p f)
// for every pair of a head at position p, and the row formats of
// include/wal.h (bf16, or int8 codes with one fp32 scale per token and head).
//
// All three calls are one pass over memory, bound by its bandwidth for many
// tokens and by one round trip for few.  The work is cut into units of 16
// elements of one head: eight pairs (two pieces of eight elements in the half
// layout, 16 neighbours in the interleaved one) or 16 unrotated elements, so
// every access is 16 bytes a lane and the D / 16 lanes of a head sit side by
// side for the row maximum.  A workgroup takes whole tokens; it computes the
// sines of its tokens once, into LDS, for all their heads, while the first
// units' loads are on their way.
//
// Angles: a position times a frequency in units of 2^-64 turns, mod 2^64, is
// the exact fraction of a turn in one 64-bit product; its top 32 bits give
// the quadrant (2 bits) and the rest, |angle| <= pi / 4, goes through the Taylor
// sums of sine and cosine in fp32 (next terms below 2e-9).  In fp32 the
// product itself would be off by 0.06 rad at position 10^6.
//
// Measured: 16001 tokens of 40 heads of 128 rotated bf16 to bf16 66 us (5.0 TB/s; a copy
// reaches 5.2), 8191 tokens written as int8 with their q rows 52 us, 100003 tokens
// read back from int8 123 us (5.0 TB/s); one token of 32 heads 2.3 us.
#include <hip/hip_runtime.h>

#include "wal_args.h"
#include "wal_device.h"

namespace {

constexpr uint32_t kRopeThreads = 256;
constexpr uint32_t kRopeLdsPairs = 1024;   // sines of one workgroup's tokens, 8 KB
constexpr uint32_t kMaxRopeDim = 512;      // at most 256 pairs a token

struct RopeKv {
  const char* q;                  // the q rows, and from there to the k rows, from those to the v rows
  int64_t to_k, to_v;             // (bytes; pitches likewise: sums of what a unit's kind selects stay in registers)
  int64_t ldq, ld_to_k, ld_to_v;  // pitches, elements
  void* q_out;
  uint8_t* cache;
  const int32_t* slots;
  const uint64_t* turns;
  const int32_t* pos;
  uint64_t ldqo;
  uint64_t off_k, k_to_v, off_ks, ks_to_vs;   // bytes from the cache's start, from plane to plane
  float magnitude;
  uint32_t n, tokens;             // tokens of the call, of a workgroup
  uint32_t slice;                 // units of a token that a workgroup takes
  uint32_t units, q_units, k_units;   // units of a token, of its q and its k heads
  uint32_t per_head, rot_units;   // units of a head, rotated ones among them
  uint32_t rot, n_slots, page_shift, kv_heads, dim;
  uint32_t interleaved, out_bf16, int8;
};

__device__ __forceinline__ float2 turn(int32_t pos, uint64_t t, float m) {
  const uint32_t f = (uint32_t)(((uint64_t)(int64_t)pos * t) >> 32);
  const uint32_t quad = (f + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(f - (quad << 30)) * 1.4629180792671596e-9f;   // 2 pi 2^-32
  const float z = x * x;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(z * x, s, x);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  const float cs = (quad & 1) ? s : c, sn = (quad & 1) ? c : s;
  return make_float2((quad == 1 || quad == 2) ? -cs * m : cs * m, (quad & 2) ? -sn * m : sn * m);
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float2 w) {
  const float p = a, q = b;
  a = p * w.x - q * w.y;
  b = q * w.x + p * w.y;
}

// Eight elements at p.
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, uint64_t e, float* v) {
  if constexpr (BF16) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const f32x4_t* src = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + e);
    const f32x4_t a = src[0], b = src[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

__device__ __forceinline__ u32x4_t pack8(const float* v) {
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2_t b = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};   // to nearest even, NaN kept
    w[i] = __builtin_bit_cast(uint32_t, b);
  }
  return w;
}

__device__ __forceinline__ void store8(void* p, uint64_t e, const float* v, bool bf16) {
  if (bf16) {
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + e) = pack8(v);
  } else {
    f32x4_t* d = reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + e);
    d[0] = f32x4_t{v[0], v[1], v[2], v[3]};
    d[1] = f32x4_t{v[4], v[5], v[6], v[7]};
  }
}

__device__ __forceinline__ u32x2_t codes8(const float* v, float inv) {
  u32x2_t w = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i / 4] |= ((uint32_t)(int)rintf(v[i] * inv) & 0xFFu) << (8 * (i % 4));
  return w;
}

// One unit: where it comes from and goes to.
struct Unit {
  uint32_t t, kind, head, j;   // token, 0 q / 1 k / 2 v, head, unit of the head
  uint32_t lo, hi;             // element of its two pieces of eight in the head
  bool rotated;
};

__device__ __forceinline__ Unit unit_of(const RopeKv& a, uint32_t t, uint32_t u) {
  Unit x;
  x.t = t;
  x.kind = u < a.q_units ? 0u : u < a.q_units + a.k_units ? 1u : 2u;
  const uint32_t w = x.kind == 0 ? u : x.kind == 1 ? u - a.q_units : u - a.q_units - a.k_units;
  x.head = w / a.per_head;
  x.j = w - x.head * a.per_head;
  x.rotated = x.kind < 2 && x.j < a.rot_units;
  const bool split = x.rotated && !a.interleaved;
  x.lo = split ? 8 * x.j : 16 * x.j;
  x.hi = split ? a.rot / 2 + 8 * x.j : 16 * x.j + 8;
  return x;
}

template <bool BF16>
__device__ __forceinline__ void load_unit(const RopeKv& a, const Unit& x, float* v) {
  const char* p = a.q + (x.kind ? a.to_k : 0) + (x.kind == 2 ? a.to_v : 0);
  const uint64_t at = x.t * (uint64_t)(a.ldq + (x.kind ? a.ld_to_k : 0) + (x.kind == 2 ? a.ld_to_v : 0)) +
                      x.head * a.dim;
  load8<BF16>(p, at + x.lo, v);
  load8<BF16>(p, at + x.hi, v + 8);
}

template <bool BF16>
__global__ __launch_bounds__(kRopeThreads) void k_rope_kv(RopeKv a) {
  __shared__ float2 cs[kRopeLdsPairs];
  const uint32_t t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.n - t0);
  const uint32_t u0 = blockIdx.y * a.slice, nu = min(a.slice, a.units - u0), total = nt * nu;
  uint32_t i = threadIdx.x;
  Unit x{};
  float v[16];
  if (i < total) {
    const uint32_t t = i / nu;
    x = unit_of(a, t0 + t, u0 + i - t * nu);
    load_unit<BF16>(a, x, v);
  }
  const uint32_t pairs = a.rot / 2;
  if (pairs) {
    for (uint32_t p = threadIdx.x; p < nt * pairs; p += kRopeThreads) {
      const uint32_t t = p / pairs;
      cs[p] = turn(a.pos[t0 + t], a.turns[p - t * pairs], a.magnitude);
    }
    __syncthreads();
  }
  while (i < total) {
    if (x.rotated) {
      const float2* c = cs + (x.t - t0) * pairs + 8 * x.j;
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(v[2 * e], v[2 * e + 1], c[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(v[e], v[8 + e], c[e]);
      }
    }
    if (x.kind == 0) {
      const uint64_t at = x.t * a.ldqo + x.head * a.dim;
      store8(a.q_out, at + x.lo, v, a.out_bf16);
      store8(a.q_out, at + x.hi, v + 8, a.out_bf16);
    } else {
      // the row maximum first: every lane of the head takes part
      float inv = 0.f, scale = 0.f;
      if (a.int8) {
        uint32_t top = 0;   // of |x| as bits: NaN above infinity above numbers
#pragma unroll
        for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        for (uint32_t m = 1; m < a.per_head; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, (int)m));
        if (top >= 0x7F800000u) {
          scale = __uint_as_float(0x7FC00000u);
        } else if (top >= 0x0D800000u) {   // 2^-100
          inv = 127.0f / __uint_as_float(top);
          scale = __uint_as_float(top) * (1.0f / 127.0f);
        }
      }
      const uint32_t slot = (uint32_t)a.slots[x.t];
      if (slot < a.n_slots) {
        const uint64_t page = slot >> a.page_shift, at = slot & ((1u << a.page_shift) - 1);
        const uint64_t row = ((page * a.kv_heads + x.head) << a.page_shift) + at;
        uint8_t* plane = a.cache + a.off_k + (x.kind == 2 ? a.k_to_v : 0);
        if (a.int8) {
          if (!(inv > 0.f)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
          }
          *reinterpret_cast<u32x2_t*>(plane + row * a.dim + x.lo) = codes8(v, inv);
          *reinterpret_cast<u32x2_t*>(plane + row * a.dim + x.hi) = codes8(v + 8, inv);
          if (x.j == 0) reinterpret_cast<float*>(a.cache + a.off_ks + (x.kind == 2 ? a.ks_to_vs : 0))[row] = scale;
        } else {
          *reinterpret_cast<u32x4_t*>(plane + 2 * (row * a.dim + x.lo)) = pack8(v);
          *reinterpret_cast<u32x4_t*>(plane + 2 * (row * a.dim + x.hi)) = pack8(v + 8);
        }
      }
    }
    i += kRopeThreads;
    if (i < total) {
      const uint32_t t = i / nu;
      x = unit_of(a, t0 + t, u0 + i - t * nu);
      load_unit<BF16>(a, x, v);
    }
  }
}

struct KvRead {
  const uint8_t* cache;
  const int32_t* slots;
  char* out;
  int64_t out_to_v;               // bytes from the k rows of the output to the v rows
  int64_t ld, ld_to_v;
  uint64_t off, off_to_v, off_s, off_s_to_v;
  uint32_t n, units, per_head_shift, n_slots, page_shift, kv_heads, dim, int8, out_bf16;
};

// A thread reads 16 elements of a row: 16 bytes of codes and the row's scale, or
// 32 bytes of bf16.
__global__ __launch_bounds__(kRopeThreads) void k_kv_read(KvRead a) {
  const uint64_t i = (uint64_t)blockIdx.x * kRopeThreads + threadIdx.x;
  const uint32_t t = (uint32_t)(i / a.units), u = (uint32_t)(i - (uint64_t)t * a.units);
  const bool z = blockIdx.y;
  if (t >= a.n) return;
  const uint32_t head = u >> a.per_head_shift, e = 16 * (u & ((1u << a.per_head_shift) - 1));
  const uint32_t slot = (uint32_t)a.slots[t];
  float v[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = 0.f;
  if (slot < a.n_slots) {
    const uint64_t page = slot >> a.page_shift, at = slot & ((1u << a.page_shift) - 1);
    const uint64_t row = ((page * a.kv_heads + head) << a.page_shift) + at;
    const uint8_t* plane = a.cache + a.off + (z ? a.off_to_v : 0);
    if (a.int8) {
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(plane + row * a.dim + e);
      const float s = reinterpret_cast<const float*>(a.cache + a.off_s + (z ? a.off_s_to_v : 0))[row];
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = (float)(int8_t)(w[k / 4] >> (8 * (k % 4))) * s;
    } else {
      load8<true>(plane, row * a.dim + e, v);
      load8<true>(plane, row * a.dim + e + 8, v + 8);
    }
  }
  const uint64_t o = t * (uint64_t)(a.ld + (z ? a.ld_to_v : 0)) + (uint64_t)head * a.dim + e;
  char* out = a.out + (z ? a.out_to_v : 0);
  store8(out, o, v, a.out_bf16);
  store8(out, o + 8, v + 8, a.out_bf16);
}

int check_rotary(const wal_rotary* r, uint32_t head_dim) {
  if (!r || !r->turns_dev || !r->pos_dev) return WAL_ERR_ARG;
  if (r->layout > WAL_ROPE_INTERLEAVED) return WAL_ERR_ARG;
  if (!r->rot_dim || r->rot_dim % 16 || r->rot_dim > head_dim) return WAL_ERR_SHAPE;
  if (!aligned(r->turns_dev, 8) || !aligned(r->pos_dev, 4)) return WAL_ERR_ALIGN;
  return WAL_OK;
}

// Tokens of a workgroup and the slice of their units: whole tokens, about four units a thread
// when there are many, a unit a thread over more workgroups when there are few.
int launch(RopeKv& a, bool bf16_in, hipStream_t s) {
  const uint32_t by_lds = a.rot ? kRopeLdsPairs / (a.rot / 2) : 64;
  a.tokens = 1;
  a.slice = a.units;
  if ((uint64_t)a.n * a.units <= 512 * kRopeThreads) {
    a.slice = kRopeThreads / a.per_head * a.per_head;
    if (a.slice > a.units) a.slice = a.units;
  } else {
    while (a.tokens < by_lds && a.tokens * a.units < 4 * kRopeThreads) ++a.tokens;
  }
  const dim3 grid((a.n + a.tokens - 1) / a.tokens, (a.units + a.slice - 1) / a.slice);
  if (bf16_in)
    hipLaunchKernelGGL(k_rope_kv<true>, grid, dim3(kRopeThreads), 0, s, a);
  else
    hipLaunchKernelGGL(k_rope_kv<false>, grid, dim3(kRopeThreads), 0, s, a);
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}

}  // namespace

extern "C" int wal_rope(const void* x_dev, int x_dtype, uint32_t n, uint32_t heads, uint32_t head_dim, uint32_t ldx,
                        const wal_rotary* r, void* out_dev, int out_dtype, uint32_t ldo, void* stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype)) return WAL_ERR_ARG;
  if (!heads || heads > 65535 || !head_dim || head_dim % 16 || head_dim > kMaxRopeDim || n > (1u << 30))
    return WAL_ERR_SHAPE;
  int st = check_rotary(r, head_dim);
  if (st) return st;
  const uint64_t width = (uint64_t)heads * head_dim;
  if ((st = check_rows(x_dev, ldx, width, x_dtype)) || (st = check_rows(out_dev, ldo, width, out_dtype))) return st;
  const Rows xs = rows(x_dev, n, ldx, width, elem_bytes(x_dtype)), os = rows(out_dev, n, ldo, width, elem_bytes(out_dtype));
  const bool same = x_dev == out_dev && x_dtype == out_dtype && ldx == ldo;
  if (!same && meet(xs, os)) return WAL_ERR_ARG;
  if (meet(os, flat(r->pos_dev, 4ull * n)) || meet(os, flat(r->turns_dev, 4ull * r->rot_dim))) return WAL_ERR_ARG;
  if (!n) return WAL_OK;
  RopeKv a{};
  a.q = static_cast<const char*>(x_dev);
  a.q_out = out_dev;
  a.turns = r->turns_dev;
  a.pos = r->pos_dev;
  a.ldq = ldx;
  a.ldqo = ldo;
  a.magnitude = r->magnitude;
  a.n = n;
  a.per_head = head_dim / 16;
  a.units = a.q_units = heads * a.per_head;
  a.rot = r->rot_dim;
  a.rot_units = r->rot_dim / 16;
  a.dim = head_dim;
  a.interleaved = r->layout == WAL_ROPE_INTERLEAVED;
  a.out_bf16 = out_dtype == WAL_X_BF16;
  return launch(a, x_dtype == WAL_X_BF16, static_cast<hipStream_t>(stream));
}

extern "C" int wal_kv_write(const wal_kv_desc* d, void* cache_dev, const int32_t* slots_dev, uint32_t n,
                            const void* k_dev, uint32_t ldk, const void* v_dev, uint32_t ldv, int kv_dtype,
                            const wal_rotary* r, const void* q_dev, uint32_t q_heads, uint32_t ldq, void* q_out_dev,
                            uint32_t ldqo, void* stream) {
  wal_kv_info f;
  int st = wal_kv_size(d, &f);
  if (st) return st;
  if (!cache_dev || !slots_dev || !dtype_ok(kv_dtype)) return WAL_ERR_ARG;
  if (!q_dev != !q_out_dev || (q_dev && !r)) return WAL_ERR_ARG;
  if (n > (1u << 30) || (q_dev && (!q_heads || q_heads > 16384))) return WAL_ERR_SHAPE;
  if (r && (st = check_rotary(r, d->head_dim))) return st;
  const uint64_t width = (uint64_t)d->kv_heads * d->head_dim, qw = (uint64_t)q_heads * d->head_dim;
  if ((st = check_rows(k_dev, ldk, width, kv_dtype)) || (st = check_rows(v_dev, ldv, width, kv_dtype))) return st;
  if (q_dev && ((st = check_rows(q_dev, ldq, qw, kv_dtype)) || (st = check_rows(q_out_dev, ldqo, qw, WAL_X_BF16))))
    return st;
  if (!aligned(cache_dev, 256) || !aligned(slots_dev, 4)) return WAL_ERR_ALIGN;
  const uint32_t eb = elem_bytes(kv_dtype);
  const Rows cache = flat(cache_dev, f.total_bytes);
  const Rows qo = q_dev ? rows(q_out_dev, n, ldqo, qw, 2) : Rows{};
  const Rows in[5] = {rows(k_dev, n, ldk, width, eb), rows(v_dev, n, ldv, width, eb), flat(slots_dev, 4ull * n),
                      r ? flat(r->pos_dev, 4ull * n) : Rows{},
                      r ? flat(r->turns_dev, 4ull * r->rot_dim) : Rows{}};
  for (const Rows& s : in)
    if (meet(s, cache) || meet(s, qo)) return WAL_ERR_ARG;
  if (q_dev) {
    const Rows qs = rows(q_dev, n, ldq, qw, eb);
    const bool same = q_dev == q_out_dev && kv_dtype == WAL_X_BF16 && ldq == ldqo;
    if (meet(qs, cache) || meet(qo, cache) || (!same && meet(qs, qo))) return WAL_ERR_ARG;
  }
  if (!n) return WAL_OK;
  RopeKv a{};
  a.q = static_cast<const char*>(q_dev);
  a.to_k = reinterpret_cast<intptr_t>(k_dev) - reinterpret_cast<intptr_t>(q_dev);
  a.to_v = reinterpret_cast<intptr_t>(v_dev) - reinterpret_cast<intptr_t>(k_dev);
  a.q_out = q_out_dev;
  a.cache = static_cast<uint8_t*>(cache_dev);
  a.slots = slots_dev;
  if (r) {
    a.turns = r->turns_dev;
    a.pos = r->pos_dev;
    a.rot = r->rot_dim;
    a.rot_units = r->rot_dim / 16;
    a.interleaved = r->layout == WAL_ROPE_INTERLEAVED;
    a.magnitude = r->magnitude;
  }
  a.ldq = ldq;
  a.ld_to_k = (int64_t)ldk - ldq;
  a.ld_to_v = (int64_t)ldv - ldk;
  a.ldqo = ldqo;
  a.off_k = f.off_k;
  a.k_to_v = f.off_v - f.off_k;
  a.off_ks = f.off_ks;
  a.ks_to_vs = f.off_vs - f.off_ks;
  a.n = n;
  a.per_head = d->head_dim / 16;
  a.q_units = q_dev ? q_heads * a.per_head : 0;
  a.k_units = d->kv_heads * a.per_head;
  a.units = a.q_units + 2 * a.k_units;
  a.n_slots = d->n_pages * d->page_size;
  a.page_shift = (uint32_t)__builtin_ctz(d->page_size);
  a.kv_heads = d->kv_heads;
  a.dim = d->head_dim;
  a.out_bf16 = 1;
  a.int8 = d->fmt == WAL_KV_INT8;
  return launch(a, kv_dtype == WAL_X_BF16, static_cast<hipStream_t>(stream));
}

extern "C" int wal_kv_read(const wal_kv_desc* d, const void* cache_dev, const int32_t* slots_dev, uint32_t n,
                           void* k_out_dev, uint32_t ldk, void* v_out_dev, uint32_t ldv, int out_dtype,
                           void* stream) {
  wal_kv_info f;
  int st = wal_kv_size(d, &f);
  if (st) return st;
  if (!cache_dev || !slots_dev || (!k_out_dev && !v_out_dev) || !dtype_ok(out_dtype)) return WAL_ERR_ARG;
  if (n > (1u << 30)) return WAL_ERR_SHAPE;
  const uint64_t width = (uint64_t)d->kv_heads * d->head_dim;
  if (k_out_dev && (st = check_rows(k_out_dev, ldk, width, out_dtype))) return st;
  if (v_out_dev && (st = check_rows(v_out_dev, ldv, width, out_dtype))) return st;
  if (!aligned(cache_dev, 256) || !aligned(slots_dev, 4)) return WAL_ERR_ALIGN;
  const uint32_t eb = elem_bytes(out_dtype);
  const Rows cache = flat(cache_dev, f.total_bytes), sl = flat(slots_dev, 4ull * n);
  const Rows ko = k_out_dev ? rows(k_out_dev, n, ldk, width, eb) : Rows{};
  const Rows vo = v_out_dev ? rows(v_out_dev, n, ldv, width, eb) : Rows{};
  if (meet(ko, vo) || meet(ko, cache) || meet(vo, cache) || meet(ko, sl) || meet(vo, sl)) return WAL_ERR_ARG;
  if (!n) return WAL_OK;
  KvRead a{};
  a.cache = static_cast<const uint8_t*>(cache_dev);
  a.slots = slots_dev;
  if (k_out_dev) {
    a.out = static_cast<char*>(k_out_dev);
    a.ld = ldk;
    a.off = f.off_k;
    a.off_s = f.off_ks;
    if (v_out_dev) {
      a.out_to_v = reinterpret_cast<intptr_t>(v_out_dev) - reinterpret_cast<intptr_t>(k_out_dev);
      a.ld_to_v = (int64_t)ldv - ldk;
      a.off_to_v = f.off_v - f.off_k;
      a.off_s_to_v = f.off_vs - f.off_ks;
    }
  } else {
    a.out = static_cast<char*>(v_out_dev);
    a.ld = ldv;
    a.off = f.off_v;
    a.off_s = f.off_vs;
  }
  a.n = n;
  a.units = (uint32_t)(width / 16);
  a.per_head_shift = (uint32_t)__builtin_ctz(d->head_dim / 16);
  a.n_slots = d->n_pages * d->page_size;
  a.page_shift = (uint32_t)__builtin_ctz(d->page_size);
  a.kv_heads = d->kv_heads;
  a.dim = d->head_dim;
  a.int8 = d->fmt == WAL_KV_INT8;
  a.out_bf16 = out_dtype == WAL_X_BF16;
  const uint64_t blocks = ((uint64_t)n * a.units + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7FFFFFFFull) return WAL_ERR_SHAPE;
  hipLaunchKernelGGL(k_kv_read, dim3((uint32_t)blocks, k_out_dev && v_out_dev ? 2 : 1),
                     dim3(kRopeThreads), 0, static_cast<hipStream_t>(stream), a);
  return hipGetLastError() == hipSuccess ? WAL_OK : WAL_ERR_DEVICE;
}
