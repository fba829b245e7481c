// mobi_norm.cu — the step between two blocks of a model in one pass over the rows:
//   z = post(block) * post_weight + post_bias
//   r = x + scale * gate * z
//   n = norm(r) * weight + bias, also as e4m3 blocks of 128 (mobi_device.cuh, "8-bit blocks")
//
// Memory-bound: block and x are read once and r and n written once. A row lives
// in registers between (eight consecutive values per thread and octet), so both
// norms' statistics are exact two-pass sums in fp32 (mean first, then squares of
// the differences) at no extra traffic. Sixteen lanes hold the 128 values of an
// e4m3 block. A CTA walks over rows: the next row's loads are in flight while
// this one is summed; the weights stay in L1 for all of them (held in registers
// they cost the second CTA of an SM).
#include <cmath>
#include <cstdint>

#include "mobi_device.cuh"
#include "mobi_host.h"

namespace mobi {

namespace nm {

struct Params {
  mobi_norm_args a;
  int vx, vb, vg, vw, vr, vn;  // rows of x, block, gate, weights, r, n may be accessed 16 bytes at a time
  int tpr;                     // threads of a row
  uint32_t lx, lb, lr, ln;     // pitches of x, block, r and n in bytes (aligned rows)
};

// Eight raw elements of ES bytes.
template <int ES>
struct Raw8 {
  uint32_t w[2 * ES];
};

// An octet as fp32; `dtype` tells the two 16-bit types apart.
template <int ES>
__device__ __forceinline__ void widen8(const Raw8<ES>& r, int dtype, float (&v)[8]) {
  const uint32_t* w = r.w;
  if constexpr (ES == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else if (dtype == MOBI_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = elem_f32<__half>((uint16_t)w[i]);
      v[2 * i + 1] = elem_f32<__half>((uint16_t)(w[i] >> 16));
    }
  }
}

// Elements d .. d+7 of a row at `base` + off elements, zeros from D on.
template <int ES>
__device__ __forceinline__ Raw8<ES> load8(const void* base, int64_t off, int d, int D, int vec) {
  Raw8<ES> r;
#pragma unroll
  for (int i = 0; i < 2 * ES; ++i) r.w[i] = 0;
  if (d >= D) return r;
  const uint8_t* p = static_cast<const uint8_t*>(base) + (off + d) * ES;
  if (vec && d + 8 <= D) {
#pragma unroll
    for (int i = 0; i < ES / 2; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
    return r;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (d + i < D) {
      if constexpr (ES == 4) r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      else r.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    }
  return r;
}

// The same of a type known at run time only, as fp32.
__device__ __forceinline__ void load8_f32(const void* base, int dtype, int64_t off, int d, int D, int vec,
                                          float (&v)[8]) {
  if (dtype == MOBI_F32) widen8<4>(load8<4>(base, off, d, D, vec), dtype, v);
  else widen8<2>(load8<2>(base, off, d, D, vec), dtype, v);
}

__device__ __forceinline__ void store8(void* base, int dtype, int64_t off, int d, int D, int vec, const float (&v)[8]) {
  if (d >= D) return;
  uint32_t w[8];
  int es = 2;
  if (dtype == MOBI_F32) {
    es = 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
  } else if (dtype == MOBI_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  uint8_t* p = static_cast<uint8_t*>(base) + (off + d) * es;
  if (vec && d + 8 <= D) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    if (es == 4) *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (d + i < D) {
      if (es == 4) reinterpret_cast<uint32_t*>(p)[i] = w[i];
      else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
}

// Sum over the threads of a row; `slot` is this reduction's own shared row, so
// one barrier suffices. tpr = 32: one warp, no barrier.
__device__ __forceinline__ float row_sum(float v, int tpr, float (*red)[32], int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr == 32) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[slot][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < tpr / 32 ? red[slot][lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(m): the approximate reciprocal root with one Newton step (fp32 to the
// last place or two). Zero and infinity keep the first estimate, infinity and
// 0, which the step would turn into a NaN.
__device__ __forceinline__ float root(float m) {
  const float y = rsqrtf(m);
  return m == 0.0f || y == 0.0f ? y : y * fmaf(-0.5f * m * y, y, 1.5f);
}

// v <- kind(v) * w + b over a row (zeros past D stay out of the sums).
template <int NCH>
__device__ __forceinline__ void norm_row(float (&v)[NCH][8], int kind, float eps, const void* weight, const void* bias,
                                         const Params& p, int l, float inv, float (*red)[32], int slot) {
  const int D = (int)p.a.D, tpr = p.tpr;
  float mean = 0.0f, s = 0.0f;
  if (kind == MOBI_NORM_LAYER) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[c][i];
    mean = row_sum(s, tpr, red, slot) * inv;
    s = 0.0f;
  }
  float rstd = 1.0f;
  if (kind != MOBI_NORM_NONE) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int d = (c * tpr + l) * 8;
      if (d + 8 <= D) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(v[c][i] - mean, v[c][i] - mean, s);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (d + i < D) s = fmaf(v[c][i] - mean, v[c][i] - mean, s);
      }
    }
    rstd = root(row_sum(s, tpr, red, slot + 1) * inv + eps);
  }
  const float one = p.a.unit_offset ? 1.0f : 0.0f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int d = (c * tpr + l) * 8;
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = (v[c][i] - mean) * rstd;
    if (weight) {
      load8_f32(weight, p.a.weight_dtype, 0, d, D, p.vw, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= e[i] + one;
    }
    if (bias) {
      load8_f32(bias, p.a.weight_dtype, 0, d, D, p.vw, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] += e[i];
    }
  }
}

// XS, BS: bytes of x's and the block's elements (0: no block).
// MIN: CTAs that an SM is to hold.
template <int XS, int BS, int NCH, int MAXT, int MIN>
__global__ void __launch_bounds__(MAXT, MIN) norm_kernel(const __grid_constant__ Params p) {
  __shared__ float red[2][4][32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const mobi_norm_args& a = p.a;
  const int tpr = p.tpr, D = (int)a.D;
  const int rows = tpr == 32 ? blockDim.x / 32 : 1;  // rows of a CTA at a time
  const int64_t stride = (int64_t)gridDim.x * rows;
  int64_t t = (int64_t)blockIdx.x * rows + (tpr == 32 ? threadIdx.x >> 5 : 0);
  const int l = tpr == 32 ? (threadIdx.x & 31) : threadIdx.x;
  if (t >= a.T) return;  // whole warps, and only where a row is one warp
  const float inv = 1.0f / (float)D;

  constexpr int BE = BS ? BS : 2;
  Raw8<XS> rx[NCH];
  Raw8<BE> rb[NCH];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int d = (c * tpr + l) * 8;
      if constexpr (BS != 0) rb[c] = load8<BE>(a.block, row * a.ldb, d, D, p.vb);
      rx[c] = load8<XS>(a.x, row * a.ldx, d, D, p.vx);
    }
  };
  fetch(t);

  for (int par = 0; t < a.T; t += stride, par ^= 1) {  // sums of consecutive rows use their own shared rows
    float r[NCH][8];
    if constexpr (BS != 0) {
      Raw8<XS> cx[NCH];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        widen8<BE>(rb[c], a.block_dtype, r[c]);
        cx[c] = rx[c];
      }
      if (t + stride < a.T) fetch(t + stride);
      if (a.post != MOBI_NORM_NONE || a.post_weight || a.post_bias)
        norm_row<NCH>(r, a.post, a.post_eps, a.post_weight, a.post_bias, p, l, inv, red[par], 0);
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int d = (c * tpr + l) * 8;
        if (a.gate) {
          float g[8];
          if (a.gate_sd == 1) {
            load8_f32(a.gate, a.gate_dtype, t * a.gate_st, d, D, p.vg, g);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int64_t at = t * a.gate_st + (int64_t)(d + i < D ? d + i : 0) * a.gate_sd;
              g[i] = a.gate_dtype == MOBI_F32    ? static_cast<const float*>(a.gate)[at]
                     : a.gate_dtype == MOBI_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(a.gate)[at])
                                                 : to_f32(static_cast<const __half*>(a.gate)[at]);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) r[c][i] *= g[i];
        }
        float x[8];
        widen8<XS>(cx[c], a.x_dtype, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[c][i] = fmaf(a.scale, r[c][i], x[i]);
        if (d + 8 > D) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (d + i >= D) r[c][i] = 0.0f;
        }
        if (a.r_out) store8(a.r_out, a.x_dtype, t * a.ldr, d, D, p.vr, r[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < NCH; ++c) widen8<XS>(rx[c], a.x_dtype, r[c]);
      if (t + stride < a.T) fetch(t + stride);
    }

    norm_row<NCH>(r, a.kind, a.eps, a.weight, a.bias, p, l, inv, red[par], 2);
    if (a.out_dtype != MOBI_E4M3) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) store8(a.n_out, a.out_dtype, t * a.ldn, (c * tpr + l) * 8, D, p.vn, r[c]);
      continue;
    }
    uint8_t* q = static_cast<uint8_t*>(a.n_out) + t * a.ldn;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int d = (c * tpr + l) * 8;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (d + i < D) m = max(m, abs_bits(r[c][i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (d >= D) continue;
      const float s = block_scale(m), f = 1.0f / s;
      if ((l & 15) == 0) a.n_scale[(int64_t)(d / 128) * a.T + t] = s;
      const uint32_t lo = e4m3x2(r[c][0] * f, r[c][1] * f) | (e4m3x2(r[c][2] * f, r[c][3] * f) << 16);
      const uint32_t hi = e4m3x2(r[c][4] * f, r[c][5] * f) | (e4m3x2(r[c][6] * f, r[c][7] * f) << 16);
      if (p.vn && d + 8 <= D) {
        *reinterpret_cast<uint2*>(q + d) = make_uint2(lo, hi);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (d + i < D) q[d + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
      }
    }
  }
}

constexpr int kMaxD = 16384;  // 512 threads x 4 octets

// ---- aligned rows ------------------------------------------------------------------
//
// The same steps where every row is 16-byte aligned and D is a multiple of 8,
// with the types of x and the block known to the compiler and values in pairs.
// Both kernels are bound by issuing (and the barriers between) rather than by memory, so
// options are tested once a row, not once an octet, and addresses are 32-bit products
// (T = 8192, D = 4096, x, gate and block bf16, norms on both sides, e4m3 out: this one 55 to 57 us, of
// which post costs 12 and the gate 4, 39 us at 6.0 TB/s without both; weights and gate fp16 or fp32: 69 and 71.
// The general kernel takes 117 us there where x alone starts at an odd element, and 190 to 350 us at
// D = 4095, 4097 and 4100, where every operand's rows are read element by element).

struct Oct {
  float2 v[4];
};

// Octet of type DT (a mobi_dtype) at p.
template <int DT>
struct RawOct {
  uint4 w[DT == MOBI_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p) {
    w[0] = *static_cast<const uint4*>(p);
    if constexpr (DT == MOBI_F32) w[1] = static_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void zero() {
    w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (DT == MOBI_F32) w[1] = w[0];
  }
  __device__ __forceinline__ Oct widen() const {
    Oct o;
    if constexpr (DT == MOBI_F32) {
      o.v[0] = make_float2(__uint_as_float(w[0].x), __uint_as_float(w[0].y));
      o.v[1] = make_float2(__uint_as_float(w[0].z), __uint_as_float(w[0].w));
      o.v[2] = make_float2(__uint_as_float(w[1].x), __uint_as_float(w[1].y));
      o.v[3] = make_float2(__uint_as_float(w[1].z), __uint_as_float(w[1].w));
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DT == MOBI_BF16) o.v[i] = make_float2(bf16lo(u[i]), bf16hi(u[i]));
        else o.v[i] = make_float2(elem_f32<__half>((uint16_t)u[i]), elem_f32<__half>((uint16_t)(u[i] >> 16)));
      }
    }
    return o;
  }
};

// Weights, biases and gates have a type known at run time only. bf16 is inline;
// the others are calls, since inlined their conversions were run beside bf16's.
__device__ __noinline__ Oct load_oct_other(const void* base, int dtype, int64_t at) {
  if (dtype == MOBI_F32) {
    RawOct<MOBI_F32> r;
    r.load(static_cast<const float*>(base) + at);
    return r.widen();
  }
  RawOct<MOBI_F16> r;
  r.load(static_cast<const __half*>(base) + at);
  return r.widen();
}
__device__ __forceinline__ Oct load_oct(const void* base, int dtype, int64_t at) {
  if (dtype != MOBI_BF16) return load_oct_other(base, dtype, at);
  RawOct<MOBI_BF16> r;
  r.load(static_cast<const __nv_bfloat16*>(base) + at);
  return r.widen();
}

__device__ __forceinline__ void store_oct(void* to, int dtype, const Oct& o) {
  if (dtype == MOBI_F32) {
    float4* q = static_cast<float4*>(to);
    q[0] = make_float4(o.v[0].x, o.v[0].y, o.v[1].x, o.v[1].y);
    q[1] = make_float4(o.v[2].x, o.v[2].y, o.v[3].x, o.v[3].y);
    return;
  }
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dtype == MOBI_BF16) {
      const __nv_bfloat162 h = __float22bfloat162_rn(o.v[i]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __float22half2_rn(o.v[i]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *static_cast<uint4*>(to) = make_uint4(u[0], u[1], u[2], u[3]);
}

// max(a, |x|, |y|) for a >= 0, NaN if any is.
__device__ __forceinline__ float max3_abs(float a, float x, float y) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(x), "f"(y));
  return r;
}

// Sum over the threads of a row (at most 16 warps); `slot` as in row_sum, its unused entries are zero.
__device__ __forceinline__ float row_sum16(float v, int tpr, float4* slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr == 32) return v;
  if ((threadIdx.x & 31) == 0) reinterpret_cast<float*>(slot)[threadIdx.x >> 5] = v;
  __syncthreads();
  float4 a = slot[0], b = slot[1];
  v = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
  if (tpr > 256) {
    a = slot[2];
    b = slot[3];
    v += ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
  }
  return v;
}

template <int NCH>
__device__ __forceinline__ void norm_octs(Oct (&r)[NCH], int kind, float eps, const void* weight, const void* bias,
                                          const Params& p, uint32_t l, float inv, float4 (*red)[4]) {
  const uint32_t D = (uint32_t)p.a.D, tpr = p.tpr;
  if (kind == MOBI_NORM_LAYER) {
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) s = __fadd2_rn(s, r[c].v[i]);
    const float mean = row_sum16(s.x + s.y, tpr, red[0]) * inv;
    const float2 neg = make_float2(-mean, -mean);
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      if ((c * tpr + l) * 8 < D) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[c].v[i] = __fadd2_rn(r[c].v[i], neg);
      }
  }
  float2 rstd = make_float2(1.0f, 1.0f);
  if (kind != MOBI_NORM_NONE) {
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) s = __ffma2_rn(r[c].v[i], r[c].v[i], s);
    rstd.x = rstd.y = root(row_sum16(s.x + s.y, tpr, red[1]) * inv + eps);
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) r[c].v[i] = __fmul2_rn(r[c].v[i], rstd);
  if (weight) {
    auto times = [&](Oct& v, Oct w) {
      if (p.a.unit_offset) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w.v[i] = __fadd2_rn(w.v[i], make_float2(1.0f, 1.0f));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v.v[i] = __fmul2_rn(v.v[i], w.v[i]);
    };
    if (p.a.weight_dtype == MOBI_BF16) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const uint32_t d = (c * tpr + l) * 8;
        if (d < D) times(r[c], load_oct(weight, MOBI_BF16, d));
      }
    } else {
#pragma unroll
      for (int c = 0; c < NCH; ++c)
        if ((c * tpr + l) * 8 < D) times(r[c], load_oct_other(weight, p.a.weight_dtype, (c * tpr + l) * 8));
    }
  }
  if (bias) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const uint32_t d = (c * tpr + l) * 8;
      if (d >= D) break;
      const Oct b = load_oct(bias, p.a.weight_dtype, d);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[c].v[i] = __fadd2_rn(r[c].v[i], b.v[i]);
    }
  }
}

// XT, BT: types of x and of the block (-1: no block).
template <int XT, int BT, int NCH, int MAXT, int MIN>
__global__ void __launch_bounds__(MAXT, MIN) norm_aligned_kernel(const __grid_constant__ Params p) {
  __shared__ float4 red[2][4][4];
  if (threadIdx.x < 32) red[threadIdx.x >> 4][(threadIdx.x >> 2) & 3][threadIdx.x & 3] = make_float4(0, 0, 0, 0);
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  const mobi_norm_args& a = p.a;
  const uint32_t tpr = p.tpr, D = (uint32_t)a.D;
  const uint32_t rows = tpr == 32 ? blockDim.x / 32 : 1;
  const uint32_t T = (uint32_t)a.T, stride = gridDim.x * rows;
  uint32_t t = blockIdx.x * rows + (tpr == 32 ? threadIdx.x >> 5 : 0);
  const uint32_t l = tpr == 32 ? (threadIdx.x & 31) : threadIdx.x;
  if (t >= T) return;  // whole warps, and only where a row is one warp
  const float inv = 1.0f / (float)D;
  const float2 scale = make_float2(a.scale, a.scale);

  // Row numbers and pitches (bytes) are 32-bit: one multiplication for an address. 64-bit ones took 3 us of
  // 60 at T = 8192, D = 4096; pointers moved on from row to row spilled (65 us).
  constexpr uint32_t XB = XT == MOBI_F32 ? 4 : 2, BB = BT == MOBI_F32 ? 4 : 2;
  const uint32_t nb = a.out_dtype == MOBI_E4M3 ? 1 : (a.out_dtype == MOBI_F32 ? 4 : 2);
  const auto at = [](const void* base, uint32_t row, uint32_t pitch, uint32_t off) {
    return const_cast<uint8_t*>(static_cast<const uint8_t*>(base)) + (uint64_t)row * pitch + off;
  };

  RawOct<XT> rx[NCH];
  RawOct<BT < 0 ? MOBI_BF16 : BT> rb[NCH];
  auto fetch = [&](uint32_t row) {
    const uint8_t* px = at(a.x, row, p.lx, 8 * XB * l);
    const uint8_t* pb = BT < 0 ? nullptr : at(a.block, row, p.lb, 8 * BB * l);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      if ((c * tpr + l) * 8 < D) {
        if constexpr (BT >= 0) rb[c].load(pb + c * tpr * 8 * BB);
        rx[c].load(px + c * tpr * 8 * XB);
      } else {
        if constexpr (BT >= 0) rb[c].zero();
        rx[c].zero();
      }
    }
  };
  fetch(t);
  for (int par = 0; t < T; t += stride, par ^= 1) {
    Oct r[NCH];
    if constexpr (BT >= 0) {
      RawOct<XT> cx[NCH];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        r[c] = rb[c].widen();
        cx[c] = rx[c];
      }
      if (t + stride < T) fetch(t + stride);
      if (a.post != MOBI_NORM_NONE || a.post_weight || a.post_bias)
        norm_octs<NCH>(r, a.post, a.post_eps, a.post_weight, a.post_bias, p, l, inv, red[par]);
      if (a.gate) {
        auto times = [](Oct& v, const Oct& g) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v.v[i] = __fmul2_rn(v.v[i], g.v[i]);
        };
        const int64_t first = t * a.gate_st;
        if (a.gate_sd == 0) {  // one value for the row
          const float f = a.gate_dtype == MOBI_F32    ? static_cast<const float*>(a.gate)[first]
                          : a.gate_dtype == MOBI_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(a.gate)[first])
                                                      : to_f32(static_cast<const __half*>(a.gate)[first]);
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int c = 0; c < NCH; ++c)
            if ((c * tpr + l) * 8 < D) times(r[c], Oct{{f2, f2, f2, f2}});
        } else if (a.gate_dtype == MOBI_BF16) {
#pragma unroll
          for (int c = 0; c < NCH; ++c) {
            const uint32_t d = (c * tpr + l) * 8;
            if (d < D) times(r[c], load_oct(a.gate, MOBI_BF16, first + d));
          }
        } else {
#pragma unroll
          for (int c = 0; c < NCH; ++c) {
            const uint32_t d = (c * tpr + l) * 8;
            if (d < D) times(r[c], load_oct_other(a.gate, a.gate_dtype, first + d));
          }
        }
      }
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const uint32_t d = (c * tpr + l) * 8;
        if (d >= D) break;
        const Oct x = cx[c].widen();
#pragma unroll
        for (int i = 0; i < 4; ++i) r[c].v[i] = __ffma2_rn(scale, r[c].v[i], x.v[i]);
        if (a.r_out) store_oct(at(a.r_out, t, p.lr, d * XB), XT, r[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < NCH; ++c) r[c] = rx[c].widen();
      if (t + stride < T) fetch(t + stride);
    }

    norm_octs<NCH>(r, a.kind, a.eps, a.weight, a.bias, p, l, inv, red[par] + 2);
    if (a.out_dtype != MOBI_E4M3) {
#pragma unroll
      for (int c = 0; c < NCH; ++c)
        if ((c * tpr + l) * 8 < D) store_oct(at(a.n_out, t, p.ln, (c * tpr + l) * 8 * nb), a.out_dtype, r[c]);
    } else {
      // All octets' maxima first: one octet's exchanges hide the other's latency.
      float m[NCH];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        m[c] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m[c] = max3_abs(m[c], r[c].v[i].x, r[c].v[i].y);
        if ((c * tpr + l) * 8 >= D) m[c] = 0.0f;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int c = 0; c < NCH; ++c) m[c] = max_abs(m[c], __shfl_xor_sync(0xffffffffu, m[c], o));
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        if ((c * tpr + l) * 8 >= D) break;
        const float s = block_scale(__float_as_uint(m[c])), f = __frcp_rn(s);
        if ((l & 15) == 0) a.n_scale[(uint64_t)((c * tpr + l) >> 4) * T + t] = s;
        const float2 f2 = make_float2(f, f);
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = __fmul2_rn(r[c].v[i], f2);
          u[i] = e4m3x2(y.x, y.y);
        }
        *reinterpret_cast<uint2*>(at(a.n_out, t, p.ln, (c * tpr + l) * 8)) = make_uint2(u[0] | (u[1] << 16), u[2] | (u[3] << 16));
      }
    }
  }
}

// `few`: one octet per thread, so that a row's latency is one load deep; else
// two, since sums and scales cost a thread the same for sixteen values as for
// eight. Four past D = 8192. As many CTAs as run at once.
template <typename Go>
static cudaError_t plan_rows(Params& p, bool few, Go go) {
  const int64_t T = p.a.T, oct = (p.a.D + 7) / 8;
  const int nch = oct > 1024 ? 4 : (oct > 512 || (!few && oct > 32) ? 2 : 1);
  p.tpr = (int)((oct + 32 * nch - 1) / (32 * nch)) * 32;
  const int threads = p.tpr == 32 ? 128 : p.tpr, rows = p.tpr == 32 ? 4 : 1;
  return go(nch, threads, (T + rows - 1) / rows);
}

template <int XT, int BT>
static cudaError_t launch_aligned(Params& p, cudaStream_t stream) {
  return plan_rows(p, p.a.T < 4 * (int64_t)num_sms(), [&](int nch, int threads, int64_t need) {
    auto run = [&](auto kernel, int maxt, int min) {
      const int64_t most = (int64_t)num_sms() * (min * maxt / threads);
      return launch_dependent(kernel, dim3((unsigned)(need < most ? need : most)), threads, 0, 1, stream, p);
    };
    if (nch == 1) return run(norm_aligned_kernel<XT, BT, 1, 512, 2>, 512, 2);
    // Three CTAs to an SM leave 80 registers, which fp32 rows with a block spill from: two (T = 8192, D = 4096,
    // x and block fp32: 107 us with three, 91 with two; x bf16, block fp32: 68 with three, 79 with two).
    constexpr int kMin = XT == MOBI_F32 && BT >= 0 ? 2 : 3;
    if (nch == 2 && threads <= 256) return run(norm_aligned_kernel<XT, BT, 2, 256, kMin>, 256, kMin);
    if (nch == 2) return run(norm_aligned_kernel<XT, BT, 2, 512, 1>, 512, 1);
    return run(norm_aligned_kernel<XT, BT, 4, 512, 1>, 512, 1);
  });
}

template <int XT>
static cudaError_t launch_aligned_x(Params& p, cudaStream_t stream) {
  if (!p.a.block) return launch_aligned<XT, -1>(p, stream);
  if (p.a.block_dtype == MOBI_F32) return launch_aligned<XT, MOBI_F32>(p, stream);
  if (p.a.block_dtype == MOBI_BF16) return launch_aligned<XT, MOBI_BF16>(p, stream);
  return launch_aligned<XT, MOBI_F16>(p, stream);
}

template <int XS, int BS>
static cudaError_t launch_types(Params& p, cudaStream_t stream) {
  return plan_rows(p, true, [&](int nch, int threads, int64_t need) {
    auto run = [&](auto kernel, int min) {
      const int64_t most = (int64_t)num_sms() * (min * 512 / threads);
      return launch_dependent(kernel, dim3((unsigned)(need < most ? need : most)), threads, 0, 1, stream, p);
    };
    if (nch == 1) return run(norm_kernel<XS, BS, 1, 512, 2>, 2);
    if (nch == 2) return run(norm_kernel<XS, BS, 2, 512, 1>, 1);
    return run(norm_kernel<XS, BS, 4, 512, 1>, 1);
  });
}

bool plain_type(int t) { return t >= MOBI_F32 && t <= MOBI_F16; }
int64_t bytes(int t) { return t == MOBI_F32 ? 4 : (t == MOBI_E4M3 ? 1 : 2); }
bool at(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)a == 0; }
int wide(const void* p, int64_t ld, int t) { return at(p, 16) && ld * bytes(t) % 16 == 0; }

static cudaError_t launch(Params& p, cudaStream_t stream) {
  const mobi_norm_args& a = p.a;
  const int64_t lx = a.ldx * bytes(a.x_dtype), lb = a.block ? a.ldb * bytes(a.block_dtype) : 0,
                lr = a.r_out ? a.ldr * bytes(a.x_dtype) : 0, ln = a.ldn * bytes(a.out_dtype);
  p.lx = (uint32_t)lx;
  p.lb = (uint32_t)lb;
  p.lr = (uint32_t)lr;
  p.ln = (uint32_t)ln;
  const bool short_rows = ((lx | lb | lr | ln) >> 32) == 0;
  if (short_rows && a.D % 8 == 0 && p.vx && p.vn && p.vw && (!a.block || p.vb) && (!a.r_out || p.vr) &&
      (!a.gate || a.gate_sd == 0 || (a.gate_sd == 1 && p.vg))) {
    if (a.x_dtype == MOBI_F32) return launch_aligned_x<MOBI_F32>(p, stream);
    if (a.x_dtype == MOBI_BF16) return launch_aligned_x<MOBI_BF16>(p, stream);
    return launch_aligned_x<MOBI_F16>(p, stream);
  }
  const bool wide = p.a.x_dtype == MOBI_F32;
  if (!p.a.block) return wide ? launch_types<4, 0>(p, stream) : launch_types<2, 0>(p, stream);
  if (p.a.block_dtype == MOBI_F32) return wide ? launch_types<4, 4>(p, stream) : launch_types<2, 4>(p, stream);
  return wide ? launch_types<4, 2>(p, stream) : launch_types<2, 2>(p, stream);
}

}  // namespace nm

}  // namespace mobi

using namespace mobi;

extern "C" mobi_status mobi_norm(const mobi_norm_args* args, void* stream) {
  clear_message();
  if (!args) return MOBI_ERR_INVALID_ARG;
  nm::Params p = {};
  p.a = *args;
  mobi_norm_args& a = p.a;
  if (!a.block) {  // a plain norm of x
    a.gate = a.post_weight = a.post_bias = nullptr;
    a.r_out = nullptr;
    a.post = MOBI_NORM_NONE;
  }
  if (a.T < 0 || a.D < 1 || !nm::plain_type(a.x_dtype) || a.out_dtype < MOBI_F32 || a.out_dtype > MOBI_E4M3 ||
      a.post < MOBI_NORM_NONE || a.post > MOBI_NORM_LAYER || a.kind < MOBI_NORM_NONE || a.kind > MOBI_NORM_LAYER)
    return MOBI_ERR_INVALID_ARG;
  if ((a.block && !nm::plain_type(a.block_dtype)) || (a.gate && !nm::plain_type(a.gate_dtype)) ||
      ((a.weight || a.bias || a.post_weight || a.post_bias) && !nm::plain_type(a.weight_dtype)))
    return MOBI_ERR_INVALID_ARG;
  if (!(a.eps >= 0.0f) || !std::isfinite(a.eps)) return MOBI_ERR_INVALID_ARG;
  if (a.block && (!(a.post_eps >= 0.0f) || !std::isfinite(a.post_eps) || !std::isfinite(a.scale)))
    return MOBI_ERR_INVALID_ARG;
  if (a.D > nm::kMaxD || a.T > (int64_t(1) << 28)) return MOBI_ERR_UNSUPPORTED_SHAPE;
  if (a.T == 0) return MOBI_OK;
  if (!a.x || !a.n_out || (a.out_dtype == MOBI_E4M3 && !a.n_scale)) return MOBI_ERR_INVALID_ARG;
  if (a.ldx < a.D || a.ldn < a.D || (a.block && a.ldb < a.D) || (a.r_out && a.ldr < a.D) ||
      (a.r_out == a.x && a.r_out && a.ldr != a.ldx))
    return MOBI_ERR_INVALID_ARG;
  const int64_t wb = nm::bytes(a.weight_dtype);
  if (!nm::at(a.x, nm::bytes(a.x_dtype)) || !nm::at(a.n_out, nm::bytes(a.out_dtype)) || !nm::at(a.n_scale, 4) ||
      (a.block && !nm::at(a.block, nm::bytes(a.block_dtype))) || (a.r_out && !nm::at(a.r_out, nm::bytes(a.x_dtype))) ||
      (a.gate && !nm::at(a.gate, nm::bytes(a.gate_dtype))) || (a.weight && !nm::at(a.weight, wb)) ||
      (a.bias && !nm::at(a.bias, wb)) || (a.post_weight && !nm::at(a.post_weight, wb)) ||
      (a.post_bias && !nm::at(a.post_bias, wb)))
    return MOBI_ERR_MISALIGNED;
  p.vx = nm::wide(a.x, a.ldx, a.x_dtype);
  p.vb = nm::wide(a.block, a.ldb, a.block_dtype);
  p.vg = nm::wide(a.gate, a.gate_st, a.gate_dtype);
  p.vw = nm::at(a.weight, 16) && nm::at(a.bias, 16) && nm::at(a.post_weight, 16) && nm::at(a.post_bias, 16);
  p.vr = nm::wide(a.r_out, a.ldr, a.x_dtype);
  p.vn = a.out_dtype == MOBI_E4M3 ? nm::at(a.n_out, 8) && a.ldn % 8 == 0 : nm::wide(a.n_out, a.ldn, a.out_dtype);
  return status_of(note_error("norm launch", nm::launch(p, static_cast<cudaStream_t>(stream))));
}
