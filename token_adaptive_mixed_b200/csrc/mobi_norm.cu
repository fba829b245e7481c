// mobi_norm.cu — the step between two blocks of a model in one pass over the rows:
//   z = post(block) * post_weight + post_bias
//   r = x + scale * gate * z
//   n = norm(r) * weight + bias, also as e4m3 blocks of 128 (mobi_device.cuh, "8-bit blocks")
//
// Memory-bound: block and x are read once and r and n written once; a row
// lives in registers between (eight consecutive values per thread and chunk,
// NCH chunks), so both norms' statistics are exact two-pass sums in fp32 (mean
// first, then squares of the differences) at no extra traffic. Sixteen lanes
// hold the 128 values of an e4m3 block.
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
};

// Eight raw elements: `a` holds 16-bit types, `a` and `b` fp32.
struct Raw8 {
  uint4 a, b;
};

// Element `i` of a raw octet of `dtype` as fp32.
__device__ __forceinline__ void widen8(const Raw8& r, int dtype, float (&v)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  if (dtype == MOBI_F32) {
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

// Elements d .. d+7 of a row at `base` + off elements (stride 1), zeros from D on.
__device__ __forceinline__ Raw8 load8(const void* base, int dtype, int64_t off, int d, int D, int vec) {
  Raw8 r;
  r.a = r.b = make_uint4(0, 0, 0, 0);
  if (d >= D) return r;
  const int es = dtype == MOBI_F32 ? 4 : 2;
  const uint8_t* p = static_cast<const uint8_t*>(base) + (off + d) * es;
  if (vec && d + 8 <= D) {
    r.a = *reinterpret_cast<const uint4*>(p);
    if (es == 4) r.b = *reinterpret_cast<const uint4*>(p + 16);
    return r;
  }
  uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (d + i < D) {
      if (es == 4) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      else w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    }
  r.a = make_uint4(w[0], w[1], w[2], w[3]);
  r.b = make_uint4(w[4], w[5], w[6], w[7]);
  return r;
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

// v <- kind(v) * w + b over a row.
template <int NCH>
__device__ __forceinline__ void norm_row(float (&v)[NCH][8], int kind, float eps, const void* weight, const void* bias,
                                         const Params& p, int l, float (*red)[32], int slot) {
  const int D = (int)p.a.D, tpr = p.tpr;
  const float inv = 1.0f / (float)D;
  float mean = 0.0f, s = 0.0f;
  if (kind == MOBI_NORM_LAYER) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[c][i];  // zeros past D
    mean = row_sum(s, tpr, red, slot) * inv;
    s = 0.0f;
  }
  float rstd = 1.0f;
  if (kind != MOBI_NORM_NONE) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = (c * tpr + l) * 8 + i < D ? v[c][i] - mean : 0.0f;
        s = fmaf(e, e, s);
      }
    rstd = 1.0f / sqrtf(row_sum(s, tpr, red, slot + 1) * inv + eps);
  }
  const float one = p.a.unit_offset ? 1.0f : 0.0f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int d = (c * tpr + l) * 8;
    float w[8], b[8];
    if (weight) widen8(load8(weight, p.a.weight_dtype, 0, d, D, p.vw), p.a.weight_dtype, w);
    if (bias) widen8(load8(bias, p.a.weight_dtype, 0, d, D, p.vw), p.a.weight_dtype, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float e = (v[c][i] - mean) * rstd;
      if (weight) e *= w[i] + one;
      if (bias) e += b[i];
      v[c][i] = e;
    }
  }
}

template <int NCH>
__global__ void __launch_bounds__(NCH == 1 ? 1024 : 512) norm_kernel(const __grid_constant__ Params p) {
  __shared__ float red[4][32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const mobi_norm_args& a = p.a;
  const int tpr = p.tpr, D = (int)a.D;
  const int64_t t = tpr == 32 ? (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const int l = tpr == 32 ? (threadIdx.x & 31) : threadIdx.x;
  if (t >= a.T) return;  // whole warps, and only where a row is one warp

  // Every load of the row is issued before the first sum waits for one.
  Raw8 rx[NCH], rb[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int d = (c * tpr + l) * 8;
    if (a.block) rb[c] = load8(a.block, a.block_dtype, t * a.ldb, d, D, p.vb);
    rx[c] = load8(a.x, a.x_dtype, t * a.ldx, d, D, p.vx);
  }
  float r[NCH][8];
  if (a.block) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) widen8(rb[c], a.block_dtype, r[c]);
    if (a.post != MOBI_NORM_NONE || a.post_weight || a.post_bias)
      norm_row<NCH>(r, a.post, a.post_eps, a.post_weight, a.post_bias, p, l, red, 0);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int d = (c * tpr + l) * 8;
      float x[8], g[8];
      widen8(rx[c], a.x_dtype, x);
      if (a.gate) {
        if (a.gate_sd == 1) {
          widen8(load8(a.gate, a.gate_dtype, t * a.gate_st, d, D, p.vg), a.gate_dtype, g);
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
#pragma unroll
      for (int i = 0; i < 8; ++i) r[c][i] = d + i < D ? fmaf(a.scale, r[c][i], x[i]) : 0.0f;
      if (a.r_out) store8(a.r_out, a.x_dtype, t * a.ldr, d, D, p.vr, r[c]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < NCH; ++c) widen8(rx[c], a.x_dtype, r[c]);
  }

  norm_row<NCH>(r, a.kind, a.eps, a.weight, a.bias, p, l, red, 2);
  if (a.out_dtype != MOBI_E4M3) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) store8(a.n_out, a.out_dtype, t * a.ldn, (c * tpr + l) * 8, D, p.vn, r[c]);
    return;
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
    const float s = block_scale(m), inv = 1.0f / s;
    if ((l & 15) == 0) a.n_scale[(int64_t)(d / 128) * a.T + t] = s;
    const uint32_t lo = e4m3x2(r[c][0] * inv, r[c][1] * inv) | (e4m3x2(r[c][2] * inv, r[c][3] * inv) << 16);
    const uint32_t hi = e4m3x2(r[c][4] * inv, r[c][5] * inv) | (e4m3x2(r[c][6] * inv, r[c][7] * inv) << 16);
    if (p.vn && d + 8 <= D) {
      *reinterpret_cast<uint2*>(q + d) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (d + i < D) q[d + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
  }
}

constexpr int kMaxD = 16384;  // 512 threads x 4 chunks x 8 values

static cudaError_t launch(Params& p, cudaStream_t stream) {
  const int64_t T = p.a.T, oct = (p.a.D + 7) / 8;
  // Few rows: one octet per thread (up to 1024 threads), so that a row's latency
  // is one load deep. Many rows: two, which keeps more bytes in flight per
  // thread and needs half the warps at the row's barriers; four past D = 8192.
  const int nch = oct > 1024 ? 4 : (T >= 2 * num_sms() && oct > 32 ? 2 : 1);
  const int64_t tpr = ((oct + nch - 1) / nch + 31) / 32 * 32;
  p.tpr = (int)tpr;
  const int threads = tpr == 32 ? 256 : (int)tpr;
  const int64_t grid = tpr == 32 ? (T + 7) / 8 : T;
  const dim3 g((unsigned)grid);
  if (nch == 1) return launch_dependent(norm_kernel<1>, g, threads, 0, 1, stream, p);
  if (nch == 2) return launch_dependent(norm_kernel<2>, g, threads, 0, 1, stream, p);
  return launch_dependent(norm_kernel<4>, g, threads, 0, 1, stream, p);
}

bool plain_type(int t) { return t >= MOBI_F32 && t <= MOBI_F16; }
int64_t bytes(int t) { return t == MOBI_F32 ? 4 : (t == MOBI_E4M3 ? 1 : 2); }
bool at(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)a == 0; }
int wide(const void* p, int64_t ld, int t) { return at(p, 16) && ld * bytes(t) % 16 == 0; }

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
