// mobi_quant.cu — blocks of 128 values along K as e4m3 with one fp32 scale each
// (activations: 1 x 128, weights: 128 x 128); the formulas are in mobi_device.cuh
// ("8-bit blocks").
//
// Memory-bound: each value is read once, held in registers while the block's
// maximum is reduced, and written once. Sixteen lanes hold a row's 128 values,
// eight each, so a 16-bit block is sixteen 16-byte loads. Rows that are not
// 16-byte aligned take the same kernels with element accesses (VEC = false).
#include <cstdint>

#include "mobi_device.cuh"
#include "mobi_host.h"

namespace mobi {

namespace qz {

// Eight values of a row starting at column k (zeros from K on), as stored.
template <typename E>
struct Oct {
  uint32_t w[2 * sizeof(E)];

  // The largest |x| as an fp32 bit pattern. 16-bit patterns of |x| order as integers too, so pairs are reduced as stored.
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t a = 0;
    if constexpr (sizeof(E) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) a = max(a, w[i] & 0x7fffffffu);
      return a;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) a = __vmaxu2(a, w[i] & 0x7fff7fffu);
      return abs_bits(elem_f32<E>((uint16_t)max(a & 0xffffu, a >> 16)));
    }
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    if constexpr (sizeof(E) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = elem_f32<E>((uint16_t)w[i]);
        v[2 * i + 1] = elem_f32<E>((uint16_t)(w[i] >> 16));
      }
    }
  }
};

template <typename E, bool VEC>
__device__ __forceinline__ Oct<E> load8(const E* row, int64_t k, int64_t K) {
  Oct<E> o;
  if (VEC && k + 8 <= K) {
    const uint4* p = reinterpret_cast<const uint4*>(row + k);
#pragma unroll
    for (int i = 0; i < (int)sizeof(E) / 2; ++i) reinterpret_cast<uint4*>(o.w)[i] = p[i];
    return o;
  }
#pragma unroll
  for (int i = 0; i < 2 * (int)sizeof(E); ++i) o.w[i] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < K) {
      if constexpr (sizeof(E) == 4) o.w[i] = reinterpret_cast<const uint32_t*>(row)[k + i];
      else o.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[k + i] << (16 * (i & 1));
    }
  return o;
}

template <typename E, bool VEC>
__device__ __forceinline__ void store8(uint8_t* row, int64_t k, int64_t K, const Oct<E>& o, float r) {
  float v[8];
  o.widen(v);
  uint32_t lo = e4m3x2(v[0] * r, v[1] * r) | (e4m3x2(v[2] * r, v[3] * r) << 16);
  uint32_t hi = e4m3x2(v[4] * r, v[5] * r) | (e4m3x2(v[6] * r, v[7] * r) << 16);
  if (VEC && k + 8 <= K) {
    *reinterpret_cast<uint2*>(row + k) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) row[k + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
  }
}

constexpr int kThreads = 256;
constexpr int kRowBlocks = 4;  // K blocks of a half-warp: their loads are all in flight at once

// 1 x 128: a CTA takes 16 tokens x kRowBlocks blocks, a half-warp one token's.
template <typename E, bool VEC>
__global__ void __launch_bounds__(kThreads) quant_row_kernel(const E* X, int64_t T, int64_t K, int64_t ldx,
                                                             uint8_t* Q, int64_t ldq,
                                                             float* scale) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t t = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4), kb0 = (int64_t)blockIdx.y * kRowBlocks;
  const int64_t nkb = (K + 127) / 128;
  const int l = threadIdx.x & 15;
  if (t >= T) return;  // whole half-warps
  const unsigned mask = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
  Oct<E> v[kRowBlocks];
#pragma unroll
  for (int b = 0; b < kRowBlocks; ++b) v[b] = load8<E, VEC>(X + t * ldx, (kb0 + b) * 128 + 8 * l, K);
#pragma unroll
  for (int b = 0; b < kRowBlocks; ++b) {
    if (kb0 + b >= nkb) break;
    uint32_t a = v[b].amax();
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(mask, a, o));
    const float s = block_scale(a);
    if (l == 0) scale[(kb0 + b) * T + t] = s;
    store8<E, VEC>(Q + t * ldq, (kb0 + b) * 128 + 8 * l, K, v[b], 1.0f / s);
  }
}

// 128 x 128: a CTA takes one block; thread -> rows (tid / 16) + 16 i, columns 8 (tid % 16) ..
template <typename E, bool VEC>
__global__ void __launch_bounds__(kThreads) quant_block_kernel(const E* X, int64_t T, int64_t K,
                                                               int64_t ldx, uint8_t* Q, int64_t ldq,
                                                               float* scale) {
  __shared__ uint32_t wmax[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t nkb = (K + 127) / 128, kb = blockIdx.x % nkb, rb = blockIdx.x / nkb;
  const int64_t k = kb * 128 + 8 * (threadIdx.x & 15), t0 = rb * 128 + (threadIdx.x >> 4);
  Oct<E> v[8];
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = load8<E, VEC>(X + (t0 + 16 * i) * ldx, k, t0 + 16 * i < T ? K : 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, v[i].amax());
  a = __reduce_max_sync(0xffffffffu, a);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) a = max(a, wmax[i]);
  const float s = block_scale(a), r = 1.0f / s;
  if (threadIdx.x == 0) scale[kb * ((T + 127) / 128) + rb] = s;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (t0 + 16 * i < T) store8<E, VEC>(Q + (t0 + 16 * i) * ldq, k, K, v[i], r);
}

template <typename E, bool VEC>
static cudaError_t launch(const void* X, int64_t T, int64_t K, int64_t ldx, int block_rows, void* Q, int64_t ldq,
                          float* scale, cudaStream_t stream) {
  const int64_t nkb = (K + 127) / 128;
  const E* x = static_cast<const E*>(X);
  uint8_t* q = static_cast<uint8_t*>(Q);
  if (block_rows == 1) {
    const dim3 grid((unsigned)((T + 15) / 16), (unsigned)((nkb + kRowBlocks - 1) / kRowBlocks));
    return launch_dependent(quant_row_kernel<E, VEC>, grid, kThreads, 0, 1, stream, x, T, K, ldx, q, ldq, scale);
  }
  const dim3 grid((unsigned)(nkb * ((T + 127) / 128)));
  return launch_dependent(quant_block_kernel<E, VEC>, grid, kThreads, 0, 1, stream, x, T, K, ldx, q, ldq, scale);
}

}  // namespace qz

}  // namespace mobi

using namespace mobi;

extern "C" mobi_status mobi_fp8_quant(const void* X, int dtype, int64_t T, int64_t K, int64_t ldx, int block_rows,
                                      void* Q, int64_t ldq, float* scale, void* stream) {
  clear_message();
  if (T < 0 || K < 0 || dtype < MOBI_F32 || dtype > MOBI_F16 || (block_rows != 1 && block_rows != 128))
    return MOBI_ERR_INVALID_ARG;
  constexpr int64_t kMaxT = int64_t(1) << 28;
  constexpr int64_t kMaxK = int64_t(1) << 23;  // grid.y of the row kernel, grid.x of the block kernel with T
  if (T > kMaxT || K > kMaxT || (block_rows == 1 && K > kMaxK)) return MOBI_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || K == 0) return MOBI_OK;
  if (block_rows == 128 && ((T + 127) / 128) * ((K + 127) / 128) > 0x7fffffff) return MOBI_ERR_UNSUPPORTED_SHAPE;
  if (!X || !Q || !scale || ldx < K || ldq < K) return MOBI_ERR_INVALID_ARG;
  const uintptr_t es = dtype == MOBI_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(X) % es != 0 || reinterpret_cast<uintptr_t>(scale) % 4 != 0)
    return MOBI_ERR_MISALIGNED;
  const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && (ldx * es) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(Q) % 8 == 0 && ldq % 8 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MOBI_F32)
    e = vec ? qz::launch<float, true>(X, T, K, ldx, block_rows, Q, ldq, scale, s)
            : qz::launch<float, false>(X, T, K, ldx, block_rows, Q, ldq, scale, s);
  else if (dtype == MOBI_BF16)
    e = vec ? qz::launch<__nv_bfloat16, true>(X, T, K, ldx, block_rows, Q, ldq, scale, s)
            : qz::launch<__nv_bfloat16, false>(X, T, K, ldx, block_rows, Q, ldq, scale, s);
  else
    e = vec ? qz::launch<__half, true>(X, T, K, ldx, block_rows, Q, ldq, scale, s)
            : qz::launch<__half, false>(X, T, K, ldx, block_rows, Q, ldq, scale, s);
  return status_of(note_error("quant launch", e));
}
