// mobi_fp8.cu — products of e4m3 operands with one fp32 scale for each block of
// 128 values along K (activations: 1 x 128, weights: 128 x 128), on tcgen05:
//
//   mobi_fp8_gemm    y[t,n] = sum_b xs[b,t] ws[b,n/128] sum_{k in b} x[t,k] w[n,k]
//   mobi_fp8_gated   h[t,n] = act(g[t,n]) u[t,n], g and u as above with their own weights,
//                    optionally requantised to e4m3 in blocks of 128 columns
//
// Products of e4m3 values are exact in fp32; one block's sum is accumulated by
// the tensor core in TMEM and promoted, acc = fma(xs ws, D, acc), in fp32
// registers before the next block's sum replaces it. Nothing is rounded to
// fewer bits before the output.
//
// Two kernels. "wide" puts tokens on the TMEM lanes: a persistent pair of CTAs
// (cta_group::2) per two SMs takes tiles of 256 tokens x 256 output columns (or
// 128 gate + 128 up columns), each CTA holding half of the tokens and half of
// the weight rows; the promotion's scale is one register per thread. Few tiles
// are made twice as many of 128 columns. "narrow" puts
// weight rows on the lanes (128 rows x 16..128 tokens), so that one token costs
// a 16-wide tile and not a 128-wide one, and splits K over a cluster whose CTAs
// read each other's sums through distributed shared memory and add them in rank
// order.
//
// All mbarrier waits are bounded; on a timeout the kernel records the error,
// drains its copies and MMAs in flight, frees TMEM and returns.
#include <cstdint>

#include "mobi_device.cuh"
#include "mobi_host.h"

namespace mobi {

namespace f8 {
constexpr int BK = 128;                     // one scale block along K = one 128-byte swizzled row
constexpr uint32_t kTileBytes = 128 * BK;   // 128 rows of one block
constexpr int kEpiWarps = 8;

enum Act { kSilu = 0, kGelu = 1, kGeluTanh = 2, kRelu = 3 };

// Phi(-a), the normal distribution's left tail, for a >= 0: e^(-a^2 / 2) r Q(t) with r = 1 / (a + 3.75) and
// t = 1 - 7.5 r in [-1, 1). Q is the polynomial of degree 8 with the least largest relative error (1.5e-8 for
// a <= 14.5, where the tail passes 2^-126), found by least squares with reweighting on Chebyshev points against 64 bits.
__device__ __forceinline__ float normal_tail(float a) {
  const float r = __fdividef(1.0f, a + 3.75f), t = fmaf(-7.5f, r, 1.0f);
  float q = 0.00044344988418743014f;
  q = fmaf(q, t, 0.000509629026055336f);
  q = fmaf(q, t, -0.004169017542153597f);
  q = fmaf(q, t, 0.0012000735150650144f);
  q = fmaf(q, t, 0.037492506206035614f);
  q = fmaf(q, t, -0.15152083337306976f);
  q = fmaf(q, t, 0.3529396057128906f);
  q = fmaf(q, t, -0.5881882905960083f);
  q = fmaf(q, t, 0.7502940893173218f);
  return ex2(a * a * -0.72134752044448170f) * (r * q);
}

// Each form keeps its relative accuracy where it nears 0 on the left: no sum
// 1 + f with f near -1. silu and gelu's tanh form, g / (1 + e^-w) with w = g or
// 2 sqrt(2 / pi) (g + 0.044715 g^3), use the fast exponential and division, off by a few fp32
// steps and by about 1.2 |w| more where e^-w counts. gelu is max(g, 0) - |g| Phi(-|g|), off by a few steps and,
// on the left, by the argument's rounding times g^2. (T = 2048, N = 11008, K = 4096, gelu: 1 + erf, which loses
// its value there, 197 us; erfc 220; this 197. The tanh form by tanh 194, by the exponential 189.)
template <int ACT>
__device__ __forceinline__ float activate_as(float g) {
  if (ACT == kSilu) return __fdividef(g, 1.0f + __expf(-g));
  if (ACT == kGelu) {
    // |g|, cut at 64 on the right, where the tail is 0 from 15 on: an infinite g stays infinite there and becomes NaN
    // on the left, as in the formula.
    const float a = fmaxf(-g, fminf(g, 64.0f));
    return fmaf(-a, normal_tail(a), max_nan(g, 0.0f));
  }
  if (ACT == kGeluTanh) return __fdividef(g, 1.0f + __expf(-1.59576912160573071f * fmaf(0.044715f * g * g, g, g)));
  return g > 0.0f ? g : (g == g ? 0.0f : g);
}
__device__ __forceinline__ float activate(float g, int act) {
  switch (act) {
    case kSilu: return activate_as<kSilu>(g);
    case kGelu: return activate_as<kGelu>(g);
    case kGeluTanh: return activate_as<kGeluTanh>(g);
    default: return activate_as<kRelu>(g);
  }
}
// h = act(g) u for a row's gate values (acc[0]) and up values (acc[1]); one straight run of code per activation, since it is executed once a tile.
template <int ACT>
__device__ __forceinline__ void gate_row(const float2 (&acc)[2][32], float (&h)[64]) {
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    h[2 * c] = activate_as<ACT>(acc[0][c].x) * acc[1][c].x;
    h[2 * c + 1] = activate_as<ACT>(acc[0][c].y) * acc[1][c].y;
  }
}

struct Out {
  void* y;          // [T][ld] of `type`
  float* scale;     // e4m3: [ceil(N/128)][T]
  int64_t ld;
  int type;         // MOBI_F32, MOBI_BF16, MOBI_F16, MOBI_E4M3
  int vec;          // rows may be written 16 bytes at a time
};

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
}  // namespace f8

// ---- wide: tokens on lanes ---------------------------------------------------------

namespace f8w {
constexpr int BM = 256;                     // tokens of a pair's tile
constexpr int kThreads = 12 * 32;           // 0 producer, 1 and 2 MMA, 3 scales, 4-11 epilogue
constexpr int kGroupM = 8;                  // token tiles swept together over the weight tiles (L2 reuse)
constexpr int kRing = 8, kAhead = 6;        // fetched scales: slots, and blocks between the fetch and the use
constexpr uint64_t kDrainLimit = 1 << 16;   // polls while the last copies land (only an abort runs them out)

// BN: weight rows of a tile, 256 (gated: 128 gate + 128 up) or 128.
template <int BN>
struct Smem {
  static constexpr int ST = BN == 256 ? 5 : 7;      // pipeline stages (one block of K each)
  static constexpr int NB = 512 / BN;               // accumulator buffers in TMEM
  static constexpr uint32_t kB = BN / 2 * f8::BK;   // a CTA's half of the weight rows
  static constexpr uint32_t kStage = f8::kTileBytes + kB;
  uint8_t a[ST][f8::kTileBytes];            // 1024-byte aligned (offset 0)
  uint8_t b[ST][kB];
  uint8_t out[f8::kEpiWarps][32 * 128];     // per warp: 32 rows x 128 bytes, 16-byte chunk j of row r at j ^ (r & 7)
  float xs[kRing][128];                     // fetched scales of the CTA's tokens and of the tile's weight blocks
  float ws[kRing][4];
  float scale[2 * NB][BN / 128][128];       // their products: [slot][weight block][token]
  uint32_t rowmax[2][128];                  // e4m3 output: |h| maxima of a row's two halves
  // full and d_empty are used in the first CTA of the pair (it issues the MMAs), empty and d_full in both.
  uint64_t full[ST], empty[ST], d_full[NB], d_empty[NB], drain;
  uint32_t tmem_base;
  int32_t abort_flag;
  // A parity wait tells a phase from the one before it only. An MMA thread tests block u + 2's stage once
  // block u's buffer is free, which says that u - NB and all before it have gone through.
  static_assert(ST >= NB + 2, "stages");
};

// Tile index -> (token tile, weight tile): kGroupM token tiles at a time, weight
// tiles outermost within them, so CTAs that run together share both operands.
__device__ __forceinline__ void tile_at(int64_t i, int64_t n_mt, int64_t n_nt, int64_t* m, int64_t* n) {
  const int64_t per = kGroupM * n_nt, g = i / per, r = i % per;
  const int64_t left = n_mt - g * kGroupM, rows = left < kGroupM ? left : kGroupM;
  *m = g * kGroupM + r % rows;
  *n = r / rows;
}

// Writes a warp's staged 32 rows (row pitch 128 bytes, `cols` elements of ES
// bytes each) to y[t0 + row][n0 + col], clipped to T and N.
template <int ES, int COLS>
__device__ __forceinline__ void store_rows(const uint8_t* stage, uint8_t* y, int64_t ld, int64_t t0, int64_t T,
                                           int64_t n0, int64_t N, bool vec, int lane) {
  constexpr int CH = COLS * ES / 16, EC = 16 / ES;  // 16-byte chunks of a row, elements of a chunk
  if (vec && t0 + 32 <= T && n0 + COLS <= N) {
    const int row0 = lane / CH, ch = lane % CH;
    uint8_t* p = y + ((t0 + row0) * ld + n0 + ch * EC) * ES;
    const int64_t step = (32 / CH) * ld * ES;
#pragma unroll
    for (int i = 0; i < CH; ++i, p += step) {
      const int row = row0 + i * (32 / CH);
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(stage + row * 128 + 16 * (ch ^ (row & 7)));
    }
    return;
  }
  // Ragged tiles and rows that are not 16-byte aligned: an element per lane, so
  // that a warp still writes whole sectors (T = 333, N = 4099, bf16: eight elements per lane took 32 us, this 23.8).
  const int rows = T - t0 < 32 ? (int)(T - t0) : 32;
  for (int row = 0; row < rows; ++row) {
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += 32) {
      const int c = c0 + lane, at = row * 128 + 16 * ((c / EC) ^ (row & 7)) + c % EC * ES;
      if (n0 + c >= N) continue;
      uint8_t* p = y + ((t0 + row) * ld + n0 + c) * ES;
      if (ES == 4) *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(stage + at);
      if (ES == 2) *reinterpret_cast<uint16_t*>(p) = *reinterpret_cast<const uint16_t*>(stage + at);
      if (ES == 1) *p = stage[at];
    }
  }
}

// One warp's 32 rows x NC columns (acc, a row per lane) to y, through its staging rows.
template <int NC>
__device__ __forceinline__ void write_out(const float (&v)[NC], uint8_t* stage, const f8::Out& o, int64_t t0, int64_t T,
                                          int64_t n0, int64_t N, int lane) {
  uint8_t* y = static_cast<uint8_t*>(o.y);
  uint8_t* row = stage + lane * 128;
  if (o.type == MOBI_F32) {
#pragma unroll
    for (int c = 0; c < NC / 32; ++c) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(row + 16 * (j ^ (lane & 7))) =
            make_float4(v[32 * c + 4 * j], v[32 * c + 4 * j + 1], v[32 * c + 4 * j + 2], v[32 * c + 4 * j + 3]);
      __syncwarp();
      store_rows<4, 32>(stage, y, o.ld, t0, T, n0 + 32 * c, N, o.vec, lane);
    }
  } else {
    const bool half = o.type == MOBI_F16;
#pragma unroll
    for (int c = 0; c < NC / 64; ++c) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = v[64 * c + 8 * j + 2 * e], hi = v[64 * c + 8 * j + 2 * e + 1];
          w[e] = half ? f8::pack_f16(lo, hi) : f8::pack_bf16(lo, hi);
        }
        *reinterpret_cast<uint4*>(row + 16 * (j ^ (lane & 7))) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      __syncwarp();
      store_rows<2, 64>(stage, y, o.ld, t0, T, n0 + 64 * c, N, o.vec, lane);
    }
  }
}
}  // namespace f8w

template <bool GATED, int BN>
__global__ void __launch_bounds__(f8w::kThreads, 1)
    fp8_wide_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_u, const float* xs,
                    const float* ws, const float* us, int64_t T, int64_t N, int nkb, int act,
                    f8::Out out, DeviceStatus* st, uint64_t limit) {
  using namespace f8w;
  static_assert(BN == 256 || (BN == 128 && !GATED), "tile");
  using SM = Smem<BN>;
  constexpr int TN = GATED ? 128 : BN;  // output columns of a tile
  constexpr int ST = SM::ST, NB = SM::NB, WB = BN / 128;  // WB: weight blocks of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int32_t* abort_flag = &sm.abort_flag;
  const uint32_t rank = cluster_rank();
  const int64_t n_mt = (T + BM - 1) / BM, n_nt = (N + TN - 1) / TN, ntiles = n_mt * n_nt;
  const int64_t first = blockIdx.x / 2, stride = gridDim.x / 2;  // this pair's tiles
  const int64_t units = (ntiles - first + stride - 1) / stride * nkb;  // and their blocks (first < ntiles)

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) { mbar_init(&sm.full[i], 1); mbar_init(&sm.empty[i], 1); }
    for (int i = 0; i < NB; ++i) { mbar_init(&sm.d_full[i], 2); mbar_init(&sm.d_empty[i], 2 * f8::kEpiWarps); }
    mbar_init(&sm.drain, 2);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(&sm.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // both CTAs' barriers are set up before either signals the other's
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // 384 threads x 168 registers at launch = 128 x 56 + 256 x 224.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // ---- TMA producer: this CTA's tokens and its half of the weight rows (gated: gate or up) ----
      const CUtensorMap* tw = GATED && rank ? &tm_u : &tm_w;
      const uint32_t full0 = map_to_rank(&sm.full[0], 0);
      prefetch_tmap(&tm_x);
      prefetch_tmap(tw);
      uint32_t s = 0, ph = 1;
      int64_t issued = 0;
      bool ok = true;
      for (int64_t i = first; i < ntiles && ok; i += stride) {
        int64_t m, n;
        tile_at(i, n_mt, n_nt, &m, &n);
        const int xr = (int)(m * BM) + 128 * rank, wr = (int)(n * TN) + (GATED ? 0 : BN / 2 * rank);
        for (int kb = 0; kb < nkb; ++kb, ++issued) {
          if (!(ok = mbar_wait_abort(&sm.empty[s], ph, limit, st, 0x501, abort_flag))) break;
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * SM::kStage);
          const uint32_t bar = full0 + s * 8;
          tma_load_2d_pair(&sm.a[s][0], &tm_x, kb * f8::BK, xr, bar);
          tma_load_2d_pair(&sm.b[s][0], tw, kb * f8::BK, wr, bar);
          if (++s == ST) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // A stage's release says that its copies have landed and been read.
      for (int j = 0; j < ST && j < issued; ++j) {
        s = s == 0 ? ST - 1 : s - 1;
        if (s == ST - 1) ph ^= 1;
        mbar_wait(&sm.empty[s], ph ^ 1, kDrainLimit, st, 0x5F1);
      }
    } else if (warp == 1 || warp == 2) {
      // ---- MMA issuers, for both CTAs: warp 1 takes the even blocks, warp 2 the odd ones ----
      // Issuing waits for room in the tensor pipe's short queue, a barrier check
      // takes about 100 clocks even where it is ready, and a commit half of that:
      // one thread alone left the pipe idle for half of the time. Each thread
      // tests its next block's stage while it issues this one.
      if (lane == 0 && rank == 0) {
        constexpr uint32_t idesc = idesc_e4m3(BM, BN);
        const uint64_t a0 = desc_sw128(smem_addr(&sm.a[0][0])), b0 = desc_sw128(smem_addr(&sm.b[0][0]));
        uint32_t s = (uint32_t)(warp - 1), ph = 0, db = s, dph = 1;
        bool have = false;
        // A test-sized limit waits for what nothing completes, so that the timeout path always runs.
        const bool go = limit >= 64 || mbar_wait_abort(&sm.drain, 0, limit, st, 0x510, abort_flag);
        for (int64_t it = go ? warp - 1 : units; it < units; it += 2) {
          if (!mbar_wait_abort(&sm.d_empty[db], dph, limit, st, 0x512, abort_flag)) break;
          if (!have && !mbar_wait_abort(&sm.full[s], ph, limit, st, 0x511, abort_flag)) break;
          tc_fence_after();
          const uint32_t s0 = s, db0 = db, d = tmem + db * BN;
          const uint64_t a = a0 + s * (f8::kTileBytes / 16), b = b0 + s * (SM::kB / 16);
          db += 2;
          if (db >= NB) {
            db -= NB;
            dph ^= 1;
          }
          s += 2;
          if (s >= ST) {
            s -= ST;
            ph ^= 1;
          }
          have = mbar_test_wait(&sm.full[s], ph);
          mma_ss_f8_pair<false>(d, a, b, idesc);
          mma_ss_f8_pair<true>(d, a + 2, b + 2, idesc);
          mma_ss_f8_pair<true>(d, a + 4, b + 4, idesc);
          mma_ss_f8_pair<true>(d, a + 6, b + 6, idesc);
          mma_commit_pair(&sm.d_full[db0]);
          mma_commit_pair(&sm.empty[s0]);
        }
        mma_commit_pair_local(&sm.drain);  // every MMA issued is done before TMEM is released
        mbar_wait(&sm.drain, 0, kDefaultWaitLimit, st, 0x5F2);
      }
    } else if (warp == 3) {
      // ---- scales: fetched kAhead blocks before their use (under the tile loads' traffic a global load takes
      // longer than a block's MMAs), multiplied, and handed over with the block's sums (d_full counts both) ----
      const int64_t nblk = (N + 127) / 128;
      int64_t ftile = first;  // the next block to fetch
      int fkb = 0;
      const float *px = xs, *pw = ws;
      bool in[4];
      auto aim = [&]() {  // px, pw <- block 0 of tile ftile
        int64_t m, n;
        tile_at(ftile, n_mt, n_nt, &m, &n);
        const int64_t t = m * BM + 128 * rank + lane;
        px = xs + t;
#pragma unroll
        for (int j = 0; j < 4; ++j) in[j] = t + 32 * j < T;
        // Plain: the tile's columns are weight blocks WB n .. (where the tile ends
        // before the second, its sums are not written). Gated: block n of either matrix.
        const int64_t wb = GATED ? n : (WB * n + lane < nblk ? WB * n + lane : nblk - 1);
        pw = (GATED && lane == 1 ? us : ws) + wb;
      };
      auto fetch = [&](int64_t unit) {
        if (ftile < ntiles) {
          if (fkb == 0) aim();
          const int slot = (int)(unit % kRing);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (in[j]) copy4_async(&sm.xs[slot][lane + 32 * j], px + 32 * j);
          if (lane < WB) copy4_async(&sm.ws[slot][lane], pw);
          px += T;
          pw += nblk;
          if (++fkb == nkb) {
            fkb = 0;
            ftile += stride;
          }
        }
        copy_async_commit();
      };
      for (int j = 0; j < kAhead; ++j) fetch(j);
      for (int64_t it = 0; it < units; ++it) {
        // The slot's last readers took block it - 2 NB; block it - NB having its sums says that they are done.
        if (it >= NB && !mbar_wait_abort_warp(&sm.d_full[it % NB], (it / NB - 1) & 1, limit, st, 0x561, abort_flag))
          break;
        copy_async_wait<kAhead - 1>();
        __syncwarp();
        const int slot = (int)(it % kRing);
        float(*to)[128] = sm.scale[it % (2 * NB)];
#pragma unroll
        for (int w = 0; w < WB; ++w) {
          const float f = sm.ws[slot][w];
#pragma unroll
          for (int j = 0; j < 4; ++j) to[w][lane + 32 * j] = sm.xs[slot][lane + 32 * j] * f;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.d_full[it % NB]);
        fetch(it + kAhead);
      }
      copy_async_wait<0>();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ---- epilogue: promotion by the block scales, then the output ----
    const int e = warp - 4, q = warp & 3, half = e >> 2;
    const uint32_t lane_addr = (uint32_t)(32 * q) << 16;
    uint8_t* stage = sm.out[e];
    const uint32_t d_empty0 = map_to_rank(&sm.d_empty[0], 0);
    uint32_t it = 0;
    bool ok = true;
    // After an abort a warp still walks its tiles, without waits on mbarriers or
    // stores, since the other half of its rows may stand at their barrier.
    for (int64_t i = first; i < ntiles; i += stride) {
      int64_t m, n;
      tile_at(i, n_mt, n_nt, &m, &n);
      const int64_t trow = m * BM + 128 * rank + 32 * q, t = trow + lane;
      float2 acc[WB][32];  // plain: 64 (+ 64) columns; gated: 64 gate columns, the same 64 up columns
#pragma unroll
      for (int w = 0; w < WB; ++w)
#pragma unroll
        for (int c = 0; c < 32; ++c) acc[w][c] = make_float2(0.0f, 0.0f);
      for (int kb = 0; kb < nkb && ok; ++kb) {
        const uint32_t db = it % NB;
        if (!(ok = mbar_wait_abort_warp(&sm.d_full[db], (it / NB) & 1, limit, st, 0x521, abort_flag))) break;
        tc_fence_after();
        const float(*from)[128] = sm.scale[it % (2 * NB)];
        const float s0 = from[GATED || WB == 1 ? 0 : half][32 * q + lane];
        const float s1 = GATED ? from[WB - 1][32 * q + lane] : s0;
        ++it;
        // Loads of CW columns, each in flight while the one before is added; the
        // buffer is released as soon as the last has arrived.
        constexpr int CW = 16, NC = BN / 2 / CW;
        const uint32_t d = tmem + lane_addr + db * BN + half * (GATED ? 64 : BN / 2);
        uint32_t r[2][CW];
        tmem_ld16(d, r[0]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          tmem_ld_wait();
          if (c + 1 < NC) {
            const int col = (c + 1) * CW;
            tmem_ld16(d + (GATED ? (col / 64) * 128 + col % 64 : col), r[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(d_empty0 + db * 8);
          }
          const int h = c * CW / 64;
          const float v = h ? s1 : s0;
          const float2 s2 = make_float2(v, v);
#pragma unroll
          for (int j = 0; j < CW / 2; ++j) {
            float2& x = acc[h][(c * CW % 64) / 2 + j];
            x = __ffma2_rn(s2, make_float2(__uint_as_float(r[c & 1][2 * j]), __uint_as_float(r[c & 1][2 * j + 1])), x);
          }
        }
      }
      if constexpr (!GATED) {
        if (ok) {
          const int64_t n0 = n * BN + BN / 2 * half;
          write_out<64>(reinterpret_cast<const float(&)[64]>(acc[0]), stage, out, trow, T, n0, N, lane);
          if (WB == 2)
            write_out<64>(reinterpret_cast<const float(&)[64]>(acc[WB - 1]), stage, out, trow, T, n0 + 64, N, lane);
        }
      } else {
        float h[64];
        switch (act) {
          case f8::kSilu: f8::gate_row<f8::kSilu>(acc, h); break;
          case f8::kGelu: f8::gate_row<f8::kGelu>(acc, h); break;
          case f8::kGeluTanh: f8::gate_row<f8::kGeluTanh>(acc, h); break;
          default: f8::gate_row<f8::kRelu>(acc, h);
        }
        const int64_t n0 = n * 128 + 64 * half;
        if (out.type != MOBI_E4M3) {
          if (ok) write_out<64>(h, stage, out, trow, T, n0, N, lane);
        } else {
          // Block maximum of the row: this thread's 64 columns and, through
          // shared memory, the other half's. Columns past N are exact zeros
          // (zero-filled weights give g = u = 0).
          uint32_t a = 0;
#pragma unroll
          for (int c = 0; c < 64; ++c) a = max(a, abs_bits(h[c]));
          sm.rowmax[half][32 * q + lane] = a;
          f8::named_barrier(1 + q, 64);
          a = max(a, sm.rowmax[half ^ 1][32 * q + lane]);
          f8::named_barrier(1 + q, 64);  // read before the next tile writes it
          if (!ok) continue;
          const float s = block_scale(a), r = 1.0f / s;
          if (half == 0 && t < T) out.scale[n * T + t] = s;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = e4m3x2(h[16 * j + 4 * k] * r, h[16 * j + 4 * k + 1] * r) |
                     (e4m3x2(h[16 * j + 4 * k + 2] * r, h[16 * j + 4 * k + 3] * r) << 16);
            *reinterpret_cast<uint4*>(stage + lane * 128 + 16 * (j ^ (lane & 7))) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
          store_rows<1, 64>(stage, static_cast<uint8_t*>(out.y), out.ld, trow, T, n0, N, out.vec, lane);
        }
      }
    }
  }

  // Neither CTA leaves, or releases its TMEM, while the other may still use it.
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---- narrow: weight rows on lanes, K split over a cluster ------------------------------

namespace f8n {
constexpr int kThreads = 12 * 32;       // 0-7 epilogue, 8 producer, 9 and 10 MMA, 11 scales
constexpr int kRing = 8, kAhead = 6;    // fetched scales: slots, and blocks between the fetch and the use

template <bool GATED, int BN>
struct Cfg {
  static constexpr int MATS = GATED ? 2 : 1;
  static constexpr int COLS = MATS * BN;                     // accumulator columns of one block's sums
  static constexpr int HC = COLS / 2;                        // of which an epilogue warp takes half
  static constexpr int DST = 4;                              // accumulator buffers in TMEM (block & 3)
  static constexpr int TMEM = DST * COLS;
  static constexpr uint32_t kWBytes = MATS * f8::kTileBytes, kXBytes = BN * f8::BK;
  static constexpr uint32_t kStage = kWBytes + kXBytes;
  static constexpr int kPerSm = COLS <= 64 ? 2 : 1;          // CTAs that share an SM
  // Stages: about 100 KB (two CTAs) or 190 KB in flight, which covers the memory's latency at its bandwidth.
  static constexpr int ST = GATED ? (BN == 64 ? 5 : 3) : (BN == 16 ? 6 : (BN == 32 ? 5 : (BN == 64 ? 4 : 6)));
  static_assert(HC >= 8 && HC <= 64 && TMEM * kPerSm <= 512 && (TMEM & (TMEM - 1)) == 0, "tile");
  // CTAs of any of these kernels that fit an SM together (228 KB) fit its 512 columns together. Otherwise two clusters
  // of concurrent calls could each hold columns that the other's CTAs wait for, and the allocation waits without limit.
  static_assert(kPerSm == 2 ? ST * kStage > 76 * 1024 : ST * kStage > 152 * 1024, "shared memory");
  static constexpr int MT = ST >= 4 ? 2 : 1;                 // MMA threads (see there)
  static_assert(COLS * 512 <= ST * kStage, "the sums take the stages' place");
};

template <bool GATED, int BN>
struct Smem {
  using C = Cfg<GATED, BN>;
  union {
    struct {
      uint8_t w[C::ST][C::kWBytes];      // 1024-byte aligned (offset 0)
      uint8_t x[C::ST][C::kXBytes];
    };
    float red[C::COLS * 128];            // after the last block: this CTA's sums, [column][row]
  };
  float xs[kRing][BN];                   // fetched scales of the tile's tokens and weight blocks
  float ws[kRing][2];
  float scale[4][C::COLS];               // their products, by accumulator column
  uint32_t colmax[2][2][4];
  uint64_t full[C::ST], empty[C::ST], d_full[C::DST], d_empty[C::DST], drain;
  uint32_t tmem_base;
  int32_t abort_flag;
};
}  // namespace f8n

template <bool GATED, int BN>
__global__ void __launch_bounds__(f8n::kThreads, f8n::Cfg<GATED, BN>::kPerSm)
    fp8_narrow_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_u, const float* xs, const float* ws, const float* us,
                      int64_t T, int64_t N, int nkb, int csize, int act, f8::Out out, DeviceStatus* st,
                      uint64_t limit) {
  using CF = f8n::Cfg<GATED, BN>;
  using f8n::kAhead;
  using f8n::kRing;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  f8n::Smem<GATED, BN>& sm = *reinterpret_cast<f8n::Smem<GATED, BN>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int32_t* abort_flag = &sm.abort_flag;
  const uint32_t rank = cluster_rank();
  const int64_t n0 = (int64_t)(blockIdx.x / csize) * 128, t0 = (int64_t)blockIdx.y * BN;
  const int kb0 = (int)((int64_t)nkb * rank / csize), kb1 = (int)((int64_t)nkb * (rank + 1) / csize);
  const int64_t nblk = (N + 127) / 128, wb = n0 / 128;

  // The producer sets up the barriers and has the first stages on their way while
  // the other warps get tensor memory.
  auto load = [&](int kb, uint32_t s) {
    mbar_arrive_expect_tx(&sm.full[s], CF::kStage);
    tma_load_2d(&sm.w[s][0], &tm_w, kb * f8::BK, (int)n0, &sm.full[s]);
    if (GATED) tma_load_2d(&sm.w[s][f8::kTileBytes], &tm_u, kb * f8::BK, (int)n0, &sm.full[s]);
    tma_load_2d(&sm.x[s][0], &tm_x, kb * f8::BK, (int)t0, &sm.full[s]);
  };
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x);
    if (GATED) prefetch_tmap(&tm_u);
    for (int i = 0; i < CF::ST; ++i) { mbar_init(&sm.full[i], 1); mbar_init(&sm.empty[i], 1); }
    for (int i = 0; i < CF::DST; ++i) { mbar_init(&sm.d_full[i], 2); mbar_init(&sm.d_empty[i], f8::kEpiWarps); }
    mbar_init(&sm.drain, 2);
    sm.abort_flag = 0;
    fence_barrier_init();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = 0; i < CF::ST && kb0 + i < kb1; ++i) load(kb0 + i, (uint32_t)i);
  }
  if (warp == 9) tmem_alloc(&sm.tmem_base, CF::TMEM);
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  float2 acc[CF::HC / 2];
#pragma unroll
  for (int c = 0; c < CF::HC / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
  const int half = warp >> 2, q = warp & 3;
  const int mat = GATED ? half : 0, j0 = GATED ? 0 : half * CF::HC;  // matrix and first token of this warp's columns

  if (warp == 8) {
    if (lane == 0) {
      // ---- TMA producer (the first ST blocks are on their way) ----
      uint32_t s = 0, ph = 0;
      int kb = kb0 + CF::ST < kb1 ? kb0 + CF::ST : kb1;
      if (kb - kb0 < CF::ST) {
        s = (uint32_t)(kb - kb0);
        ph = 1;
      }
      for (; kb < kb1; ++kb) {
        if (!mbar_wait_abort(&sm.empty[s], ph, limit, st, 0x531, abort_flag)) break;
        load(kb, s);
        if (++s == CF::ST) {
          s = 0;
          ph ^= 1;
        }
      }
      for (int j = 0; j < CF::ST && j < kb - kb0; ++j) {  // every copy lands before its stage is used again
        s = s == 0 ? CF::ST - 1 : s - 1;
        if (s == CF::ST - 1) ph ^= 1;
        mbar_wait(&sm.full[s], ph ^ 1, kDefaultWaitLimit, st, 0x5F3);
      }
    }
  } else if (warp == 9 || warp == 10) {
    if (lane == 0) {
      // ---- MMA issuers: with MT = 2, warp 9 takes the even blocks and warp 10 the odd ones (a block's
      // instructions take one thread longer than its MMAs run) ----
      // A parity wait tells a phase from the one before it only, so a thread may
      // wait for block u's stage once block u - ST has gone through it. With two
      // threads that follows from the buffer: it is free when block u - 4 has been
      // added, and blocks are added in order, so ST >= 4 is needed there.
      constexpr int MT = CF::MT;
      constexpr uint32_t idesc = idesc_e4m3(128, BN);
      const uint64_t w0 = desc_sw128(smem_addr(&sm.w[0][0])), x0 = desc_sw128(smem_addr(&sm.x[0][0]));
      const int first = warp - 9;
      uint32_t s = (uint32_t)first, ph = 0, db = s, dph = 1;
      // As in the wide kernel: a test-sized limit always runs out here.
      const bool go = limit >= 64 || mbar_wait_abort(&sm.drain, 0, limit, st, 0x540, abort_flag);
      for (int kb = go && first < MT ? kb0 + first : kb1; kb < kb1; kb += MT) {
        if (!mbar_wait_abort(&sm.d_empty[db], dph, limit, st, 0x542, abort_flag)) break;
        if (!mbar_wait_abort(&sm.full[s], ph, limit, st, 0x541, abort_flag)) break;
        tc_fence_after();
        const uint64_t w = w0 + s * (CF::kWBytes / 16), x = x0 + s * (CF::kXBytes / 16);
        const uint32_t d = tmem + db * CF::COLS, s0 = s, db0 = db;
        s += MT;
        if (s >= CF::ST) {
          s -= CF::ST;
          ph ^= 1;
        }
        db += MT;
        if (db >= 4) {
          db -= 4;
          dph ^= 1;
        }
#pragma unroll
        for (int mt = 0; mt < CF::MATS; ++mt) {
          const uint64_t wm = w + mt * (f8::kTileBytes / 16);
          mma_ss_f8<false>(d + mt * BN, wm, x, idesc);
          mma_ss_f8<true>(d + mt * BN, wm + 2, x + 2, idesc);
          mma_ss_f8<true>(d + mt * BN, wm + 4, x + 4, idesc);
          mma_ss_f8<true>(d + mt * BN, wm + 6, x + 6, idesc);
        }
        mma_commit(&sm.d_full[db0]);
        mma_commit(&sm.empty[s0]);
      }
      mma_commit(&sm.drain);
      mbar_wait(&sm.drain, 0, kDefaultWaitLimit, st, 0x5F4);
    }
  } else if (warp == 11) {
    // ---- scales: fetched kAhead blocks ahead, multiplied, handed over with the block's sums ----
    constexpr int NX = (BN + 31) / 32;
    const float* px = xs + (int64_t)kb0 * T + t0 + lane;
    const float* pw = (GATED && lane == 1 ? us : ws) + (int64_t)kb0 * nblk + wb;
    bool in[NX];
#pragma unroll
    for (int j = 0; j < NX; ++j) in[j] = lane + 32 * j < BN && t0 + lane + 32 * j < T;
    auto fetch = [&](int i) {  // block kb0 + i
      if (kb0 + i < kb1) {
        const int slot = i % kRing;
#pragma unroll
        for (int j = 0; j < NX; ++j)
          if (in[j]) copy4_async(&sm.xs[slot][lane + 32 * j], px + 32 * j);
        if (lane < CF::MATS) copy4_async(&sm.ws[slot][lane], pw);
        px += T;
        pw += nblk;
      }
      copy_async_commit();
    };
    for (int i = 0; i < kAhead; ++i) fetch(i);
    bool have = true;
    for (int i = 0; kb0 + i < kb1; ++i) {
      // The slot's last readers took block i - 4, whose buffer block i's MMAs wait for as well.
      if (!__all_sync(0xffffffffu, have) &&
          !mbar_wait_abort_warp(&sm.d_empty[i & 3], ((i >> 2) - 1) & 1, limit, st, 0x562, abort_flag))
        break;
      copy_async_wait<kAhead - 1>();
      __syncwarp();
      const int slot = i % kRing;
      const float w0 = sm.ws[slot][0], w1 = sm.ws[slot][CF::MATS - 1];
#pragma unroll
      for (int j = 0; j < NX; ++j) {
        const int c = lane + 32 * j;
        if (c < BN) {
          const float x = in[j] ? sm.xs[slot][c] : 0.0f;
          sm.scale[i & 3][c] = x * w0;
          if (GATED) sm.scale[i & 3][BN + c] = x * w1;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.d_full[i & 3]);
      have = i + 1 < 4 || mbar_test_wait(&sm.d_empty[(i + 1) & 3], (((i + 1) >> 2) - 1) & 1);
      fetch(i + kAhead);
    }
    copy_async_wait<0>();
  } else {
    // ---- epilogue: promotion by the column's scale ----
    const uint32_t lane_addr = (uint32_t)(32 * q) << 16;
    for (int i = 0; kb0 + i < kb1; ++i) {
      const uint32_t db = i & 3;
      if (!mbar_wait_abort_warp(&sm.d_full[db], (i >> 2) & 1, limit, st, 0x551, abort_flag)) break;
      tc_fence_after();
      const float* sc = &sm.scale[db][half * CF::HC];
      const uint32_t d = tmem + lane_addr + db * CF::COLS + half * CF::HC;
      constexpr int LC = CF::HC < 16 ? CF::HC : (CF::kPerSm == 2 ? 16 : 32);  // columns per TMEM load
#pragma unroll
      for (int c = 0; c < CF::HC / LC; ++c) {
        uint32_t r[LC];
        if constexpr (LC == 8) tmem_ld8(d, r);
        if constexpr (LC == 16) tmem_ld16(d + 16 * c, r);
        if constexpr (LC == 32) tmem_ld32(d + 32 * c, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < LC / 4; ++j) {
          const float4 s4 = *reinterpret_cast<const float4*>(&sc[LC * c + 4 * j]);
          float2* a = &acc[LC / 2 * c + 2 * j];
          a[0] = __ffma2_rn(make_float2(s4.x, s4.y),
                            make_float2(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])), a[0]);
          a[1] = __ffma2_rn(make_float2(s4.z, s4.w),
                            make_float2(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])), a[1]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.d_empty[db]);
    }
  }

  // The cluster's sums. Every CTA lays its own out in its shared memory, in the
  // stages' place (every block of its own has been read by then: the last sums
  // say so); CTA r then reads the tokens [r tpc, (r + 1) tpc) of all of them and
  // adds them in rank order, so the result does not depend on who finishes first.
  if (warp < 8) {
    float* mine = &sm.red[(half * CF::HC) * 128 + 32 * q + lane];
#pragma unroll
    for (int c = 0; c < CF::HC; ++c) mine[c * 128] = (c & 1) ? acc[c >> 1].y : acc[c >> 1].x;
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  const int tpc = (BN + csize - 1) / csize;
  if (warp < 8) {
    const int row = threadIdx.x & 127;
    const int64_t n = n0 + row;
    uint32_t peer[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) peer[c] = map_to_rank(&sm.red[row], c < csize ? c : 0);
    for (int tl = half; tl < tpc; tl += 2) {  // tokens of this CTA, alternating between the two groups of 128 threads
      const int j = (int)rank * tpc + tl;
      const int64_t t = t0 + j;
      if (t >= T || j >= BN) break;
      float a[8], b[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        a[c] = b[c] = 0.0f;
        if (c < csize) {
          a[c] = ld_cluster(peer[c] + (uint32_t)j * 512);
          if (GATED) b[c] = ld_cluster(peer[c] + (uint32_t)(BN + j) * 512);
        }
      }
      float v = a[0], u = b[0];
#pragma unroll
      for (int c = 1; c < 8; ++c)
        if (c < csize) {
          v += a[c];
          u += b[c];
        }
      if (GATED) v = f8::activate(v, act) * u;
      if (GATED && out.type == MOBI_E4M3) {
        uint32_t m = __reduce_max_sync(0xffffffffu, abs_bits(v));
        uint32_t* cm = sm.colmax[half][(tl >> 1) & 1];
        if (lane == 0) cm[q] = m;
        f8::named_barrier(1 + half, 128);
        m = max(max(cm[0], cm[1]), max(cm[2], cm[3]));
        const float s = block_scale(m), r = 1.0f / s;
        if (row == 0) out.scale[wb * T + t] = s;
        if (n < N) static_cast<uint8_t*>(out.y)[t * out.ld + n] = (uint8_t)e4m3x2(v * r, 0.0f);
      } else if (n < N) {
        const int64_t at = t * out.ld + n;
        if (out.type == MOBI_F32) static_cast<float*>(out.y)[at] = v;
        else if (out.type == MOBI_BF16) static_cast<__nv_bfloat16*>(out.y)[at] = __float2bfloat16_rn(v);
        else static_cast<__half*>(out.y)[at] = __float2half_rn(v);
      }
    }
  }

  // No CTA leaves while another may still read its sums.
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, CF::TMEM);
  }
}

// ---- host side ---------------------------------------------------------------------

struct Fp8Job {
  const void *X, *W, *U;
  const float *xs, *ws, *us;
  int64_t ldx, ldw, ldu, T, N, K;
  f8::Out out;
  int act;
};

// Which kernel, its token tile (narrow) or weight tile (wide), and the narrow one's cluster.
struct Fp8Plan {
  bool wide;
  int bn, csize;
};

// Clusters of c = 1 .. 8 CTAs that run at once, one CTA to an SM (what
// cudaOccupancyMaxActiveClusters answers on a B200's 148 SMs).
constexpr int kClusters[9] = {0, 148, 74, 45, 33, 26, 22, 15, 15};

// The narrow kernel's token tile is the batch rounded up, to 128 (gated 64) at
// most. K is cut over a cluster, two blocks of 128 to a CTA at least: up to the
// device's room where two CTAs share an SM (T = 1, N = K = 4096, clusters of 8, 4,
// 2: 6.2, 6.9, 8.6 us; T = 8, gated, N = 11008: clusters of 3, 2, 4: 18.6, 22.3,
// 23.6 us), by the fewest blocks in a row where one does.
// From 33 tokens on the kernels' times are estimated from their waves and
// blocks, in units of 10 ns fitted at K = 4096 and 11008, N = 1024, 4096 and 11008,
// T = 64 .. 2048; shorter K and narrower N follow from the same terms, unmeasured.
// Measured at K = 4096, in us, narrow / wide with 128 and with 256 weight rows: T = 64,
// N = 11008: 15.2 / 23.2 / 22; T = 333, N = 4096: 32 / 14.0 / 20.6; T = 256, N = 11008:
// - / 24.1 / 22.8; T = 2048, N = 4096: - / 47 / 38.6.
static Fp8Plan fp8_plan(int64_t T, int64_t N, int64_t K, bool gated, int sms) {
  Fp8Plan p;
  const auto up = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
  const int64_t nkb = up(K, 128), nt = up(N, 128), mt = up(T, f8w::BM);
  p.wide = false;
  p.bn = T <= 16 ? 16 : (T <= 32 ? 32 : (T <= 64 || gated ? 64 : 128));
  const int64_t tiles = nt * up(T, p.bn);
  int64_t row, waves = 1;  // blocks in a row of a CTA, CTAs in a row on an SM
  if (p.bn * (gated ? 2 : 1) <= 64) {
    int64_t c = 2 * (int64_t)sms / tiles;
    if (c > nkb / 2) c = nkb / 2;
    p.csize = (int)(c < 1 ? 1 : (c > 8 ? 8 : c));
    row = up(nkb, p.csize);
    waves = up(tiles * p.csize, 2 * (int64_t)sms);
  } else {
    p.csize = 1;
    row = nkb;
    waves = up(tiles, kClusters[1]);
    for (int c = 2; c <= 8 && 2 * c <= nkb; ++c) {
      const int64_t r = up(nkb, c), w = up(tiles, kClusters[c]);
      if (w * r < waves * row) {
        p.csize = c;
        row = r;
        waves = w;
      }
    }
  }
  if (T <= 32) return p;
  const int64_t narrow = 600 + waves * row * 85;
  const int64_t wide256 = 450 + nkb * (56 * up(mt * (gated ? nt : up(nt, 2)), sms / 2) - 6);
  const int64_t wide128 = gated ? wide256 : 400 + nkb * (34 * up(mt * nt, sms / 2) - 4);
  if (wide256 < narrow || wide128 < narrow) {
    p.wide = true;
    p.bn = wide128 < wide256 ? 128 : 256;
  }
  return p;
}

template <bool GATED, int BN>
static cudaError_t launch_narrow(const Fp8Job& j, const Fp8Plan& p, const CUtensorMap& mx, const CUtensorMap& mw,
                                 const CUtensorMap& mu, cudaStream_t stream, DeviceStatus* st) {
  constexpr int smem = (int)sizeof(f8n::Smem<GATED, BN>) + 1024;
  static_assert(smem <= 232448, "shared memory");
  cudaError_t e = set_smem((const void*)fp8_narrow_kernel<GATED, BN>, smem);
  if (e != cudaSuccess) return e;
  const int64_t nt = (j.N + 127) / 128, tt = (j.T + BN - 1) / BN;
  e = launch_dependent(fp8_narrow_kernel<GATED, BN>, dim3((unsigned)(nt * p.csize), (unsigned)tt), f8n::kThreads, smem,
                       p.csize, stream, mx, mw, mu, j.xs, j.ws, j.us, j.T, j.N, (int)((j.K + 127) / 128), p.csize,
                       j.act, j.out, st, wait_limit());
  return note_error("fp8 narrow launch", e);
}

template <bool GATED, int BN>
static cudaError_t launch_wide(const Fp8Job& j, const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& mu,
                               cudaStream_t stream, DeviceStatus* st) {
  constexpr int smem = (int)sizeof(f8w::Smem<BN>) + 1024, TN = GATED ? 128 : BN;
  static_assert(smem <= 232448 && smem > 152 * 1024, "shared memory");  // alone on its SM, which has 512 TMEM columns
  cudaError_t e = set_smem((const void*)fp8_wide_kernel<GATED, BN>, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((j.T + f8w::BM - 1) / f8w::BM) * ((j.N + TN - 1) / TN), pairs = num_sms() / 2;
  e = launch_dependent(fp8_wide_kernel<GATED, BN>, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), f8w::kThreads,
                       smem, 2, stream, mx, mw, mu, j.xs, j.ws, j.us, j.T, j.N, (int)((j.K + 127) / 128), j.act, j.out,
                       st, wait_limit());
  return note_error("fp8 wide launch", e);
}

template <bool GATED>
static cudaError_t launch_fp8(const Fp8Job& j, cudaStream_t stream) {
  cudaError_t e;
  DeviceStatus* st = device_status(&e);
  if (!st) return e;
  const int sms = num_sms();
  const Fp8Plan p = fp8_plan(j.T, j.N, j.K, GATED, sms);
  CUtensorMap mx, mw, mu = {};
  const uint32_t rows_x = p.wide ? 128 : (uint32_t)p.bn, rows_w = p.wide && p.bn == 128 ? 64 : 128;
  if (!make_tmap_u8(&mx, j.X, (uint64_t)j.K, (uint64_t)j.T, (uint64_t)j.ldx, rows_x) ||
      !make_tmap_u8(&mw, j.W, (uint64_t)j.K, (uint64_t)j.N, (uint64_t)j.ldw, rows_w) ||
      (GATED && !make_tmap_u8(&mu, j.U, (uint64_t)j.K, (uint64_t)j.N, (uint64_t)j.ldu, rows_w)))
    return cudaErrorInvalidValue;
  if (!p.wide) {
    switch (p.bn) {
      case 16: return launch_narrow<GATED, 16>(j, p, mx, mw, mu, stream, st);
      case 32: return launch_narrow<GATED, 32>(j, p, mx, mw, mu, stream, st);
      case 64: return launch_narrow<GATED, 64>(j, p, mx, mw, mu, stream, st);
      default:
        if constexpr (!GATED) return launch_narrow<false, 128>(j, p, mx, mw, mu, stream, st);
        return cudaErrorInvalidValue;
    }
  }
  if constexpr (!GATED)
    if (p.bn == 128) return launch_wide<false, 128>(j, mx, mw, mu, stream, st);
  return launch_wide<GATED, 256>(j, mx, mw, mu, stream, st);
}

namespace {
constexpr int64_t kMaxDim = int64_t(1) << 28;

bool aligned(const void* p, int a) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(a - 1)) == 0; }

// An e4m3 operand [rows][K] with pitch ld and its scales.
mobi_status check_operand(const void* Q, int64_t ld, int64_t K, const float* s) {
  if (!Q || !s || ld < K) return MOBI_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || ld % 16 != 0 || !aligned(s, 4)) return MOBI_ERR_MISALIGNED;
  return MOBI_OK;
}

mobi_status check_sizes(int64_t T, int64_t N, int64_t K) {
  if (T < 0 || N < 0 || K < 0) return MOBI_ERR_INVALID_ARG;
  if (T > kMaxDim || N > kMaxDim || K > kMaxDim) return MOBI_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && N > 0 && K == 0) return MOBI_ERR_UNSUPPORTED_SHAPE;
  return MOBI_OK;
}

int dtype_bytes(int t) { return t == MOBI_F32 ? 4 : (t == MOBI_E4M3 ? 1 : 2); }

mobi_status check_out(void* y, int64_t ld, int64_t N, int type, f8::Out* o) {
  const int es = dtype_bytes(type);
  if (!y || ld < N) return MOBI_ERR_INVALID_ARG;
  if (!aligned(y, es)) return MOBI_ERR_MISALIGNED;
  *o = f8::Out{y, nullptr, ld, type, aligned(y, 16) && ld * es % 16 == 0};
  return MOBI_OK;
}
}  // namespace

}  // namespace mobi

using namespace mobi;

extern "C" {

mobi_status mobi_fp8_gemm(const void* X, int64_t ldx, const float* xs, int64_t T, int64_t K, const void* W, int64_t ldw,
                          const float* wsc, int64_t N, int out_dtype, void* Y, int64_t ldy, void* stream) {
  clear_message();
  if (out_dtype != MOBI_F32 && out_dtype != MOBI_BF16 && out_dtype != MOBI_F16) return MOBI_ERR_INVALID_ARG;
  mobi_status s = check_sizes(T, N, K);
  if (s != MOBI_OK || T == 0 || N == 0) return s;
  Fp8Job j = {X, W, nullptr, xs, wsc, nullptr, ldx, ldw, 0, T, N, K, {}, 0};
  if ((s = check_operand(X, ldx, K, xs)) != MOBI_OK || (s = check_operand(W, ldw, K, wsc)) != MOBI_OK ||
      (s = check_out(Y, ldy, N, out_dtype, &j.out)) != MOBI_OK)
    return s;
  return status_of(launch_fp8<false>(j, static_cast<cudaStream_t>(stream)));
}

mobi_status mobi_fp8_gated(const void* X, int64_t ldx, const float* xs, int64_t T, int64_t K, const void* Wg,
                           int64_t ldg, const float* gs, const void* Wu, int64_t ldu, const float* us, int64_t N,
                           int act, int out_dtype, void* H, int64_t ldh, float* hs, void* stream) {
  clear_message();
  if (out_dtype < MOBI_F32 || out_dtype > MOBI_E4M3 || act < MOBI_ACT_SILU || act > MOBI_ACT_RELU)
    return MOBI_ERR_INVALID_ARG;
  mobi_status s = check_sizes(T, N, K);
  if (s != MOBI_OK || T == 0 || N == 0) return s;
  Fp8Job j = {X, Wg, Wu, xs, gs, us, ldx, ldg, ldu, T, N, K, {}, act};
  if ((s = check_operand(X, ldx, K, xs)) != MOBI_OK || (s = check_operand(Wg, ldg, K, gs)) != MOBI_OK ||
      (s = check_operand(Wu, ldu, K, us)) != MOBI_OK || (s = check_out(H, ldh, N, out_dtype, &j.out)) != MOBI_OK)
    return s;
  if (out_dtype == MOBI_E4M3) {
    if (!hs) return MOBI_ERR_INVALID_ARG;
    if (!aligned(hs, 4)) return MOBI_ERR_MISALIGNED;
    j.out.scale = hs;
  }
  return status_of(launch_fp8<true>(j, static_cast<cudaStream_t>(stream)));
}

mobi_status mobi_debug_fp8_plan(int64_t T, int64_t N, int64_t K, int gated, int sms, int64_t plan[5]) {
  clear_message();
  if (T < 1 || N < 1 || K < 1 || gated < 0 || gated > 1 || sms < 2 || !plan) return MOBI_ERR_INVALID_ARG;
  if (T > kMaxDim || N > kMaxDim || K > kMaxDim) return MOBI_ERR_UNSUPPORTED_SHAPE;
  const Fp8Plan p = fp8_plan(T, N, K, gated != 0, sms);
  const int64_t tt = p.wide ? f8w::BM : p.bn, tn = p.wide && !gated ? p.bn : 128;  // tokens and outputs of a tile
  plan[0] = p.wide;
  plan[1] = p.bn;
  plan[2] = p.wide ? 2 : p.csize;
  plan[3] = ((T + tt - 1) / tt) * ((N + tn - 1) / tn);
  plan[4] = p.wide ? (plan[3] + sms / 2 - 1) / (sms / 2) : 1;
  return MOBI_OK;
}

}  // extern "C"
