// mobi_logprobs.cu — log probabilities of given tokens, entropy and the top
// alternatives of rows of logits.
//
// With c = log2(e) / temperature, m the running maximum and w = (x - m) c:
//   S = sum 2^w,  W = sum 2^w w     (rescaled when m grows: W <- f (W + d S), S <- f S, f = 2^d)
//   logprob = (x_target - m) / temperature - ln S,   entropy = ln S - ln 2 * W / S
// one pass over the row in fp32, no logarithm per element.
//
// An entry of -infinity is counted as "floor" (-1e30, or fp16's lowest), which
// spares a guard against 0 * infinity per value; with the running maximum
// starting there too, such entries vanish once a real one is seen. A part
// whose maximum is not far above the floor is summed again, value by value.
// Values are taken in pairs: about six instructions each, of which the
// exponential's unit is the next bound (bf16).
//
// Top alternatives without a second pass over the row: neighbouring threads
// form 128 groups, and the k-th largest of the groups' maxima (k <= 32) is a bound tau
// that at least k entries reach. Only groups whose maximum reaches it can hold
// one, so about k/128 of the row is read again, and the entries >= tau are
// gathered and ranked. The second reading adds 12%, 43% and 60% to the bytes of fp32 rows
// for k = 5, 20 and 32, and 8%, 33% and 52% to those of bf16 rows (T = 1024, V = 128000). (Keeping
// entries as they come by instead, against a bound from the first loads: when fp32 rows took 272 us
// at T = 2048, V = 128000 that made them 195, and bf16 rows 146 instead of 108 at V = 128001. One form
// stands for all types, the faster one for 16 bits.) Many equal entries would overflow the gather: then the
// entries above tau are gathered and the first ones equal to it are found in
// index order. Where that does not do (even those overflow, or fewer than k
// groups have an entry above the floor, as under a mask of the type's lowest
// value), the row is searched for the next lower value and its first entries
// until there are k.
//
// Few rows: a cluster of up to eight CTAs shares a row; CTA 0 joins their
// statistics and candidates through distributed shared memory, in rank order.
#include <cmath>
#include <cstdint>

#include "mobi_device.cuh"
#include "mobi_host.h"

namespace mobi {

namespace lp {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Group g is lanes 2 (g % 16) and the next of warp g / 16: 32 bytes in a row of every load, one sector when read again.
constexpr int kGroups = kThreads / 2;
constexpr int kMaxK = 32;
constexpr int kCap = 1024;   // gathered candidates
constexpr float kLowest = -3.402823466e38f;

// What -infinity counts as, and the same as a pair of 16-bit patterns.
template <typename E>
struct Floor {
  static constexpr float value = -1.0e30f;  // fp32
};
template <>
struct Floor<__nv_bfloat16> {
  static constexpr uint32_t pair = 0xf149f149u;
  static constexpr float value = -9.95303792e+29f;  // 0xf149
};
template <>
struct Floor<__half> {
  static constexpr uint32_t pair = 0xfbfffbffu;
  static constexpr float value = -65504.0f;
};

struct Stat {
  float m, s, w;
};

// a joined with b. A part without entries has m = kLowest, s = w = 0; f > 0 keeps 0 * infinity out of w.
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float da = (a.m - m) * c, db = (b.m - m) * c, fa = ex2(da), fb = ex2(db);
  Stat r;
  r.m = m;
  r.s = a.s * fa + b.s * fb;
  r.w = (fa > 0.0f ? fa * fmaf(da, a.s, a.w) : 0.0f) + (fb > 0.0f ? fb * fmaf(db, b.s, b.w) : 0.0f);
  return r;
}

// max(a, b, c), ignoring NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Larger of two pairs of 16-bit values, NaN if either is.
template <typename E>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (Floor<E>::pair == Floor<__half>::pair)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Adds U times 16 bytes of logits to a running state that starts at the floor;
// one rescaling for all of them.
template <typename E, int U>
__device__ __forceinline__ void add_chunks(Stat& a, const uint4 (&r)[U], float c) {
  uint32_t w[4 * U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    w[4 * u] = r[u].x;
    w[4 * u + 1] = r[u].y;
    w[4 * u + 2] = r[u].z;
    w[4 * u + 3] = r[u].w;
  }
  float m = a.m;
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) w[i] = __float_as_uint(max_nan(__uint_as_float(w[i]), Floor<E>::value));
#pragma unroll
    for (int i = 0; i < 4 * U; i += 2) m = max3(m, __uint_as_float(w[i]), __uint_as_float(w[i + 1]));
  } else {
    // A NaN would carry through the packed maximum into m; it shows in the sums all the same.
    uint32_t x = Floor<E>::pair;
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) {
      w[i] = max_pair<E>(w[i], Floor<E>::pair);
      x = i ? max_pair<E>(x, w[i]) : w[i];
    }
    m = max3(m, elem_f32<E>((uint16_t)x), elem_f32<E>((uint16_t)(x >> 16)));
  }
  if (m > a.m) {
    const float d = (a.m - m) * c, f = ex2(d);
    a.w = f > 0.0f ? f * fmaf(d, a.s, a.w) : 0.0f;
    a.s *= f;
    a.m = m;
  }
  const float2 neg = make_float2(-a.m, -a.m), c2 = make_float2(c, c);
  float2 s = make_float2(0.0f, 0.0f), t = s;
  auto one = [&](float2 x) {
    const float2 v = __fmul2_rn(__fadd2_rn(x, neg), c2);
    const float2 e = make_float2(ex2(v.x), ex2(v.y));
    s = __fadd2_rn(s, e);
    t = __ffma2_rn(e, v, t);
  };
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < 4 * U; i += 2) one(make_float2(__uint_as_float(w[i]), __uint_as_float(w[i + 1])));
  } else {
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) one(make_float2(elem_f32<E>((uint16_t)w[i]), elem_f32<E>((uint16_t)(w[i] >> 16))));
  }
  a.s += s.x + s.y;
  a.w += t.x + t.y;
}

// Adds N values (fp32) to a running state that starts at {kLowest, 0, 0}.
template <int N>
__device__ __forceinline__ void add(Stat& a, const float (&x)[N], float c) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
  if (m > a.m) {
    const float d = (a.m - m) * c, f = ex2(d);
    a.w = f > 0.0f ? f * fmaf(d, a.s, a.w) : 0.0f;
    a.s *= f;
    a.m = m;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float w = (x[i] - a.m) * c, e = ex2(w);  // -infinity: e = 0
    a.s += e;
    a.w = fmaf(e, fmaxf(w, -1.0e4f), a.w);           // e = 0 long before -1e4: 0 and not 0 * infinity
  }
}

// Candidates order by value, then the lower index first, as one integer.
__device__ __forceinline__ uint64_t make_key(float x, uint32_t index) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 and 0 are equal
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((uint64_t)o << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return ~(uint32_t)k; }

// A CTA's part of a row: elements [lo, hi), of which [body, body + 16-byte chunks) are aligned.
template <typename E>
struct Part {
  static constexpr int EC = 16 / sizeof(E);
  const E* row;
  int64_t lo, hi, body, tail;  // tail = body + EC * chunks
  int chunks;

  __device__ __forceinline__ void chunk(int i, float (&x)[EC]) const { widen(raw(i), x); }
  __device__ __forceinline__ uint4 raw(int i) const { return reinterpret_cast<const uint4*>(row + body)[i]; }
  static __device__ __forceinline__ void widen(const uint4& a, float (&x)[EC]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(E) == 4) {
        x[j] = __uint_as_float(w[j]);
      } else {
        x[2 * j] = elem_f32<E>((uint16_t)w[j]);
        x[2 * j + 1] = elem_f32<E>((uint16_t)(w[j] >> 16));
      }
    }
  }
  // The j-th element outside the aligned body (there are edge() of them, at most 2 (EC - 1)).
  __device__ __forceinline__ int edge() const { return (int)(body - lo + hi - tail); }
  __device__ __forceinline__ int64_t edge_at(int j) const {
    return lo + j < body ? lo + j : tail + (j - (body - lo));
  }
};

template <typename E>
__device__ __forceinline__ Part<E> make_part(const E* row, int64_t lo, int64_t hi) {
  constexpr int EC = Part<E>::EC;
  Part<E> p;
  p.row = row;
  p.lo = lo;
  p.hi = hi;
  const uintptr_t a = reinterpret_cast<uintptr_t>(row + lo);
  int64_t head = (int64_t)((16 - a % 16) % 16 / sizeof(E));
  if (head > hi - lo) head = hi - lo;
  p.body = lo + head;
  p.chunks = (int)((hi - p.body) / EC);
  p.tail = p.body + (int64_t)p.chunks * EC;
  return p;
}

struct Smem {
  Stat warp[kWarps];
  alignas(16) float gmax[kGroups];  // the groups' maxima
  float tau;
  int n, groups;
  int list[kGroups];
  uint64_t key[kCap + kMaxK];
  float best[kWarps];
  uint64_t top[kMaxK];             // this CTA's part, in order (0: none)
  Stat total;
  int count[kWarps];
};

__device__ __forceinline__ void push(Smem& sm, float x, int64_t i) {
  if (*(volatile int*)&sm.n > kCap) return;  // already overflowed: the count only has to stay above kCap
  const int at = atomicAdd(&sm.n, 1);
  if (at < kCap) sm.key[at] = make_key(x, (uint32_t)i);
}

// Gathers the entries >= tau (strict: > tau) of the part into sm.key, sm.n their count.
template <typename E>
__device__ void gather(Smem& sm, const Part<E>& p, float tau, bool strict) {
  constexpr int EC = Part<E>::EC;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) sm.n = sm.groups = 0;
  __syncthreads();
  if (tid < kGroups && (strict ? sm.gmax[tid] > tau : sm.gmax[tid] >= tau)) sm.list[atomicAdd(&sm.groups, 1)] = tid;
  __syncthreads();
  const int ng = sm.groups, per = (p.chunks + kThreads - 1) / kThreads;  // chunks of a thread
  for (int g = warp; g < ng; g += kWarps) {
    const int id = sm.list[g], base = 32 * (id / 16) + 2 * (id % 16);
    for (int j0 = lane; j0 < 2 * per; j0 += 4 * 32) {
      uint4 r[4];
      int at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + 32 * u;
        at[u] = (j >> 1) * kThreads + base + (j & 1);
        if (at[u] < p.chunks) r[u] = p.raw(at[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (at[u] >= p.chunks) continue;
        float x[EC];
        Part<E>::widen(r[u], x);
#pragma unroll
        for (int e = 0; e < EC; ++e)
          if ((strict ? x[e] > tau : x[e] >= tau) && x[e] > -INFINITY)
            push(sm, x[e], p.body + (int64_t)at[u] * EC + e);
      }
    }
  }
  if (tid < p.edge()) {
    const int64_t i = p.edge_at(tid);
    const float x = to_f32(p.row[i]);
    if ((strict ? x > tau : x >= tau) && x > -INFINITY) push(sm, x, i);
  }
  __syncthreads();
}

// Appends the first `need` entries equal to v, in index order, as candidates n, n + 1, ..; returns how many there were (at most need).
template <typename E>
__device__ int first_equal(Smem& sm, const Part<E>& p, float v, int need, int n) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int have = 0;
  for (int64_t i0 = p.lo; i0 < p.hi && have < need; i0 += kThreads) {
    const int64_t i = i0 + tid;
    const bool eq = i < p.hi && to_f32(p.row[i]) == v;
    const unsigned b = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) sm.count[warp] = __popc(b);
    __syncthreads();
    int before = have, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm.count[w];
      all += sm.count[w];
    }
    before += __popc(b & ((1u << lane) - 1));
    if (eq && before < need) sm.key[n + before] = make_key(v, (uint32_t)i);
    have += all;
  }
  __syncthreads();
  return have < need ? have : need;
}

// The part's largest entry below `bound` (equal: or equal to it), -infinity if there is none.
template <typename E>
__device__ float next_value(Smem& sm, const Part<E>& p, float bound, bool equal) {
  constexpr int EC = Part<E>::EC;
  const int tid = threadIdx.x;
  float best = -INFINITY;
  for (int i = tid; i < p.chunks; i += kThreads) {
    float x[EC];
    p.chunk(i, x);
#pragma unroll
    for (int e = 0; e < EC; ++e)
      if (x[e] < bound || (equal && x[e] == bound)) best = fmaxf(best, x[e]);
  }
  if (tid < p.edge()) {
    const float x = to_f32(p.row[p.edge_at(tid)]);
    if (x < bound || (equal && x == bound)) best = fmaxf(best, x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  __syncthreads();
  if ((tid & 31) == 0) sm.best[tid >> 5] = best;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) best = fmaxf(best, sm.best[w]);
  return best;
}

// sm.top[0..k) <- the part's k largest keys in order (0 where there are fewer).
template <typename E>
__device__ void top_keys(Smem& sm, const Part<E>& p, int k) {
  const int tid = threadIdx.x;
  if (tid < kMaxK) sm.top[tid] = 0;
  __syncthreads();
  // The k-th largest group maximum. A warp ranks sixteen groups: lanes l and
  // l + 16 count one group's larger and equal ones among half of the others each.
  {
    const int lane = tid & 31, half = lane >> 4;
    const float v = sm.gmax[16 * (tid >> 5) + (lane & 15)];
    int more = 0, same = 0;
    const float4* other = reinterpret_cast<const float4*>(&sm.gmax[half * (kGroups / 2)]);
#pragma unroll
    for (int i = 0; i < kGroups / 8; ++i) {
      const float4 o = other[i];
      more += (o.x > v) + (o.y > v) + (o.z > v) + (o.w > v);
      same += (o.x == v) + (o.y == v) + (o.z == v) + (o.w == v);
    }
    more += __shfl_xor_sync(0xffffffffu, more, 16);
    same += __shfl_xor_sync(0xffffffffu, same, 16);
    if (more < k && k <= more + same) sm.tau = v;  // equal values only
  }
  __syncthreads();
  const float tau = sm.tau, floor = Floor<E>::value;
  const bool floored = tau <= floor;  // group maxima at the floor stand for -infinity and for what is below it
  int n = 0;
  float bound = INFINITY;
  bool equal = false, more = true;
  gather(sm, p, floored ? floor : tau, floored);
  if (sm.n <= kCap) {
    n = sm.n;
    more = floored;
    bound = floor;
    equal = true;
  } else if (!floored) {
    __syncthreads();
    gather(sm, p, tau, true);
    if (sm.n <= kCap) {
      n = sm.n;
      bound = tau;
      equal = true;
    }
  }
  __syncthreads();
  while (more && n < k) {
    const float v = next_value(sm, p, bound, equal);
    if (v == -INFINITY) break;
    n += first_equal(sm, p, v, k - n, n);
    bound = v;
    equal = false;
  }
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t key = sm.key[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += sm.key[j] > key;
    if (rank < k) sm.top[rank] = key;
  }
  __syncthreads();
}

// sm.total <- the threads' states joined, in a fixed order: the maximum first,
// then sums of states rescaled to it.
__device__ __forceinline__ void block_join(Smem& sm, Stat a, float c) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto over = [&](int first) {
    float m = a.m;
    for (int o = first; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float d = (a.m - m) * c, f = ex2(d);
    a.w = f > 0.0f ? f * fmaf(d, a.s, a.w) : 0.0f;
    a.s *= f;
    a.m = m;
    for (int o = first; o > 0; o >>= 1) {
      a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
      a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
    }
  };
  over(16);
  if (lane == 0) sm.warp[warp] = a;
  __syncthreads();
  if (warp == 0) {
    a = sm.warp[lane % kWarps];
    over(kWarps / 2);
    if (lane == 0) sm.total = a;
  }
  __syncthreads();
}

// An 8-byte or 4-byte word of CTA `rank`'s shared memory (the same variable there).
template <typename V>
__device__ __forceinline__ V remote(const V* p, uint32_t rank) {
  const uint32_t a = map_to_rank(p, rank);
  V v;
  if constexpr (sizeof(V) == 8)
    asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  else
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

template <typename E>
__global__ void __launch_bounds__(kThreads, 6)
    logprobs_kernel(const E* logits, int64_t V, int64_t ld, const int64_t* targets, float temperature, int k,
                    int csize, float* logprob, float* entropy, float* top_logprob, int32_t* top_index,
                    DeviceStatus* st) {
  constexpr int EC = Part<E>::EC, U = 4;  // chunks of a thread in flight
  __shared__ Smem sm;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x / csize;
  const int rank = blockIdx.x % csize;
  const E* row = logits + t * ld;
  const float c = 1.44269504088896341f / temperature;
  const Part<E> p = make_part(row, V * rank / csize, V * (rank + 1) / csize);

  // The target's logit is on its way while the row is summed.
  int64_t y = -1;
  float xt = 0.0f;
  if (tid == 0 && rank == 0 && targets) {
    y = targets[t];
    if (y >= 0 && y < V) xt = to_f32(row[y]);
  }
  Stat a = {Floor<E>::value, 0.0f, 0.0f};
  for (int i = tid; i < p.chunks; i += U * kThreads) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      constexpr uint32_t none = sizeof(E) == 4 ? 0xff800000u : (Floor<E>::value == -65504.0f ? 0xfc00fc00u : 0xff80ff80u);
      r[u] = make_uint4(none, none, none, none);  // -infinity
      if (i + u * kThreads < p.chunks) r[u] = p.raw(i + u * kThreads);
    }
    add_chunks<E, U>(a, r, c);
  }
  if (tid < p.edge()) {
    const float x[1] = {max_nan(to_f32(row[p.edge_at(tid)]), Floor<E>::value)};
    add<1>(a, x, c);
  }

  if (k > 0) {
    const float pair = fmaxf(a.m, __shfl_xor_sync(0xffffffffu, a.m, 1));
    const float g = __shfl_sync(0xffffffffu, pair, 2 * tid & 31);  // lanes 0 .. 15 hold the warp's groups in order
    if ((tid & 31) < 16) sm.gmax[16 * (tid >> 5) + (tid & 31)] = g;
  }
  block_join(sm, a, c);
  // Entries at the floor have to be nothing beside the largest one, and no
  // exponent may overflow (far larger logits or smaller temperatures than a model's).
  const float span = (sm.total.m - Floor<E>::value) * c;
  if (!(span >= 150.0f && span <= 1.0e37f)) {
    a = Stat{kLowest, 0.0f, 0.0f};
    for (int i = tid; i < p.chunks; i += kThreads) {
      float x[EC];
      p.chunk(i, x);
      add<EC>(a, x, c);
    }
    if (tid < p.edge()) {
      const float x[1] = {to_f32(row[p.edge_at(tid)])};
      add<1>(a, x, c);
    }
    __syncthreads();
    block_join(sm, a, c);
  }
  if (k > 0) top_keys(sm, p, k);

  if (csize > 1) {
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    if (rank == 0) {
      if (tid == 0) {
        Stat all = sm.total;
        for (int r = 1; r < csize; ++r) {
          const Stat b = {remote(&sm.total.m, r), remote(&sm.total.s, r), remote(&sm.total.w, r)};
          all = join(all, b, c);
        }
        sm.total = all;
      }
      const int n = csize * k;  // <= 8 * 32
      if (tid < n) sm.key[tid] = remote(&sm.top[tid % k], tid / k);
      __syncthreads();
      const uint64_t key = tid < n ? sm.key[tid] : 0;
      if (tid < kMaxK) sm.top[tid] = 0;
      __syncthreads();
      if (key) {
        int at = 0;
        for (int j = 0; j < n; ++j) at += sm.key[j] > key;
        if (at < k) sm.top[at] = key;
      }
    }
    // CTA 0 has read the others' shared memory before they leave.
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
  }
  __syncthreads();
  a = sm.total;
  const float log_s = logf(a.s);
  const bool empty = a.s == 0.0f;
  if (tid < k) {
    const uint64_t key = sm.top[tid];
    top_index[t * k + tid] = key ? (int32_t)key_index(key) : -1;
    top_logprob[t * k + tid] = key ? (key_value(key) - a.m) / temperature - log_s : -INFINITY;
  }
  if (tid == 0) {
    if (entropy) entropy[t] = empty ? 0.0f : log_s - 0.693147180559945309f * (a.w / a.s);
    if (targets) {
      float v = 0.0f;
      if (y >= V) {
        v = NAN;
        report_error(st, kErrTargetRange, 0x601);
      } else if (y >= 0) {
        v = empty ? -INFINITY : (xt - a.m) / temperature - log_s;
      }
      logprob[t] = v;
    }
  }
}

template <typename E>
static cudaError_t launch(const void* logits, int64_t T, int64_t V, int64_t ld, const int64_t* targets,
                          float temperature, int k, float* logprob, float* entropy, float* top_logprob,
                          int32_t* top_index, cudaStream_t stream) {
  cudaError_t e;
  DeviceStatus* st = device_status(&e);
  if (!st) return e;
  // A cluster shares a row while the rows leave SMs idle and each CTA keeps a
  // load or more per thread.
  int csize = 1;
  while (csize < 8 && T * csize * 2 <= num_sms() && V >= (int64_t)csize * 2 * kThreads * Part<E>::EC) csize *= 2;
  return launch_dependent(logprobs_kernel<E>, dim3((unsigned)(T * csize)), kThreads, 0, csize, stream,
                          static_cast<const E*>(logits), V, ld, targets, temperature, k, csize, logprob, entropy,
                          top_logprob, top_index, st);
}

}  // namespace lp

}  // namespace mobi

using namespace mobi;

extern "C" mobi_status mobi_logprobs(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                                     const int64_t* targets, float temperature, int top_k, float* logprob,
                                     float* entropy, float* top_logprob, int32_t* top_index, void* stream) {
  clear_message();
  if (T < 0 || V < 1 || dtype < MOBI_F32 || dtype > MOBI_F16 || top_k < 0 || top_k > lp::kMaxK)
    return MOBI_ERR_INVALID_ARG;
  if (!(temperature >= 1e-30f) || !std::isfinite(temperature)) return MOBI_ERR_INVALID_ARG;
  if (T > (int64_t(1) << 28) || V > (int64_t(1) << 28)) return MOBI_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOBI_OK;
  if (!logits || ld < V || (targets && !logprob) || (top_k > 0 && (!top_logprob || !top_index)))
    return MOBI_ERR_INVALID_ARG;
  auto off = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
  if (off(logits, dtype == MOBI_F32 ? 4 : 2) || off(targets, 8) || off(logprob, 4) || off(entropy, 4) ||
      off(top_logprob, 4) || off(top_index, 4))
    return MOBI_ERR_MISALIGNED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto fn = dtype == MOBI_F32 ? lp::launch<float> : (dtype == MOBI_BF16 ? lp::launch<__nv_bfloat16> : lp::launch<__half>);
  return status_of(note_error("logprobs launch", fn(logits, T, V, ld, targets, temperature, top_k, logprob, entropy,
                                                    top_logprob, top_index, s)));
}
