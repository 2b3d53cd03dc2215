// Sampling: one token from each row of logits, by temperature, top-k, top-p,
// min-p and a given random number.
//
// The kept tokens are those above a border: a logit K, and how many of the equal
// ones at it (the lowest ids) still belong.  Top-k looks for the border by counts,
// top-p by masses; neither sorts.  A row's logits are read once and stay in the
// shared memory of a cluster of CTAs, a slice each.  A histogram of 2048 equal
// steps of (max - l) / temperature, summed over the cluster, says in which step the
// border lies; that step's logits, some hundreds at most in a vocabulary's usual
// spread, are gathered from all slices and compared with one another.  (Bins of the
// numbers' leading bits, as a radix sort has them, put most of a row into a dozen
// bins, and their atomics took 200 of 237 us for one row of 248320.)  Where more
// than 1024 lie in the step, as where logits are equal, the border is found digit by
// digit.  A top_k of up to 256 needs no histogram: the threads' own largest logits bound
// the top_k-th from below, the few logits above that bound go to the first CTA, and it
// orders them.  The token then is the first id, in the vocabulary's order, where the
// running sum of the kept weights passes u times their sum.
//
// A weight is exp((l - max) / temperature) in fixed point, 44 bits behind the
// point, and sums are of 64-bit integers: a row of 393216 equal ones still fits, sums
// are exact, and no order of atomics or CTAs moves a border or a token.
//
// Measured: one row of 248320 fp32 with top_k 20 and top_p 0.8 10 us, 64 rows of 151936
// fp16 with top_p 0.95 and min_p 0.02 27 us.  Bytes (0.15 and 2.9 us) bound neither:
// a row's path is a handful of passes over shared memory with a wait for the whole
// cluster after each (1000 to 2500 cycles), and of a batch the weights' arithmetic
// (15 instructions a logit and pass) and, without min_p, the bins' atomics.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kq_device.cuh"
#include "kq_gdn.cuh"
#include "kq_internal.h"
#include "kq_kv.cuh"

namespace kq {
namespace sample {

namespace cg = cooperative_groups;

__device__ unsigned int g_sample_status = 0;
__device__ __forceinline__ void sample_flag(int status) { atomicOr(&g_sample_status, 1u << status); }

constexpr int kMostVocab = 393216;
constexpr int kPortable = 8, kMostCluster = 16;
constexpr int kMostSlice = kMostVocab / kPortable;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kSubs = 1024;
constexpr float kOne = 17592186044416.f;  // 2^44

struct Args {
  const void* logits;
  int64_t row_stride;
  int32_t vocab, slice;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* token;
  float* prob;
};

typedef unsigned long long u64;

constexpr int kList = 1024;
// top_k up to which the candidates are gathered without a histogram (one row of 248320 fp32 with a top_k of 128, 256, 257: 14, 18,
// 30 us; 64 rows of 151936 fp16 with 256, 257: 27, 43)
constexpr int kFewK = 256;

// What each CTA of a cluster tells all others: its largest and least logit, whether it has a NaN, its bounds for the top_k-th,
// how many logits it listed, the sum of its share of the bins, its weight, and of that what min_p leaves, and what is kept, how
// many at the border it has.
enum { kRange, kNan, kBounds, kListed, kBinned, kWhole, kOver, kKept, kTies, kTold };

// What the CTAs of a cluster show one another.
struct alignas(16) Shared {  // the slice lies behind it, in words of 16 bytes
  union {
    struct {
      uint32_t low[kBins], high[kBins];  // sums of 64 bits
    } hist;
    struct {
      u64 weight[kList];
      uint32_t key[kList];  // of all slices
    } all;
    u64 sorted[kList];      // key above the complement of the id
  };
  struct {
    uint32_t low[kSubs], high[kSubs];
  } sub;
  union {
    uint32_t list[kList];  // keys of this slice's logits in the border's step
    u64 top[kList];        // of those that may be among the top_k, each above the complement of its id
  };
  u64 told[kTold][kMostCluster];
  u64 part[kWarps];
  uint32_t at_k, at_share;
  int32_t lowest, listed, members;
  int32_t bin, subbin;
  u64 above, inside, rest;
  uint32_t key;
  u64 equal, need;
};

__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// A row's weights.  EXACT: the difference from the largest is kept to its rounding error too.  Of 16-bit logits it is not: where a
// large one is the largest and others are small (16.5 and odd multiples of 2^-24) it has one, 2^-24 of itself, and a weight is
// off by 2^-24 of its exponent, which is 31 at most before nothing is left of the weight; such logits' own rounding is 2^-12 of
// them and more (64 rows of 151936 f16 with top_p 0.95, with and without min_p 0.02: 26.6 and 53 us, exactly 29 and 57).
template <bool EXACT>
struct Row {
  float most;      // the largest logit
  float hi, lo;    // log2(e) / temperature in two floats
  // exp((v - most) / temperature) of two logits, in packed operations: the product with the factor is kept to twice fp32's
  // bits, so the error is that of the exponential instruction (2^-22) and the difference's.  Infinitely far below the
  // largest, the exponential is 0 and what the product lacks is no number: 0 then, whatever the temperature.
  __device__ __forceinline__ float2 exp_of(float2 v) const {
    const float2 d = add2(v, make_float2(-most, -most)), h = make_float2(hi, hi), p = mul2(d, h);
    float2 rest = fma2(d, make_float2(lo, lo), fma2(d, h, make_float2(-p.x, -p.y)));
    if (EXACT) {
      const float2 minus = make_float2(-1.f, -1.f), b = fma2(v, minus, d);  // v - most = d + err exactly
      const float2 err = add2(fma2(fma2(b, minus, d), minus, v), fma2(b, minus, make_float2(-most, -most)));
      rest = fma2(err, h, rest);
    }
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(p.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(p.y));
    e = fma2(mul2(e, rest), make_float2(0.69314718f, 0.69314718f), e);
    return make_float2(fmaxf(e.x, 0.f), fmaxf(e.y, 0.f));
  }
  __device__ __forceinline__ float exp_of(float v) const { return exp_of(make_float2(v, v)).x; }
  // In units of 2^-44, by additions that leave the wanted bits at the end of a number: 22 in front, then the rest (signed),
  // each above what `none` has.
  static __device__ __forceinline__ void fixed(float2 e, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
    const float2 top = add2(e, make_float2(2.0f, 2.0f)), less = add2(top, make_float2(-2.0f, -2.0f));
    const float2 rest = fma2(fma2(less, make_float2(-1.f, -1.f), e), make_float2(kOne, kOne), make_float2(12582912.0f, 12582912.0f));
    hi[0] = __float_as_uint(top.x), hi[1] = __float_as_uint(top.y);
    lo[0] = __float_as_uint(rest.x), lo[1] = __float_as_uint(rest.y);
  }
  static constexpr uint32_t kNoneHi = 0x40000000u, kNoneLo = 0x4B400000u;  // of a weight of zero
  // The sum of `count` weights from the sums of their parts, which so many as a thread sees do not carry over 32 bits but for
  // the multiples of `none`.
  static __device__ __forceinline__ u64 joined(uint32_t hi, uint32_t lo, uint32_t count) {
    return ((u64)(hi - count * kNoneHi) << 22) + (int64_t)(int32_t)(lo - count * kNoneLo);
  }
  static __device__ __forceinline__ u64 fixed(float e) {
    uint32_t hi[2], lo[2];
    fixed(make_float2(e, e), hi, lo);
    return joined(hi[0], lo[0], 1);
  }
  __device__ __forceinline__ u64 weight(float v) const { return fixed(exp_of(v)); }
};

// Sorts 512 keys, one a thread, the largest first.
__device__ __forceinline__ uint32_t sort_threads(uint32_t k, uint32_t* swap) {
  const int tid = threadIdx.x;
  for (int size = 2; size <= kThreads; size *= 2)
    for (int stride = size / 2; stride; stride /= 2) {
      uint32_t o;
      if (stride < 32) {
        o = __shfl_xor_sync(~0u, k, stride);
      } else {
        __syncthreads();
        swap[tid] = k;
        __syncthreads();
        o = swap[tid ^ stride];
      }
      const bool larger = ((tid & size) == 0) == ((tid & stride) == 0);
      k = larger ? max(k, o) : min(k, o);
    }
  return k;
}

// Sorts the first `count` (a power of two up to kList) of v, the largest first; v is written before and read after by any
// thread.  Up to 512 a thread has one in registers, and lanes exchange theirs where they can.
__device__ __forceinline__ void sort_list(u64* v, int count) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (count <= kThreads) {
    u64 k = tid < count ? v[tid] : 0;
    for (int size = 2; size <= count; size *= 2)
      for (int stride = size / 2; stride; stride /= 2) {
        u64 o;
        if (stride < 32) {
          if (tid / 32 * 32 >= count) continue;
          o = __shfl_xor_sync(~0u, k, stride);
        } else {
          __syncthreads();
          if (tid < count) v[tid] = k;
          __syncthreads();
          o = tid < count ? v[tid ^ stride] : 0;
        }
        const bool larger = ((tid & size) == 0) == ((tid & stride) == 0);
        k = (k < o) == larger ? o : k;
      }
    __syncthreads();
    if (tid < count) v[tid] = k;
  } else {
    for (int size = 2; size <= count; size *= 2)
      for (int stride = size / 2; stride; stride /= 2) {
        __syncthreads();
        const int i = tid / stride * 2 * stride + tid % stride;  // kThreads = kList / 2
        const u64 x = v[i], y = v[i + stride];
        if ((x < y) == ((i & size) == 0)) v[i] = y, v[i + stride] = x;
      }
  }
  __syncthreads();
}

// How many of the n numbers of v, up to kRanked, are more than one of them, and how many are equal to it: that of this thread's
// group of four, tid / 4.  (For so few it takes a quarter of the time that sorting them does.)
constexpr int kRanked = kThreads / 4;
template <typename V>
__device__ __forceinline__ void ranked(const V* v, int n, V mine, int& more, int& same) {
  more = same = 0;
  for (int j = threadIdx.x % 4; j < n; j += 4) {
    const V o = v[j];
    more += o > mine, same += o == mine;
  }
#pragma unroll
  for (int o = 1; o < 4; o *= 2) more += __shfl_xor_sync(~0u, more, o), same += __shfl_xor_sync(~0u, same, o);
}

// The first n of v into falling order, in `to` (n up to kRanked; equal ones are zero, and are left out) or else in place;
// returns where.
__device__ __forceinline__ u64* ordered(u64* v, u64* to, int n) {
  const int tid = threadIdx.x;
  if (n <= kRanked) {
    if (tid < kRanked) to[tid] = 0;
    __syncthreads();
    const u64 mine = tid / 4 < n ? v[tid / 4] : 0;
    int more, same;
    ranked(v, n, mine, more, same);
    if (tid % 4 == 0 && mine) to[more] = mine;
    __syncthreads();
    return to;
  }
  int wide = 2;
  while (wide < n) wide *= 2;
  for (int i = n + tid; i < wide; i += kThreads) v[i] = 0;
  sort_list(v, wide);
  return v;
}

template <typename V, typename F>
__device__ __forceinline__ V block_reduce(V v, V* part, F join, V none) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = join(v, __shfl_xor_sync(~0u, v, o));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int warps = kWarps;
  __syncthreads();
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : none;
#pragma unroll
  for (int o = 16; o; o >>= 1) v = join(v, __shfl_xor_sync(~0u, v, o));
  return v;
}

// That all CTAs of the cluster run, before one writes another's memory.
struct Started {
  __device__ __forceinline__ Started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
  __device__ __forceinline__ void wait() const { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  Shared& s = *reinterpret_cast<Shared*>(s_raw);
  T* s_l = reinterpret_cast<T*>(s_raw + sizeof(Shared));
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int64_t row = blockIdx.x / ranks;
  constexpr int warps = kWarps;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int first = rank * a.slice, n = max(0, min(a.slice, a.vocab - first));
  Started started;
  grid_dependency_wait();
  allow_dependent_launch();

  const float t = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
  const float min_p = a.min_p ? a.min_p[row] : 0.f;
  const int32_t top_k = a.top_k ? a.top_k[row] : 0;
  const float u = a.u[row];
  const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.f, few = by_k && top_k <= kFewK;

  // the slice, its largest
  const T* src = static_cast<const T*>(a.logits) + row * a.row_stride + first;
  float most = -INFINITY, lowest = INFINITY;
  int nan = 0;
  auto see = [&](T x) {
    const float v = kv::to_float(x);
    most = fmaxf(most, v);
    lowest = fminf(lowest, v);
    nan |= isnan(v);
  };
  constexpr int kVec = 16 / sizeof(T);
  if (((uintptr_t)src & 15) == 0) {
    for (int i = tid; i < n / kVec; i += kThreads) {
      union { uint4 u; T t[kVec]; } x;
      x.u = reinterpret_cast<const uint4*>(src)[i];  // (no read-only load: the grid may have begun while the logits were written)
      reinterpret_cast<uint4*>(s_l)[i] = x.u;
#pragma unroll
      for (int e = 0; e < kVec; ++e) see(x.t[e]);
    }
    for (int i = n / kVec * kVec + tid; i < n; i += kThreads) see(s_l[i] = src[i]);
  } else {
    for (int i = tid; i < n; i += kThreads) see(s_l[i] = src[i]);
  }
  const int vecs = (n + kVec - 1) / kVec;
  for (int i = n + tid; i < vecs * kVec; i += kThreads) s_l[i] = kv::from_float<T>(-INFINITY);  // weighs nothing
  // f(value) of each logit of the slice, in any order
  auto each = [&](auto f) {
    for (int i = tid; i < vecs; i += kThreads) {
      union { uint4 u; T t[kVec]; } x;
      x.u = reinterpret_cast<const uint4*>(s_l)[i];
#pragma unroll
      for (int e = 0; e < kVec; ++e) f(kv::to_float(x.t[e]));
    }
  };
  auto each2 = [&](auto f) {
    for (int i = tid; i < vecs; i += kThreads) {
      union { uint4 u; T t[kVec]; } x;
      x.u = reinterpret_cast<const uint4*>(s_l)[i];
#pragma unroll
      for (int e = 0; e < kVec; e += 2) f(make_float2(kv::to_float(x.t[e]), kv::to_float(x.t[e + 1])));
    }
  };
  // Told to all, before the cluster's barrier, and read from this CTA's own memory after it, a lane each.  (Read by every warp
  // from the others' memory, one word of one CTA a lane, it took 2 to 4 us each time that 16 CTAs met.)
  auto tell = [&](int what, u64 x) {
    if (tid < ranks) cluster.map_shared_rank(&s, tid)->told[what][rank] = x;
  };
  auto told = [&](int what, u64 none) { return lane < ranks ? s.told[what][lane] : none; };
  float* fpart = reinterpret_cast<float*>(s.part);
  int* ipart = reinterpret_cast<int*>(s.part);
  if (few) {  // what the top_k-th largest of all cannot lie below: a CTA's own, or the least of the CTAs' shares of top_k
    uint32_t k = most == -INFINITY ? 0 : key_of(most);
    const int share = (top_k + ranks - 1) / ranks;
    if (top_k <= kRanked / 2) {  // of groups of four threads
      k = max(k, __shfl_xor_sync(~0u, k, 1));
      k = max(k, __shfl_xor_sync(~0u, k, 2));
      if (tid % 4 == 0) s.list[tid / 4] = k;
      __syncthreads();
      int more, same;
      ranked(s.list, kRanked, k, more, same);
      if (more < top_k && top_k <= more + same) s.at_k = k;
      if (more < share && share <= more + same) s.at_share = k;
    } else {
      k = sort_threads(k, s.list);
      if (tid == top_k - 1) s.at_k = k;
      if (tid == share - 1) s.at_share = k;
    }
  }
  most = block_reduce(most, fpart, [](float x, float y) { return fmaxf(x, y); }, -INFINITY);
  lowest = block_reduce(lowest, fpart, [](float x, float y) { return fminf(x, y); }, INFINITY);
  nan = __syncthreads_or(nan);
  started.wait();
  const auto pair = [](uint32_t high, uint32_t low) { return (u64)high << 32 | low; };
  tell(kRange, pair(__float_as_uint(most), __float_as_uint(lowest)));
  tell(kNan, nan);
  if (few) tell(kBounds, pair(s.at_k, s.at_share));
  cluster.sync();
  const u64 range = told(kRange, pair(__float_as_uint(-INFINITY), __float_as_uint(INFINITY)));
  most = __uint_as_float((uint32_t)(range >> 32)), lowest = __uint_as_float((uint32_t)range);
  nan = (int)told(kNan, 0);
#pragma unroll
  for (int o = 8; o; o >>= 1) {
    most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
    lowest = fminf(lowest, __shfl_xor_sync(~0u, lowest, o));
  }
  most = __shfl_sync(~0u, most, 0), lowest = __shfl_sync(~0u, lowest, 0);
  nan = __any_sync(~0u, nan);
  uint32_t bound = 0;
  if (few) {
    const u64 bounds = told(kBounds, 0xFFFFFFFFu);
    bound = max(__reduce_max_sync(~0u, (uint32_t)(bounds >> 32)), __reduce_min_sync(~0u, (uint32_t)bounds));
  }

  const bool bad = nan || most == -INFINITY || !(t >= 0.f) || isinf(t) || isnan(top_p) || isnan(min_p);
  if (bad) {
    if (rank == 0 && tid == 0) {
      sample_flag(KQ_ERR_NONFINITE);
      a.token[row] = -1;
      if (a.prob) a.prob[row] = 0.f;
    }
    cluster.sync();  // nobody leaves while its memory is read
    return;
  }

  if (t == 0.f || top_k == 1 || top_p <= 0.f || min_p > 1.f) {  // the largest alone, its lowest id
    int at = 0x7fffffff;
    for (int i = tid; i < n; i += kThreads)
      if (kv::to_float(s_l[i]) == most) at = min(at, first + i);
    at = block_reduce(at, ipart, [](int x, int y) { return min(x, y); }, 0x7fffffff);
    if (tid == 0) s.lowest = at;
    cluster.sync();
    if (rank == 0 && tid == 0) {
      for (int c = 1; c < ranks; ++c) at = min(at, cluster.map_shared_rank(&s, c)->lowest);
      a.token[row] = at;
      if (a.prob) a.prob[row] = 1.f;
    }
    cluster.sync();
    return;
  }
  if (isinf(most)) {  // those alone weigh, one each
    for (int i = tid; i < vecs * kVec; i += kThreads) s_l[i] = kv::from_float<T>(kv::to_float(s_l[i]) == most ? 0.f : -INFINITY);
    most = 0.f;
    bound = min(bound, key_of(0.f));
    __syncthreads();
  }
  Row<sizeof(T) == 4> w;
  w.most = most;
  // log2(e) / t: the quotient, and what it lacks (1.44269502 + 1.925963e-8 is log2(e) to 48 bits)
  w.hi = fminf(1.44269502f / t, 3.0e38f);
  w.lo = (fmaf(-w.hi, t, 1.44269502f) + 1.92596303e-8f) / t;
  if (!(fabsf(w.lo) < 1.0e30f)) w.lo = 0.f;

  // This thread's running sum of x over the CTA, and the sum of all.
  auto scan = [&](u64 x, u64& all) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const u64 y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s.part[warp] = x;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) x += all;
      all += s.part[w];
    }
    __syncthreads();
    return x;
  };
  auto target_of = [&](double share, u64 all) {  // the least sum that is over that share, all at most
    return min((u64)(share * (double)all) + 1, all);
  };
  const double share = (double)(u > 0.f ? fminf(u, 1.f) : 0.f);

  if (few) {
    if (tid == 0) s.listed = 0;
    __syncthreads();
    const float from = bound ? value_of(bound) : -INFINITY;
    for (int i = tid; i < vecs; i += kThreads) {
      union { uint4 u; T t[kVec]; } x;
      x.u = reinterpret_cast<const uint4*>(s_l)[i];
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float v = kv::to_float(x.t[e]);
        if (!(v >= from) || v == -INFINITY) continue;
        const int at = atomicAdd(&s.listed, 1);
        if (at < kList) s.top[at] = (u64)key_of(v) << 32 | (uint32_t)~(first + i * kVec + e);
      }
    }
    __syncthreads();
    tell(kListed, s.listed);
    cluster.sync();
    const int part = (int)told(kListed, 0);
    const int count = __reduce_add_sync(~0u, part);
    if (count <= kList) {  // the first CTA has them all then, and does the rest by itself
      if (rank == 0) {
        if (warp < ranks) {
          const Shared* o = cluster.map_shared_rank(&s, warp);
          const int at = __reduce_add_sync(~0u, lane < warp ? part : 0), m = __shfl_sync(~0u, part, warp);
          for (int i = lane; i < m; i += 32) s.sorted[at + i] = o->top[i];
        }
        u64* const spare = reinterpret_cast<u64*>(&s.sub);
        __syncthreads();
        u64* v = ordered(s.sorted, spare, count);
        const int most_kept = min(count, top_k);
        u64 x[2], y[2], all;
        bool in[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = 2 * tid + i;
          y[i] = at < most_kept ? v[at] : 0;
          in[i] = at < most_kept;
          x[i] = in[i] ? w.weight(value_of((uint32_t)(y[i] >> 32))) : 0;
        }
        u64 run = scan(x[0] + x[1], all) - x[0] - x[1];
        const u64 target = by_p ? max((u64)ceil((double)top_p * (double)all), (u64)1) : ~0ull;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          in[i] = in[i] && run < target && (2 * tid + i == 0 || w.exp_of(value_of((uint32_t)(y[i] >> 32))) >= min_p);
          run += x[i];
        }
        // in the vocabulary's order: the id's complement in front
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (2 * tid + i < most_kept) s.sorted[2 * tid + i] = in[i] ? y[i] << 32 | y[i] >> 32 : 0;
        v = ordered(s.sorted, spare, most_kept);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          y[i] = 2 * tid + i < most_kept ? v[2 * tid + i] : 0;
          x[i] = y[i] ? w.weight(value_of((uint32_t)y[i])) : 0;
        }
        run = scan(x[0] + x[1], all) - x[0] - x[1];
        const u64 at = target_of(share, all);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (run < at && at <= run + x[i]) {
            a.token[row] = (int32_t)~(uint32_t)(y[i] >> 32);
            if (a.prob) a.prob[row] = (float)((double)x[i] / (double)all);
          }
          run += x[i];
        }
      }
      cluster.sync();
      return;
    }
  }

  auto add = [&](uint32_t* low, uint32_t* high, int bin, u64 x) {  // 64 bits by two words: the carry goes with the high one
    const uint32_t lo = (uint32_t)x, old = atomicAdd(&low[bin], lo);
    const uint32_t hi = (uint32_t)(x >> 32) + (old + lo < old);
    if (hi) atomicAdd(&high[bin], hi);
  };
  auto clear = [&](int bins) {
    for (int b = tid; b < bins; b += kThreads) s.hist.low[b] = s.hist.high[b] = 0;
    __syncthreads();
  };
  // The cluster's sum of what was told, and that of the CTAs before this one.
  auto ranks_sum = [&](int what, u64& lower, u64& all) {
    const u64 own = told(what, 0);
    u64 x = own;
#pragma unroll
    for (int o = 1; o < kMostCluster; o *= 2) {
      const u64 y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    all = __shfl_sync(~0u, x, kMostCluster - 1);
    lower = __shfl_sync(~0u, x - own, rank);
  };
  // Sums the histogram over the cluster, a share of the bins in each CTA, and finds the bin, from the first on, in which the
  // running sum comes to `target`: s.bin, what lies before it (s.above) and in it (s.inside).  share >= 0: the target is that
  // share of the sum of all, rounded up, one at least.
  auto find = [&](int bins, u64& target, double share) {
    cluster.sync();
    // four words of each kind a thread: four CTAs' of a bin, or fewer CTAs' of two or four bins
    const int mine = bins / ranks, threads = max(1, ranks / 4), wide = max(1, 4 / ranks);
    const int from = rank * mine + tid / threads * wide;
    const bool here = tid / threads * wide < mine;
    u64 bin[4] = {0, 0, 0, 0};
    if (here) {
      uint32_t low[4], high[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = ranks >= 4 ? tid % threads * 4 + i : i % ranks, b = from + (ranks >= 4 ? 0 : i / ranks);
        const Shared* o = cluster.map_shared_rank(&s, c);
        low[i] = o->hist.low[b], high[i] = o->hist.high[b];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) bin[i] = (u64)high[i] << 32 | low[i];
      if (ranks == 2) bin[0] += bin[1], bin[1] = bin[2] + bin[3], bin[2] = bin[3] = 0;
      if (ranks >= 4) bin[0] += bin[1] + bin[2] + bin[3], bin[1] = bin[2] = bin[3] = 0;
    }
    for (int o = threads / 2; o; o >>= 1) bin[0] += __shfl_xor_sync(~0u, bin[0], o);
    if (tid % threads) bin[0] = 0;
    const u64 own = bin[0] + bin[1] + bin[2] + bin[3];
    u64 all = 0, x = scan(own, all);
    tell(kBinned, all);
    cluster.sync();
    u64 lower;
    ranks_sum(kBinned, lower, all);
    if (share >= 0.0) target = max((u64)ceil(share * (double)all), (u64)1);
    x += lower;
    if (x - own < target && target <= x) {
      u64 before = x - own;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (before < target && target <= before + bin[i])
          for (int c = 0; c < ranks; ++c) {
            Shared* o = cluster.map_shared_rank(&s, c);
            o->bin = from + i, o->above = before, o->inside = bin[i];
          }
        before += bin[i];
      }
    }
    cluster.sync();
  };

  // The border at which the running sum, from the largest logit down, of one each (mass false) or of the weights of those at
  // `least` and above comes to `target`: the key there, how many of the equal ones belong, and how many there are.  False
  // where it lies below what min_p leaves, and so moves nothing: what min_p takes is summed, but neither binned nor gathered
  // (64 rows of 151936 with top_p 0.95: 27 us with min_p 0.02, 53 without).
  const float steps = 2047.f / fminf(fmaxf((most - lowest) * (1.0f / t), 1e-6f), 32.f) / t;
  auto step_of = [&](float v) {  // falls as v grows
    return (int)(__float_as_uint(fminf((most - v) * steps, 2047.f) + 8388608.f) & (kBins - 1));
  };
  auto border = [&](bool mass, u64 target, double share, uint32_t least, u64 least_ties, uint32_t& key, u64& ties, u64& equal) -> bool {
    auto one = [&](float v) { return mass ? w.weight(v) : (u64)1; };
    clear(kBins);
    const float above_value = least ? value_of(least) : -INFINITY, least_e = fmaxf(min_p, 0x1p-45f);  // below weighs nothing
    if (mass) {
      uint32_t hi_sum = 0, lo_sum = 0, seen = 0;  // of all that `least` leaves
      u64 over = 0;                               // of those that min_p leaves too
      each2([&](float2 v) {
        float2 e = w.exp_of(v);
        if (least) e.x = v.x > above_value ? e.x : 0.f, e.y = v.y > above_value ? e.y : 0.f;
        uint32_t hi[2], lo[2];
        w.fixed(e, hi, lo);
        hi_sum += hi[0] + hi[1], lo_sum += lo[0] + lo[1], seen += 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!((i ? e.y : e.x) >= least_e)) continue;
          const u64 x = w.joined(hi[i], lo[i], 1);
          add(s.hist.low, s.hist.high, step_of(i ? v.y : v.x), x);
          over += x;
        }
      });
      u64 whole = w.joined(hi_sum, lo_sum, seen), lower;
      if (least_ties && rank == 0 && tid == 0) {
        const u64 x = least_ties * one(above_value);
        whole += x;
        if (w.exp_of(above_value) >= least_e) add(s.hist.low, s.hist.high, step_of(above_value), x), over += x;
      }
      if (min_p > 0.f) {
        scan(whole, whole), scan(over, over);
        tell(kWhole, whole), tell(kOver, over);
        cluster.sync();
        ranks_sum(kWhole, lower, whole);
        ranks_sum(kOver, lower, over);
        target = max((u64)ceil(share * (double)whole), (u64)1), share = -1.0;
        if (target > over) return false;
      }
    } else {
      each([&](float v) { atomicAdd(&s.hist.low[step_of(v)], 1u); });
    }
    find(kBins, target, share);
    const int bin = s.bin;
    u64 rest = target - s.above;
    if (tid == 0) s.listed = 0;
    __syncthreads();
    // the step's values, and some more for the roundings; all of them where the step has no end, or so high a temperature that its
    // middle is no number
    const float middle = most - (float)bin / steps;
    const float half = bin == kBins - 1 || isinf(middle) ? INFINITY : 0.51f / steps + 1e-6f * fabsf(most);
    for (int i = tid; i < vecs; i += kThreads) {
      union { uint4 u; T t[kVec]; } x;
      x.u = reinterpret_cast<const uint4*>(s_l)[i];
      bool some = false;
#pragma unroll
      for (int e = 0; e < kVec; ++e) some |= !(fabsf(kv::to_float(x.t[e]) - middle) > half);
      if (!some) continue;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float v = kv::to_float(x.t[e]);
        if (v < above_value || step_of(v) != bin) continue;
        const int at = atomicAdd(&s.listed, 1);
        if (at < kList) s.list[at] = key_of(v);
      }
    }
    __syncthreads();
    tell(kListed, s.listed);
    cluster.sync();
    const int part = (int)told(kListed, 0);
    const int count = __reduce_add_sync(~0u, part);
    if (count <= kList) {
      if (warp < ranks) {  // a warp copies a CTA's
        const Shared* o = cluster.map_shared_rank(&s, warp);
        const int at = __reduce_add_sync(~0u, lane < warp ? part : 0), m = __shfl_sync(~0u, part, warp);
        for (int i = lane; i < m; i += 32) {
          const uint32_t k = o->list[i];
          s.all.key[at + i] = k;
          s.all.weight[at + i] = one(value_of(k));
        }
      }
      for (int i = tid; i < kSubs; i += kThreads) s.sub.low[i] = s.sub.high[i] = 0;
      if (tid == 0) s.members = 0;
      cluster.sync();  // the lists are read: they are used again
      // 1024 steps within the step; of the one that the border lies in, each with each
      auto sub_of = [&](uint32_t k) { return (int)(((most - value_of(k)) * steps - ((float)bin - 0.5f)) * (float)kSubs); };
      auto sub = [&](uint32_t k) { return bin == kBins - 1 ? 0 : min(max(sub_of(k), 0), kSubs - 1); };
      for (int i = tid; i < count; i += kThreads) add(s.sub.low, s.sub.high, sub(s.all.key[i]), s.all.weight[i]);
      __syncthreads();
      u64 bins[2], all;
#pragma unroll
      for (int i = 0; i < 2; ++i) bins[i] = (u64)s.sub.high[2 * tid + i] << 32 | s.sub.low[2 * tid + i];
      const u64 x = scan(bins[0] + bins[1], all), before = x - bins[0] - bins[1];
      if (before < rest && rest <= x) {
        const bool second = before + bins[0] < rest;
        s.subbin = 2 * tid + second, s.rest = rest - before - (second ? bins[0] : 0);
      }
      __syncthreads();
      rest = s.rest;
      for (int i = tid; i < count; i += kThreads)
        if (sub(s.all.key[i]) == s.subbin) s.list[atomicAdd(&s.members, 1)] = i;
      __syncthreads();
      const int members = s.members;
      for (int i = tid; i < members; i += kThreads) {
        const uint32_t k = s.all.key[s.list[i]];
        u64 over = 0;
        uint32_t same = 0;
        for (int j = 0; j < members; ++j) {
          const uint32_t o = s.all.key[s.list[j]];
          if (o > k) over += s.all.weight[s.list[j]];
          same += o == k;
        }
        const u64 w1 = s.all.weight[s.list[i]];
        if (over < rest && rest <= over + same * w1) s.key = k, s.equal = same, s.need = (rest - over + w1 - 1) / w1;
      }
      __syncthreads();
      key = s.key, ties = s.need, equal = s.equal;
    } else {
      uint32_t prefix = 0;
      int shift = 32;
      rest = target;
      for (int bits : {11, 11, 10}) {
        shift -= bits;
        const int bins = 1 << bits;
        cluster.sync();  // nobody reads what is cleared
        clear(bins);
        for (int i = tid; i < n; i += kThreads) {
          const float v = kv::to_float(s_l[i]);
          const uint32_t k = key_of(v);
          if (k < least || (shift + bits < 32 && k >> (shift + bits) != prefix)) continue;
          const u64 x = one(v);
          if (x) add(s.hist.low, s.hist.high, bins - 1 - (k >> shift & (bins - 1)), x);
        }
        find(bins, rest, -1.0);
        rest -= s.above;
        prefix = prefix << bits | (uint32_t)(bins - 1 - s.bin);
        if (shift == 0) equal = s.inside;
        __syncthreads();
      }
      key = prefix;
      const u64 x = one(value_of(key));
      ties = (rest + x - 1) / x;
      equal /= x;
    }
    return true;
  };

  uint32_t key = 0;  // below every logit: all belong
  u64 ties = 0, equal = 0;
  if (by_k) border(false, (u64)top_k, -1.0, 0, 0, key, ties, equal);
  const bool by_mass = by_p && border(true, 0, (double)top_p, key, ties, key, ties, equal);
  const bool at_border = by_k || by_mass, some = at_border && ties < equal;  // some of the equal ones only
  if (!some) ties = ~0ull;

  // The kept weight of each warp's run of the slice; where only some of the equal ones at the border belong, these are counted
  // off from one run to the next.
  const int run = (n + 32 * kVec * warps - 1) / (32 * kVec * warps) * (32 * kVec), lo = min(n, warp * run), hi = min(n, lo + run);
  auto kept = [&](float v) -> u64 {
    const float e = w.exp_of(v);
    return e >= min_p || v == most ? w.fixed(e) : 0;
  };
  // element i of a warp's run, which ends at `end`; all lanes together
  auto weigh = [&](int i, int end, u64& seen) -> u64 {
    const float v = i < end ? kv::to_float(s_l[i]) : -INFINITY;
    const uint32_t k = i < end ? key_of(v) : 0;
    bool in = i < end && k >= key;
    if (some) {
      const unsigned m = __ballot_sync(~0u, in && k == key);
      in = in && (k > key || seen + __popc(m & ((1u << lane) - 1)) < ties);
      seen += __popc(m);
    }
    return in ? kept(v) : 0;
  };
  const float border_value = at_border ? value_of(key) : -INFINITY, inside = some ? value_of(key + 1) : border_value;
  const u64 tie_weight = some ? kept(border_value) : 0;
  // below it no logit is kept: of min_p, a little lower than its own border
  const float filter = min_p > 0.f ? fmaxf(border_value, most - t * (0.01f - logf(min_p)) - 1e-5f * fabsf(most)) : border_value;
  // This lane's share of the kept weight of 32 kVec logits from i on, those at the border left out where only some of them
  // belong, and how many these are.
  struct Parts {
    uint32_t hi = 0, lo = 0, seen = 0;
    int tied = 0;
    __device__ __forceinline__ u64 weight() const { return decltype(w)::joined(hi, lo, seen); }
  };
  auto group = [&](int i, Parts& sum) {
    union { uint4 u; T t[kVec]; } l;
    const bool here = i + lane * kVec < hi;
    if (here) l.u = *reinterpret_cast<const uint4*>(s_l + i + lane * kVec);
#pragma unroll
    for (int e = 0; e < kVec; e += 2) {
      const float2 v = here ? make_float2(kv::to_float(l.t[e]), kv::to_float(l.t[e + 1])) : make_float2(-INFINITY, -INFINITY);
      if (!__any_sync(~0u, fmaxf(v.x, v.y) >= filter)) continue;
      const float2 x = w.exp_of(v);
      uint32_t a[2], b[2];
      w.fixed(make_float2(v.x >= inside && x.x >= min_p ? x.x : 0.f, v.y >= inside && x.y >= min_p ? x.y : 0.f), a, b);
      sum.hi += a[0] + a[1], sum.lo += b[0] + b[1], sum.seen += 2;
      if (some) sum.tied += (v.x == border_value) + (v.y == border_value);
    }
  };
  auto of_ties = [&](u64 before, int count) { return before < ties ? min(ties - before, (u64)count) * tie_weight : 0; };
  Parts parts;
  for (int i = lo; i < hi; i += 32 * kVec) group(i, parts);
  u64 sum = parts.weight(), ahead = 0;
  int tied = parts.tied;
  if (some) {
    tied = __reduce_add_sync(~0u, tied);
    __syncthreads();
    if (lane == 0) ipart[warp] = tied;
    __syncthreads();
    int all = 0;
    for (int i = 0; i < warps; ++i) {
      if (i < warp) ahead += ipart[i];
      all += ipart[i];
    }
    tell(kTies, all);
    cluster.sync();
    ahead += __reduce_add_sync(~0u, lane < rank ? (int)told(kTies, 0) : 0);
    if (lane == 0) sum += of_ties(ahead, tied);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  __syncthreads();
  if (lane == 0) s.part[warp] = sum;
  __syncthreads();
  u64 lower = 0, slice = 0;
  for (int i = 0; i < warps; ++i) {
    if (i < warp) lower += s.part[i];
    slice += s.part[i];
  }
  tell(kKept, slice);
  cluster.sync();
  u64 grand, others;
  ranks_sum(kKept, others, grand);
  lower += others;
  const u64 target = target_of(share, grand);
  if (lower < target && target <= lower + sum) {
    u64 at = lower, seen = ahead;
    int i = lo;
    for (; i + 32 * kVec < hi; i += 32 * kVec) {
      Parts parts;
      group(i, parts);
      int tied = parts.tied;
      u64 x = parts.weight();
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
      tied = __reduce_add_sync(~0u, tied);
      x += of_ties(seen, tied);
      if (at + x >= target) break;
      at += x, seen += tied;
    }
    for (; i < hi; i += 32) {
      const u64 own = weigh(i + lane, hi, seen);
      if (!__ballot_sync(~0u, own != 0)) continue;
      u64 x = own;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const u64 y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
      const unsigned m = __ballot_sync(~0u, at + x >= target);
      if (m) {
        if (lane == __ffs(m) - 1) {
          a.token[row] = first + i + lane;
          if (a.prob) a.prob[row] = (float)((double)own / (double)grand);
        }
        break;
      }
      at += __shfl_sync(~0u, x, 31);
    }
  }
  cluster.sync();
}

template <typename T>
static cudaError_t launch(const Args& a0, int64_t rows, cudaStream_t st) {
  Args a = a0;
  // Slices of 4096 logits at least, and no more CTAs than the GPU takes at a time (two an SM), for much of a pass is waiting
  // for one another (64 rows of 151936, before the last steps: 4 CTAs a row 91 us, 8 104 us); more than 8 a row only where an SM has one.
  int ranks = 1;
  while (ranks < kMostCluster && a.vocab > ranks * 4096 && rows * 2 * ranks <= (ranks < kPortable ? 304 : 152)) ranks *= 2;
  while ((int64_t)ranks * kMostSlice < a.vocab) ranks *= 2;
  a.slice = ((a.vocab + ranks - 1) / ranks + 7) / 8 * 8;
  const size_t smem = sizeof(Shared) + (size_t)a.slice * sizeof(T);
  if (cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)(sizeof(Shared) + kMostSlice * sizeof(T))))
    return e;
  if (ranks > kPortable)
    if (cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
}

}  // namespace sample

int read_sample_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, sample::g_sample_status, sizeof(v)) != cudaSuccess) return -1;
  if (clear && v) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(sample::g_sample_status, &z, sizeof(z)) != cudaSuccess) return -1;
  }
  return (int)v;
}

}  // namespace kq

using namespace kq;

extern "C" int kq_sample(int dtype, const void* d_logits, int64_t row_stride, int64_t rows, int64_t vocab,
                         const float* d_temperature, const int32_t* d_top_k, const float* d_top_p, const float* d_min_p,
                         const float* d_u, int32_t* d_token, float* d_prob, void* stream) {
  clear_error();
  if (int s = check_dtype(dtype)) return s;
  if (vocab < 1 || vocab > sample::kMostVocab)
    return fail(KQ_ERR_SHAPE, "vocab = %lld (1 to %d)", (long long)vocab, sample::kMostVocab);
  if (rows < 0 || rows > 0x7fffffffll / sample::kPortable || row_stride < 0 || (rows > 1 && row_stride < vocab))
    return fail(KQ_ERR_SHAPE, "rows = %lld, row_stride = %lld", (long long)rows, (long long)row_stride);
  if (rows == 0) return KQ_OK;
  if (!d_logits || !d_u || !d_token) return fail(KQ_ERR_INVALID_ARG, "NULL pointer");
  if ((uintptr_t)d_logits % (dtype == KQ_F32 ? 4 : 2)) return fail(KQ_ERR_ALIGNMENT, "logits not aligned to their type");
  for (const void* p : {(const void*)d_temperature, (const void*)d_top_k, (const void*)d_top_p, (const void*)d_min_p,
                        (const void*)d_u, (const void*)d_token, (const void*)d_prob})
    if ((uintptr_t)p % 4) return fail(KQ_ERR_ALIGNMENT, "an array of the rows is not aligned to 4 bytes");
  sample::Args a{d_logits, row_stride, (int32_t)vocab, 0, d_temperature, d_top_k, d_top_p, d_min_p, d_u, d_token, d_prob};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  KQ_CUDA_TRY(dtype == KQ_F32   ? sample::launch<float>(a, rows, st)
              : dtype == KQ_F16 ? sample::launch<__half>(a, rows, st)
                                : sample::launch<__nv_bfloat16>(a, rows, st));
  return KQ_OK;
}
