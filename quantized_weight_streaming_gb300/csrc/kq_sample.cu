// Sampling: one token from each row of logits, by temperature, top-k, top-p,
// min-p and a given random number.
//
// The kept tokens are those above a border: a logit K, and how many of the equal
// ones at it (the lowest ids) still belong.  Top-k looks for the border by counts,
// top-p by masses; neither sorts.  A row's logits are read once and stay in the
// shared memory of a cluster of CTAs, a slice each; a border is found by
// histograms over ever finer parts of the value range, summed over the cluster.
// The token then is the first id, in the vocabulary's order, where the running sum
// of the kept weights passes u times their sum.
//
// A weight is exp((l - max) / temperature) in fixed point, 44 bits behind the
// point, and sums are of 64-bit integers: a row of 2^18 equal ones still fits, sums
// are exact, and no order of atomics or CTAs moves a border or a token.
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
constexpr int kMostCluster = 8;
constexpr int kMostSlice = kMostVocab / kMostCluster;
constexpr int kMostThreads = 1024, kMostWarps = kMostThreads / 32;
constexpr int kBins = 2048;
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

// What the CTAs of a cluster show one another.
struct Shared {
  u64 hist[kBins];
  u64 total[kBins];     // the cluster's sums, the same in every CTA
  u64 part[kMostWarps];
  u64 kept;             // this slice's kept weight
  float most;
  int32_t nan, ties, lowest;
  int32_t bin;
  u64 above;
  u64 found;
};

__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

struct Row {
  float most;         // the largest logit
  float hi, lo;       // log2(e) / temperature in two floats
  bool infinite;      // the largest is infinity: those alone weigh, one each
  // exp((v - most) / temperature): the difference and its product with the factor are kept to twice fp32's bits, so the
  // error is that of exp2f alone however large the argument is.
  __device__ __forceinline__ float exp_of(float v) const {
    if (infinite) return v == most ? 1.f : 0.f;
    const float d = v - most, b = d - v, err = (v - (d - b)) - (most + b);  // v - most = d + err exactly
    const float p = d * hi;
    if (!(p > -160.f)) return 0.f;
    const float rest = fmaf(d, hi, -p) + fmaf(d, lo, err * hi);
    return exp2f(p) * fmaf(rest, 0.69314718f, 1.f);
  }
  __device__ __forceinline__ u64 weight(float v) const { return (u64)__float2ull_rn(exp_of(v) * kOne); }
};

template <typename V, typename F>
__device__ __forceinline__ V block_reduce(V v, V* part, F join, V none) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = join(v, __shfl_xor_sync(~0u, v, o));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  __syncthreads();
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : none;
#pragma unroll
  for (int o = 16; o; o >>= 1) v = join(v, __shfl_xor_sync(~0u, v, o));
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kMostThreads) sample_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  Shared& s = *reinterpret_cast<Shared*>(s_raw);
  T* s_l = reinterpret_cast<T*>(s_raw + sizeof(Shared));
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int64_t row = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, warps = blockDim.x / 32;
  const int first = rank * a.slice, n = max(0, min(a.slice, a.vocab - first));
  grid_dependency_wait();
  allow_dependent_launch();

  // the slice, its largest
  const T* src = static_cast<const T*>(a.logits) + row * a.row_stride + first;
  float most = -INFINITY;
  int nan = 0;
  auto see = [&](T x) {
    const float v = kv::to_float(x);
    most = fmaxf(most, v);
    nan |= isnan(v);
  };
  constexpr int kVec = 16 / sizeof(T);
  if (((uintptr_t)src & 15) == 0) {
    for (int i = tid; i < n / kVec; i += blockDim.x) {
      union { uint4 u; T t[kVec]; } x;
      x.u = __ldg(reinterpret_cast<const uint4*>(src) + i);
      reinterpret_cast<uint4*>(s_l)[i] = x.u;
#pragma unroll
      for (int e = 0; e < kVec; ++e) see(x.t[e]);
    }
    for (int i = n / kVec * kVec + tid; i < n; i += blockDim.x) see(s_l[i] = src[i]);
  } else {
    for (int i = tid; i < n; i += blockDim.x) see(s_l[i] = src[i]);
  }
  float* fpart = reinterpret_cast<float*>(s.part);
  int* ipart = reinterpret_cast<int*>(s.part);
  most = block_reduce(most, fpart, [](float x, float y) { return fmaxf(x, y); }, -INFINITY);
  nan = __syncthreads_or(nan);
  if (tid == 0) s.most = most, s.nan = nan;
  cluster.sync();
  for (int c = 0; c < ranks; ++c) {
    const Shared* o = cluster.map_shared_rank(&s, c);
    most = fmaxf(most, o->most);
    nan |= o->nan;
  }

  const float t = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
  const float min_p = a.min_p ? a.min_p[row] : 0.f;
  const int32_t top_k = a.top_k ? a.top_k[row] : 0;
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

  Row w;
  w.most = most;
  w.infinite = isinf(most);
  if (t == 0.f || top_k == 1 || top_p <= 0.f || min_p > 1.f) {  // the largest alone, its lowest id
    int at = 0x7fffffff;
    for (int i = tid; i < n; i += blockDim.x)
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
  const double factor = 1.4426950408889634 / (double)t;
  w.hi = (float)fmin(factor, 3.0e38);
  w.lo = (float)fmin(factor - (double)w.hi, 1.0e30);

  // Sums s.hist over the cluster and finds, from the highest of `bins` bins down, the one in which the running sum comes
  // to `target`; `above` gets what lies over it.
  auto find = [&](int bins, u64 target, u64 above, int& bin, u64& over) {
    cluster.sync();
    for (int b = tid; b < bins; b += blockDim.x) {
      u64 sum = 0;
      for (int c = 0; c < ranks; ++c) sum += cluster.map_shared_rank(&s, c)->hist[b];
      s.total[b] = sum;
    }
    __syncthreads();
    if (warp == 0) {  // 32 bins at a time, the highest first
      u64 run = above;
      int hit = -1;
      for (int b0 = bins - 32; b0 >= 0; b0 -= 32) {
        u64 x = s.total[b0 + 31 - lane];
        const u64 own = x;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const u64 y = __shfl_up_sync(~0u, x, o);
          if (lane >= o) x += y;
        }
        const unsigned m = __ballot_sync(~0u, run + x >= target);
        if (m) {
          const int l = __ffs(m) - 1;
          hit = b0 + 31 - l;
          run += __shfl_sync(~0u, x - own, l);
          break;
        }
        run += __shfl_sync(~0u, x, 31);
      }
      if (lane == 0) s.bin = hit, s.above = run;
    }
    cluster.sync();
    bin = s.bin;
    over = s.above;
  };

  // The border at which the running sum, from the largest logit down, of one each (MASS false) or of the weights comes to
  // `target`: the key there, and how many of the equal ones belong.
  auto border = [&](bool mass, u64 target, uint32_t& key, u64& ties, u64& over) {
    uint32_t prefix = 0;
    over = 0;
    int shift = 32;
    for (int bits : {11, 11, 10}) {
      shift -= bits;
      const int bins = 1 << bits;
      for (int b = tid; b < bins; b += blockDim.x) s.hist[b] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += blockDim.x) {
        const float v = kv::to_float(s_l[i]);
        const uint32_t k = key_of(v);
        if (shift + bits < 32 && k >> (shift + bits) != prefix) continue;
        const u64 x = mass ? w.weight(v) : 1;
        if (x) atomicAdd(&s.hist[k >> shift & (bins - 1)], x);
      }
      int bin;
      u64 now;
      find(bins, target, over, bin, now);
      over = now;
      prefix = prefix << bits | (uint32_t)bin;
    }
    key = prefix;
    const u64 one = mass ? w.weight(value_of(key)) : 1;
    ties = (target - over + one - 1) / one;
  };

  uint32_t key = 0;  // below every logit: all belong
  u64 ties = ~0ull, over = 0, total = 0;
  const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.f;
  if (by_k) border(false, (u64)top_k, key, ties, over);
  auto kept_mass = [&]() {  // of all that belong so far
    u64 sum = 0;
    for (int i = tid; i < n; i += blockDim.x) {
      const float v = kv::to_float(s_l[i]);
      if (key_of(v) > key) sum += w.weight(v);
    }
    sum = block_reduce(sum, s.part, [](u64 x, u64 y) { return x + y; }, (u64)0);
    if (tid == 0) s.kept = sum;
    cluster.sync();
    sum = 0;
    for (int c = 0; c < ranks; ++c) sum += cluster.map_shared_rank(&s, c)->kept;
    cluster.sync();
    return by_k ? sum + ties * w.weight(value_of(key)) : sum;
  };
  if (by_p) {
    total = kept_mass();
    const u64 target = (u64)ceil((double)top_p * (double)total);
    border(true, max(target, (u64)1), key, ties, over);
  }

  // The kept weight of each warp's run of the slice; equal ones at the border are counted off in order.
  const int run = (n + 32 * warps - 1) / (32 * warps) * 32, lo = min(n, warp * run), hi = min(n, lo + run);
  const bool at_border = by_k || by_p;
  int mine = 0;
  if (at_border)
    for (int i = lo; i < hi; i += 32) {
      const bool tie = i + lane < hi && key_of(kv::to_float(s_l[i + lane])) == key;
      mine += __popc(__ballot_sync(~0u, tie));
    }
  __syncthreads();
  if (lane == 0) ipart[warp] = mine;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < warps; ++i) {
    if (i < warp) before += ipart[i];
    all += ipart[i];
  }
  if (tid == 0) s.ties = all;
  cluster.sync();
  u64 ahead = before;
  for (int c = 0; c < rank; ++c) ahead += cluster.map_shared_rank(&s, c)->ties;
  auto weigh = [&](int i, u64& seen) -> u64 {  // element i of the warp's run, all lanes together
    const bool here = i < hi;
    const float v = here ? kv::to_float(s_l[i]) : -INFINITY;
    const uint32_t k = key_of(v);
    const unsigned m = __ballot_sync(~0u, here && at_border && k == key);
    const bool in = here && (!at_border || k > key || (k == key && seen + __popc(m & ((1u << lane) - 1)) < ties));
    seen += __popc(m);
    if (!in) return 0;
    const float e = w.exp_of(v);
    return e >= min_p || v == most ? (u64)__float2ull_rn(e * kOne) : 0;
  };
  u64 sum = 0, seen = ahead;
  for (int i = lo; i < hi; i += 32) sum += weigh(i + lane, seen);
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
  if (tid == 0) s.kept = slice;
  cluster.sync();
  u64 grand = 0;
  for (int c = 0; c < ranks; ++c) {
    const u64 x = cluster.map_shared_rank(&s, c)->kept;
    if (c < rank) lower += x;
    grand += x;
  }
  const float u = a.u[row];
  const double part = (double)(u > 0.f ? fminf(u, 1.f) : 0.f) * (double)grand;
  // the first whose running sum is over `part`; u = 1, or a product that rounds up to all, takes the last
  const u64 target = min((u64)part + 1, grand);
  if (lower < target && target <= lower + sum) {
    seen = ahead;
    u64 at = lower;
    for (int i = lo; i < hi; i += 32) {
      const u64 own = weigh(i + lane, seen);
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
  int ranks = 1;
  while (ranks < kMostCluster && a.vocab > ranks * 4096) ranks *= 2;
  a.slice = ((a.vocab + ranks - 1) / ranks + 7) / 8 * 8;
  const size_t smem = sizeof(Shared) + (size_t)a.slice * sizeof(T);
  if (cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)(sizeof(Shared) + kMostSlice * sizeof(T))))
    return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * ranks));
  cfg.blockDim = dim3(kMostThreads);
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
  if (rows < 0 || rows > 0x7fffffffll / sample::kMostCluster || row_stride < 0 || (rows > 1 && row_stride < vocab))
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
