// Attention of a step's new tokens over the paged 4-bit cache.
//
// A first, plain kernel: one CTA per (token, query head), one key per thread
// for the scores of a chunk of keys, one or two dimensions per thread for the
// values, running maximum and sum in between (one pass over the cache).
#include <cuda_runtime.h>

#include <cmath>

#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_kv.cuh"

namespace kq {
namespace attn {

using kv::Cache;
using kv::kGranule;
using kv::Layout;

__device__ unsigned int g_attn_status = 0;
__device__ __forceinline__ void attn_flag(int status) { atomicOr(&g_attn_status, 1u << status); }

struct Args {
  Cache cache;
  const void* q;
  void* out;
  int64_t q_token, q_head, out_token, out_head;
  const int32_t *q_start, *kv_len, *table;
  int64_t table_stride, requests, tokens, max_new, window;
  int32_t q_heads;
  float scale;
};

constexpr int kThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_plain_kernel(Args a) {
  using L = Layout<D>;
  __shared__ float s_q[D], s_p[kThreads], s_red[kThreads / 32];
  __shared__ int64_t s_base[kThreads];
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x / a.q_heads;
  const int h = (int)(blockIdx.x % a.q_heads), hk = h / (a.q_heads / a.cache.kv_heads);
  int64_t l = 0, r = a.requests;  // the last request that starts at or before t
  while (r - l > 1) {
    const int64_t m = (l + r) / 2;
    if (a.q_start[m] <= t) l = m; else r = m;
  }
  const int32_t first = a.q_start[l], end = a.q_start[l + 1];
  if (t < first || t >= end) return;
  if (end > a.tokens || end - first > a.max_new) {
    if (tid == 0) attn_flag(KQ_ERR_RANGE);
    if (t - first >= a.max_new) return;
  }
  int64_t len = a.kv_len[l];
  const int64_t pos = len - (end - first) + (t - first);
  if (len > a.table_stride * a.cache.page_size) {
    if (tid == 0) attn_flag(KQ_ERR_RANGE);
    len = a.table_stride * a.cache.page_size;
  }
  const int64_t hi = min(pos + 1, len), lo = a.window ? max((int64_t)0, pos - a.window + 1) : 0;
  for (int i = tid; i < D; i += kThreads)
    s_q[i] = kv::to_float(static_cast<const T*>(a.q)[t * a.q_token + h * a.q_head + i]);
  __syncthreads();
  float m = -INFINITY, sum = 0.f, acc[(D + kThreads - 1) / kThreads] = {};
  for (int64_t base = lo; base < hi; base += kThreads) {
    const int64_t j = base + tid;
    float s = -INFINITY;
    int64_t at = -1;
    if (j < hi) {
      const int32_t page = a.table[l * a.table_stride + j / a.cache.page_size];
      if (page < 0 || page >= a.cache.pages) {
        attn_flag(KQ_ERR_RANGE);
      } else {
        const int in_page = (int)(j % a.cache.page_size), tok = in_page % kGranule;
        at = ((int64_t)page * a.cache.kv_heads + hk) * a.cache.block_bytes + (in_page / kGranule) * L::kBytes;
        const uint8_t* g = a.cache.data + at;
        s = 0.f;
        for (int w = 0; w < D / 8; ++w) {
          const uint32_t c = *reinterpret_cast<const uint32_t*>(g + L::key_word(tok, w));
          const float d = __half2float(*reinterpret_cast<const __half*>(g + L::key_scale(tok, w / 4)));
          float x = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) x = fmaf((float)((int)(c >> (4 * i) & 15u) - 8), s_q[8 * w + i], x);
          s = fmaf(x, d, s);
        }
        s *= a.scale;
      }
    }
    s_base[tid] = at;
    float top = s;
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (tid % 32 == 0) s_red[tid / 32] = top;
    __syncthreads();
    for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, s_red[i]);
    const float now = fmaxf(m, top), keep = m == -INFINITY ? 0.f : __expf(m - now);
    s_p[tid] = at < 0 ? 0.f : __expf(s - now);
    m = now;
    __syncthreads();
    sum *= keep;
    for (int i = 0; i < kThreads; ++i) sum += s_p[i];
#pragma unroll
    for (int k = 0; k < (D + kThreads - 1) / kThreads; ++k) {
      const int e = tid + k * kThreads;
      if (e >= D) continue;
      float o = acc[k] * keep;
      for (int i = 0; i < kThreads; ++i) {
        if (s_base[i] < 0) continue;
        const uint8_t* g = a.cache.data + s_base[i];
        const int tok = (int)((base + i) % a.cache.page_size % kGranule);
        const uint32_t c = *reinterpret_cast<const uint16_t*>(g + L::value_unit(tok, e / 4));
        const float d = __half2float(*reinterpret_cast<const __half*>(g + L::key_scale(tok, e / 32) + D));
        o = fmaf(s_p[i] * d, (float)((int)(c >> (4 * (e % 4)) & 15u) - 8), o);
      }
      acc[k] = o;
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < (D + kThreads - 1) / kThreads; ++k) {
    const int e = tid + k * kThreads;
    if (e < D)
      static_cast<T*>(a.out)[t * a.out_token + h * a.out_head + e] = kv::from_float<T>(sum == 0.f ? 0.f : acc[k] / sum);
  }
}

template <typename T>
static cudaError_t launch(int d, const Args& a, cudaStream_t st) {
  const dim3 grid((unsigned)(a.tokens * a.q_heads));
  auto k = d == 64 ? attn_plain_kernel<T, 64> : (d == 128 ? attn_plain_kernel<T, 128> : attn_plain_kernel<T, 256>);
  return launch_dependent(k, grid, dim3(kThreads), 0, st, a);
}

}  // namespace attn

int read_attn_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, attn::g_attn_status, sizeof(v)) != cudaSuccess) return -1;
  if (clear && v) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(attn::g_attn_status, &z, sizeof(z)) != cudaSuccess) return -1;
  }
  return (int)v;
}

}  // namespace kq

using namespace kq;

static int check_attn(const kq_kv_cache* cache, int32_t q_heads, int64_t requests, int64_t tokens, int64_t max_new) {
  if (int s = check_cache(cache)) return s;
  if (q_heads < 1 || q_heads % cache->kv_heads)
    return fail(KQ_ERR_SHAPE, "q_heads = %d is not a positive multiple of %d key heads", q_heads, cache->kv_heads);
  if (requests < 1 || requests > 0x7fffffffll || tokens < 0 || max_new < 1 || q_heads > 4096 ||
      tokens > 0x7fffffffll / 8192)
    return fail(KQ_ERR_SHAPE, "requests = %lld, tokens = %lld, max_new = %lld, q_heads = %d", (long long)requests,
                (long long)tokens, (long long)max_new, q_heads);
  return KQ_OK;
}

extern "C" {

size_t kq_attn_workspace_bytes(const kq_kv_cache* cache, int32_t q_heads, int64_t requests, int64_t tokens,
                               int64_t max_new) {
  clear_error();
  if (check_attn(cache, q_heads, requests, tokens, max_new)) return 0;
  return 0;
}

int kq_attn_paged(const kq_kv_cache* cache, int dtype, int32_t q_heads, const kq_heads* q, const int32_t* d_q_start,
                  const int32_t* d_kv_len, const int32_t* d_block_table, int64_t table_stride, int64_t requests,
                  int64_t tokens, int64_t max_new, float scale, int64_t window, const kq_heads* out, void* d_ws,
                  size_t ws_bytes, void* stream) {
  clear_error();
  if (dtype != KQ_F32 && dtype != KQ_F16 && dtype != KQ_BF16) return fail(KQ_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (int s = check_attn(cache, q_heads, requests, tokens, max_new)) return s;
  if (!d_q_start || !d_kv_len || !d_block_table) return fail(KQ_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned16(d_q_start) || !aligned16(d_kv_len) || !aligned16(d_block_table))
    return fail(KQ_ERR_ALIGNMENT, "q_start, kv_len or block table not 16-byte aligned");
  if (table_stride < 1 || window < 0)
    return fail(KQ_ERR_SHAPE, "table_stride = %lld, window = %lld", (long long)table_stride, (long long)window);
  if (!std::isfinite(scale)) return fail(KQ_ERR_INVALID_ARG, "scale is not finite");
  if (tokens == 0) return KQ_OK;
  if (int s = check_heads(q, "q", dtype)) return s;
  if (int s = check_heads(out, "out", dtype)) return s;
  const size_t need = kq_attn_workspace_bytes(cache, q_heads, requests, tokens, max_new);
  if (need && (!d_ws || ws_bytes < need))
    return fail(KQ_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", d_ws ? ws_bytes : (size_t)0, need);
  if (d_ws && !aligned16(d_ws)) return fail(KQ_ERR_ALIGNMENT, "workspace not 16-byte aligned");
  attn::Args a{};
  a.cache = cache_view(cache);
  a.q = q->data, a.q_token = q->token_stride, a.q_head = q->head_stride;
  a.out = out->data, a.out_token = out->token_stride, a.out_head = out->head_stride;
  a.q_start = d_q_start, a.kv_len = d_kv_len, a.table = d_block_table;
  a.table_stride = table_stride, a.requests = requests, a.tokens = tokens, a.max_new = max_new, a.window = window;
  a.q_heads = q_heads, a.scale = scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  KQ_CUDA_TRY(dtype == KQ_F32 ? attn::launch<float>(cache->head_dim, a, st)
                              : (dtype == KQ_F16 ? attn::launch<__half>(cache->head_dim, a, st)
                                                 : attn::launch<__nv_bfloat16>(cache->head_dim, a, st)));
  return KQ_OK;
}

}  // extern "C"
