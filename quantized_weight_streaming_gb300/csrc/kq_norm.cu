// RMS norm of rows, with the residual's addition before it, a gate after it and
// an output in Q8_0 beside the one in the activations' type.
//
//   s = x + residual;  y = s / sqrt(mean(s^2) + eps) * weight * silu(gate)
//
// Two flops a byte: memory bounds it, so a row is read once and stays in
// registers between the sum of its squares and the output.  A thread holds
// vectors of eight elements.  A row of up to 256 elements (a head) belongs to 8,
// 16 or 32 lanes, who add their squares by shuffles; a longer one to a CTA of its
// own, with one barrier.  (Packed fp32 pairs for the arithmetic, here and in the
// convolution, took longer: 42 us for 4099 rows with codes against 36, and 67 against
// 52; where each pair is unpacked from 16-bit types the moves undo what they save.)  The weight comes from L2 each time: CTAs that kept it in
// registers and walked rows with the grid's stride, with or without the next row's
// loads ahead, had fewer bytes in flight (4099 rows of 5120 bf16 with a residual,
// an output and codes: 61 and 49 us against 39 with as many vectors a thread).
//
// Measured on 4099 rows of 5120 bf16: 27.6 us with a residual and an output (168
// MB, 6.1 TB/s, 0.90 of a copy's rate), 36.3 with codes too (191 MB, 5.3 TB/s: the
// codes' arithmetic shows); one row of fp32 2.8 us, the time of a launch that loads
// twice.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kq_device.cuh"
#include "kq_gdn.cuh"
#include "kq_internal.h"
#include "kq_kv.cuh"

namespace kq {
namespace norm {

using gdn::Rows;

__device__ unsigned int g_norm_status = 0;
__device__ __forceinline__ void norm_flag(int status) { atomicOr(&g_norm_status, 1u << status); }

struct Args {
  Rows x, residual, gate, out;
  int8_t* codes;     // of Q8_0, or null
  uint16_t* scales;
  const float* weight;
  int64_t rows;
  int32_t heads, dim;
  int32_t scale_stride;
  float eps;
};

// v / d rounded half away from zero by what the quotient is and not what a division rounds it to: the estimate is moved by
// one where the exact sign of |v| - (n - 1/2) d (20 bits of product, one rounding) says so.
__device__ __noinline__ int q8_border(float v, float d, float inverse) {
  const float m = fabsf(v);
  float n = fminf(floorf(fmaf(m, inverse, 0.5f)), 128.f);
  if (fmaf(-(n - 0.5f), d, m) < 0.f) n -= 1.f;
  if (fmaf(-(n + 0.5f), d, m) >= 0.f) n += 1.f;
  const int q = (int)fminf(n, 127.f);
  return v < 0.f ? -q : q;
}

// Eight values of a block of 32, its other 24 in the three neighbouring lanes; `valid` is the same in all four.
__device__ __forceinline__ void store_q8(const Args& a, int64_t row, int vec, const float (&y)[8], bool valid) {
  uint32_t top = 0;  // of the magnitudes' patterns, which order as the numbers do, infinity and NaN above them
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
  top = max(top, __shfl_xor_sync(~0u, top, 1));
  top = max(top, __shfl_xor_sync(~0u, top, 2));
  if (!valid) return;
  __half s = __float2half_rn(__uint_as_float(top) / 127.0f);
  if (top >= 0x7F800000u || __hisinf(s)) {
    norm_flag(top >= 0x7F800000u ? KQ_ERR_NONFINITE : KQ_ERR_RANGE);
    s = __ushort_as_half(0x7E00);
  }
  const float d = __half2float(s);
  union { int8_t c[8]; uint2 u; } q;
  q.u = make_uint2(0, 0);
  if (d > 0.f) {
    const float inverse = 1.0f / d;
    float off = 0.f;
    uint32_t n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // the nearest whole number, in the low bits of 1.5 * 2^23 + it
      const float r = y[i] * inverse, w = r + 12582912.f;
      n[i] = __float_as_uint(w);
      off = fmaxf(off, fabsf(r - (w - 12582912.f)));
    }
    q.u.x = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
    q.u.y = __byte_perm(__byte_perm(n[4], n[5], 0x0040), __byte_perm(n[6], n[7], 0x0040), 0x5410);
    if (!(off < 0.4999f && __uint_as_float(top) * inverse < 127.4f)) {  // a quotient near a border between two codes, or past the last
#pragma unroll
      for (int i = 0; i < 8; ++i) q.c[i] = (int8_t)q8_border(y[i], d, inverse);
    }
  }
  *reinterpret_cast<uint2*>(a.codes + row * a.dim + 8 * vec) = q.u;
  if ((threadIdx.x & 3) == 0) {
    uint16_t* at = a.scales + row * a.scale_stride;
    at[vec / 4] = __half_as_ushort(s);
    if (8 * vec + 32 == a.dim)
      for (int i = a.dim / 32; i < a.scale_stride; ++i) at[i] = 0;
  }
}

// Where a row's elements lie.
template <typename T>
struct Row {
  const T* x;
  T* residual;
  const T* gate;
  T* out;
  __device__ __forceinline__ Row(const Args& a, int64_t row) {
    const int64_t token = a.heads == 1 ? row : (int64_t)((uint32_t)row / (uint32_t)a.heads);
    const int head = (int)(row - token * a.heads);
    x = reinterpret_cast<const T*>(a.x.at(token, head)), residual = reinterpret_cast<T*>(a.residual.at(token, head));
    gate = reinterpret_cast<const T*>(a.gate.at(token, head)), out = reinterpret_cast<T*>(a.out.at(token, head));
  }
};

// x + residual rounded to the type, which goes back to the residual; and the squares' sum.
template <typename T>
__device__ __forceinline__ float sum_squares(const Args& a, const Row<T>& r, int vec, bool mine, kv::Raw<T, 8>& x,
                                             const kv::Raw<T, 8>& residual, float (&v)[8], float sum) {
  x.get(v);
  if (a.residual.data) {
    float other[8];
    residual.get(other);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += other[e];
    x.set(v);
    if (mine) x.store(r.residual + 8 * vec);
    x.get(v);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
  return sum;
}

template <typename T>
__device__ __forceinline__ void finish(const Args& a, const Row<T>& r, int64_t row, int vec, bool mine, float f, const float (&w)[8],
                                       kv::Raw<T, 8>& gate, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = v[e] * f * w[e];
  if (a.gate.data) {
    float z[8];
    if (a.residual.data && mine) gate.load(r.gate + 8 * vec);
    gate.get(z);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= gdn::silu<T>(z[e]);
  }
  if (a.codes) store_q8(a, row, vec, v, mine);
  if (a.out.data && mine) kv::store8(r.out + 8 * vec, v);
}

// Rows of up to 8 LANES elements, N of them a group of lanes.
template <typename T, int LANES, int N>
__global__ void __launch_bounds__(256) rms_heads_kernel(const Args a) {
  constexpr int kRows = 256 / LANES;  // that a CTA takes N times
  const int vec = threadIdx.x % LANES;
  const bool in = 8 * vec < a.dim;
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t row0 = (int64_t)blockIdx.x * kRows * N + threadIdx.x / LANES;
  kv::Raw<T, 8> raw[N], other[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t row = row0 + i * kRows;
    raw[i].clear();
    other[i].clear();
    if (!in || row >= a.rows) continue;
    const Row<T> r(a, row);
    raw[i].load(r.x + 8 * vec);
    if (a.residual.data) other[i].load(r.residual + 8 * vec);
    else if (a.gate.data) other[i].load(r.gate + 8 * vec);
  }
  float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  if (a.weight && in) kv::load8(a.weight + 8 * vec, w);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t row = row0 + i * kRows;
    const bool mine = in && row < a.rows;
    const Row<T> r(a, row);
    float v[8], sum = sum_squares(a, r, vec, mine, raw[i], other[i], v, 0.f);
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    finish(a, r, row, vec, mine, 1.0f / sqrtf(sum / (float)a.dim + a.eps), w, other[i], v);
  }
}

// A row a CTA, N vectors a thread.
template <typename T, int N>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const Args a) {
  __shared__ float s_part[32];
  const int step = blockDim.x, vecs = a.dim / 8;
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t row = blockIdx.x;
  const Row<T> r(a, row);
  kv::Raw<T, 8> raw[N], other[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int vec = threadIdx.x + i * step;
    raw[i].clear();
    other[i].clear();
    if (vec >= vecs) continue;
    raw[i].load(r.x + 8 * vec);
    if (a.residual.data) other[i].load(r.residual + 8 * vec);
    else if (a.gate.data) other[i].load(r.gate + 8 * vec);
  }
  float v[N][8], sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int vec = threadIdx.x + i * step;
    sum = sum_squares(a, r, vec, vec < vecs, raw[i], other[i], v[i], sum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (threadIdx.x % 32 == 0) s_part[threadIdx.x / 32] = sum;
  __syncthreads();
  sum = 0.f;
  const int warps = blockDim.x / 32;
  if (threadIdx.x % 32 < warps) sum = s_part[threadIdx.x % 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  const float f = 1.0f / sqrtf(sum / (float)a.dim + a.eps);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int vec = threadIdx.x + i * step;
    float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (a.weight && vec < vecs) kv::load8(a.weight + 8 * vec, w);
    finish(a, r, row, vec, vec < vecs, f, w, other[i], v[i]);
  }
}

template <typename T, int N>
static cudaError_t launch(const Args& a, cudaStream_t st) {
  const int threads = (a.dim / 8 + 32 * N - 1) / (32 * N) * 32;
  return launch_dependent(rms_norm_kernel<T, N>, dim3((unsigned)a.rows), dim3(threads), 0, st, a);
}
template <typename T, int LANES>
static cudaError_t launch_heads(const Args& a, cudaStream_t st) {
  // Beyond two waves of CTAs a group takes two rows, for twice the loads in flight and half the CTAs' starts (gated f16 heads of
  // 128 with 1, 2, 4 rows a group: 12288 3.9, 4.4, 4.9 us; 49152 10.6, 9.9, 10.8; 196608 43, 36, 37).
  const int64_t ctas = (a.rows + 256 / LANES - 1) / (256 / LANES);
  if (ctas <= 2 * 152 * 8) return launch_dependent(rms_heads_kernel<T, LANES, 1>, dim3((unsigned)ctas), dim3(256), 0, st, a);
  return launch_dependent(rms_heads_kernel<T, LANES, 2>, dim3((unsigned)((ctas + 1) / 2)), dim3(256), 0, st, a);
}

template <typename T>
static cudaError_t launch_norm(const Args& a, cudaStream_t st) {
  const int vecs = a.dim / 8;
  if (vecs <= 8) return launch_heads<T, 8>(a, st);
  if (vecs <= 16) return launch_heads<T, 16>(a, st);
  if (vecs <= 32) return launch_heads<T, 32>(a, st);
  // Few rows, of up to a wave of CTAs, want many threads (one row of 5120 bf16 with a residual: 2.0, 2.3, 3.1 us with 1, 2, 4
  // vectors a thread; 304 rows 4.2, 4.7, 5.1).  Many want fewer that have more in flight each (4096 rows of 5120: 36, 30, 28 us;
  // of 8192: 71, 47, 42), but for short ones (8192 rows of 2048: 26, 22, 23) and fp32, whose four vectors are more than a
  // thread's 64 registers hold (240 bytes spill: 4096 rows of 5120: 54, 51, 61; in 16-bit types 48 bytes do).
  if (vecs <= 1024 && a.rows <= 304) return launch<T, 1>(a, st);
  if (vecs <= (a.rows <= 304 || sizeof(T) == 4 ? 2048 : 512)) return launch<T, 2>(a, st);
  return launch<T, 4>(a, st);
}

}  // namespace norm

int check_out_rows(const kq_heads* h, const char* name, int dtype, int64_t tokens, int heads, int dim) {
  if (int s = check_heads(h, name, dtype)) return s;
  // the rows along the smaller stride lie apart, and those along the larger one past all of them
  const bool by_head = tokens <= 1 || (heads > 1 && h->head_stride <= h->token_stride);
  const int64_t near = by_head ? h->head_stride : h->token_stride, far = by_head ? h->token_stride : h->head_stride;
  const int64_t near_rows = by_head ? heads : tokens, far_rows = by_head ? tokens : heads;
  if ((near_rows > 1 && near < dim) || (far_rows > 1 && (far < dim || (far - dim) / std::max<int64_t>(near, 1) < near_rows - 1)))
    return fail(KQ_ERR_SHAPE, "rows of %s overlap", name);
  return KQ_OK;
}

namespace {
// Rows in bytes: `heads` blocks a token, each `wide` (neighbouring rows are one block).
struct Blocks {
  int64_t tokens, token_stride, heads, head_stride, wide;
  __int128 extent() const { return (__int128)(tokens - 1) * token_stride + (__int128)(heads - 1) * head_stride + wide; }
};
Blocks blocks_of(const kq_heads* h, int64_t tokens, int heads, int dim, int size) {
  Blocks b{tokens, h->token_stride * size, heads, h->head_stride * size, (int64_t)dim * size};
  if (b.head_stride == 0) b.heads = 1;
  if (b.token_stride == 0) b.tokens = 1;
  for (int turn = 0; turn < 2; ++turn) {
    if (b.heads > 1 && b.head_stride == b.wide) b.wide *= b.heads, b.heads = 1;
    if (b.tokens > 1 && b.token_stride == b.wide) b.wide *= b.tokens, b.tokens = 1;
  }
  return b;
}
}  // namespace

bool same_view(const kq_heads* x, const kq_heads* y, int64_t tokens, int heads) {
  return x->data == y->data && (tokens <= 1 || x->token_stride == y->token_stride) && (heads <= 1 || x->head_stride == y->head_stride);
}

bool rows_overlap(const kq_heads* x, int x_heads, const kq_heads* y, int y_heads, int64_t tokens, int dim, int dtype) {
  const int size = dtype == KQ_F32 ? 4 : 2;
  const int64_t apart = static_cast<const char*>(y->data) - static_cast<const char*>(x->data);
  const Blocks a = blocks_of(x, tokens, x_heads, dim, size), b = blocks_of(y, tokens, y_heads, dim, size);
  if (apart >= a.extent() || -(__int128)apart >= b.extent()) return false;
  const int64_t stride = b.tokens > 1 ? b.token_stride : a.token_stride;
  if (a.tokens > 1 && b.tokens > 1 && a.token_stride != b.token_stride) return false;
  if (a.heads * b.heads > 4096) return false;
  for (int64_t i = 0; i < a.heads; ++i)
    for (int64_t j = 0; j < b.heads; ++j) {
      // b's block of token n + k begins at off + k * stride from a's of token n: the first k whose ends behind that one's begin
      const __int128 off = (__int128)apart + (__int128)j * b.head_stride - (__int128)i * a.head_stride, least = -(__int128)b.wide + 1;
      __int128 k = -(a.tokens - 1);
      if (stride > 0 && least - off > k * stride) k = (least - off) / stride + ((least - off) % stride > 0);
      if (k <= b.tokens - 1 && off + k * stride >= least && off + k * stride < a.wide) return true;
    }
  return false;
}

int read_norm_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, norm::g_norm_status, sizeof(v)) != cudaSuccess) return -1;
  if (clear && v) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(norm::g_norm_status, &z, sizeof(z)) != cudaSuccess) return -1;
  }
  return (int)v;
}

}  // namespace kq

using namespace kq;

extern "C" int kq_rms_norm(const kq_rms* p, int dtype, const kq_heads* x, const kq_heads* residual,
                           const kq_heads* gate, int64_t tokens, const kq_heads* out, const kq_qmat* out_q8,
                           void* stream) {
  clear_error();
  if (int s = check_dtype(dtype)) return s;
  if (!p) return fail(KQ_ERR_INVALID_ARG, "p is NULL");
  if (p->reserved != 0) return fail(KQ_ERR_INVALID_ARG, "reserved is not 0");
  if (p->heads < 1 || p->heads > 4096 || p->dim < 8 || p->dim % 8 || p->dim > 32768)
    return fail(KQ_ERR_SHAPE, "%d heads of %d (1 to 4096, a multiple of 8 up to 32768)", p->heads, p->dim);
  if (!(p->eps >= 0.f && std::isfinite(p->eps))) return fail(KQ_ERR_INVALID_ARG, "eps is negative or not finite");
  if (p->weight && !aligned16(p->weight)) return fail(KQ_ERR_ALIGNMENT, "weight not 16-byte aligned");
  if (tokens < 0 || tokens > 0x7fffffffll / p->heads) return fail(KQ_ERR_SHAPE, "tokens = %lld", (long long)tokens);
  if (tokens == 0) return KQ_OK;
  if (!out && !out_q8) return fail(KQ_ERR_INVALID_ARG, "neither out nor out_q8");
  if (int s = check_heads(x, "x", dtype)) return s;
  if (residual)
    if (int s = check_out_rows(residual, "residual", dtype, tokens, p->heads, p->dim)) return s;
  if (gate)
    if (int s = check_heads(gate, "gate", dtype)) return s;
  if (out)
    if (int s = check_out_rows(out, "out", dtype, tokens, p->heads, p->dim)) return s;
  for (const kq_heads* from : {x, residual, gate})
    if (from && out && !same_view(from, out, tokens, p->heads) && rows_overlap(from, p->heads, out, p->heads, tokens, p->dim, dtype))
      return fail(KQ_ERR_INVALID_ARG, "out overlaps an input without being its view");
  if (residual && !same_view(x, residual, tokens, p->heads) && rows_overlap(x, p->heads, residual, p->heads, tokens, p->dim, dtype))
    return fail(KQ_ERR_INVALID_ARG, "residual overlaps x");
  if (residual && gate && rows_overlap(gate, p->heads, residual, p->heads, tokens, p->dim, dtype))
    return fail(KQ_ERR_INVALID_ARG, "residual overlaps gate");
  norm::Args a{};
  if (out_q8) {
    if (int s = check_qmat(out_q8, KQ_Q8_0)) return s;
    if (out_q8->n != tokens * p->heads || out_q8->k != p->dim)
      return fail(KQ_ERR_SHAPE, "out_q8 is %lld x %lld, %lld rows of %d are written", (long long)out_q8->n,
                  (long long)out_q8->k, (long long)(tokens * p->heads), p->dim);
    a.codes = static_cast<int8_t*>(const_cast<void*>(static_cast<const void*>(out_q8->codes)));
    a.scales = static_cast<uint16_t*>(const_cast<void*>(static_cast<const void*>(out_q8->scales)));
    a.scale_stride = (int32_t)scale_stride(KQ_Q8_0, p->dim);
  }
  const int size = dtype == KQ_F32 ? 4 : 2;
  a.x = gdn::rows_of(x, size), a.residual = gdn::rows_of(residual, size), a.gate = gdn::rows_of(gate, size);
  a.out = gdn::rows_of(out, size);
  a.weight = p->weight, a.rows = tokens * p->heads, a.heads = p->heads, a.dim = p->dim, a.eps = p->eps;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  KQ_CUDA_TRY(dtype == KQ_F32   ? norm::launch_norm<float>(a, st)
              : dtype == KQ_F16 ? norm::launch_norm<__half>(a, st)
                                : norm::launch_norm<__nv_bfloat16>(a, st));
  return KQ_OK;
}
