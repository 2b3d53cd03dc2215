// The gated delta rule over prompts, in chunks of 64 tokens, on the 5th-generation
// tensor cores.
//
// Within a chunk, with G_i the product of the decays up to token i and k, q unit
// rows, the updates u of all tokens solve one triangular system:
//
//   U = T R,  R_i = beta_i (v_i - G_i S^T k_i),  T = (1 + L)^-1,
//   L_ij = beta_i (G_i / G_j) k_i . k_j  for j < i
//   O_i = G_i S^T q_i + (X R)_i,  X = P T,  P_ij = (G_i / G_j) q_i . k_j  for j <= i
//   S <- G_64 S + sum_j (G_64 / G_j) k_j u_j^T
//
// Token by token a state's 128 x 128 numbers take part in two products and a sum
// each: 8192 tokens of 48 heads took 4931 us so, bound by a token's two passes over
// the registers and its barrier.  In chunks the same work is matrix products.  T and X do not depend on the
// state: gdn_rows_kernel lays out each key head's rows, gdn_chunk_kernel makes T and X
// for all chunks, and gdn_prompt_kernel walks down each request's chunks, a CTA a
// head, with its state in registers.
//
// The states are fp32 and stay so.  K and Q enter as fp16 with a power of two per row
// taken out, so that an element is off by at most 2^-25 of its row's largest (fp32
// rows as two parts, by 2^-23), their norms and decays as fp32 factors of rows; what
// is not a 16-bit number to begin with (S, T, X, R, U) enters as two fp16 parts, 23 bits.
// Products of two such leave out the one of the low parts.  The update of S is added
// in registers, with fp32's rounding (the tensor cores' sums cut off instead, and a
// state that adds up over thousands of tokens would drift).  S, R and U share a power
// of two per chunk and head that keeps them within fp16: |u_i| <= 64 max|v| + |S|
// because no step of the rule lets a column grow by more than |v| (|k| <= 1, beta <
// 1, decays of at most 1).  By the same bound no element of T or X passes 1.
//
// Measured: 8192 tokens, 16 key and 48 value heads, bf16, one request: 407 us (the
// bytes alone 40; 127 TFLOP/s of the rule's own operations); six ragged requests of
// 4613 tokens together, f16: 173.  Of the second, rows take 17 us, the chunk tasks 68,
// the walk 80; the first is the walk, 2.5 us a chunk, in which five waits follow one
// another (S^T K, R, U, the update, S again), each a product of 250 to 500 cycles, its
// signal (150) and a turn through registers of some hundred instructions a thread:
// neither bytes nor products bound it but their latency.
// States are within 2e-7 to 3e-7 of 64-bit ones, fp32 outputs within 3e-7 to 4e-7.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kq_device.cuh"
#include "kq_gdn.cuh"
#include "kq_internal.h"
#include "kq_kv.cuh"
#include "kq_tcgen05.cuh"

namespace kq {
namespace gdn {

using namespace tc;

__device__ unsigned int g_prompt_status = 0;
__device__ __forceinline__ void prompt_flag(int status) { atomicOr(&g_prompt_status, 1u << status); }

constexpr int kD = 128;                 // head dimension
constexpr int kTile = 32768;            // bytes of [K; Q] in fp16, or of [T; X] in two parts
// [K; Q] of fp32 has two parts as well, a tile each.
template <typename T>
constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
template <typename T>
constexpr int kKqTile = kParts<T> * kTile;
constexpr int kRowFactors = 4 * kChunk + 4;
// T, X, P and L, none of whose elements passes 1, enter as parts of 2^12 times themselves: the low part of an element as small
// as 2^-15 is a normal fp16 number then.  (Unscaled, fp32 outputs were off by 1.4e-6 instead of 1.05e-6; rounding the high parts, not cutting them off, then made it 6.4e-7.)
constexpr float kUp = 4096.f, kDown = 1.f / kUp;

struct PromptArgs {
  RuleArgs r;
  uint8_t* kq;      // [slot][key head] tiles
  uint8_t* tx;      // [slot][value head] tiles
  float* norms;     // [slot][key head]: of 64 keys and of 64 queries, what their rows are multiplied by to have unit length
  // Of each request's chunks: those that are walked down, and those that rows and tasks are done for, where these are not all
  // slots' (tasks_from < 0); `beside` where rows or tasks run beside the grid launched before them.
  int64_t from, to, tasks_from;
  int32_t beside;
  float* factors;   // [slot][value head][kRowFactors]: beta G fk, beta, fk G64/G / kUp, G fq kUp; G64, the largest value
};

// Where a request's chunks lie among the slots: q_start / 64 + r is at least the slots of the requests before it.
__device__ __forceinline__ int64_t chunk_base(int64_t first, int64_t r) { return first / kChunk + r; }

__device__ __forceinline__ uint32_t swizzled(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two numbers as high and low fp16 parts, each rounded: 23 bits, and low parts of either sign, so that the products of two low
// parts, which are left out, do not add up.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 l = fma2(__half22float2(h), make_float2(-1.f, -1.f), make_float2(a, b));
  hi = h2_bits(h);
  lo = h2_bits(__floats2half2_rn(l.x, l.y));
}

__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// c += (a_hi + a_lo) (b_hi + b_lo) of a 16 x 16 by 16 x 16 product, without that of the low parts.
__device__ __forceinline__ void mma_parts(float (&c0)[4], float (&c1)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                          const uint32_t (&bh)[4], const uint32_t (&bl)[4]) {
  mma_f16(c0, ah, bl[0], bl[1]);
  mma_f16(c1, ah, bl[2], bl[3]);
  mma_f16(c0, al, bh[0], bh[1]);
  mma_f16(c1, al, bh[2], bh[3]);
  mma_f16(c0, ah, bh[0], bh[1]);
  mma_f16(c1, ah, bh[2], bh[3]);
}
// A matrix of 8 x 8 fp16 numbers over a warp, its rows for its columns.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest magnitude of eight numbers as its pattern without the sign, which orders as the numbers do; and its value.
template <typename T>
__device__ __forceinline__ uint32_t pattern_max(const kv::Raw<T, 8>& raw) {
  uint32_t most = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int x = 0; x < 8; ++x) most = max(most, raw.u[x] & 0x7FFFFFFFu);
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x) most = __vmaxu2(most, raw.u[x] & 0x7FFF7FFFu);
    most = max(most >> 16, most & 0xFFFFu);
  }
  return most;
}
template <typename T>
__device__ __forceinline__ float pattern_value(uint32_t pattern) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(pattern);
  union { uint16_t b; T t; } top;
  top.b = (uint16_t)pattern;
  return kv::to_float(top.t);
}

// The last request whose chunks begin at or before this slot, and the chunk that lies there.
struct Place {
  Request req;
  int64_t first;  // token
  int n;          // tokens, 0 where the slot is empty
};
__device__ __forceinline__ Place place_of(const RuleArgs& a, int64_t slot) {
  const int lane = threadIdx.x % 32;
  Place p{};
  int64_t r = 0, span = a.s.requests;
  while (true) {
    const int64_t step = (span + 31) / 32, at = r + lane * step;
    const unsigned some = __ballot_sync(~0u, lane * step < span && chunk_base(max(a.s.q_start[at], 0), at) <= slot);
    if (!some) return p;
    const int last = 31 - __clz(some);
    r += last * step;
    if (step == 1) break;
    span = min(step, span - last * step);
  }
  p.req = read_request(a.s, r, a.max_new);
  if (p.req.status && threadIdx.x == 0) prompt_flag(p.req.status);
  if (!p.req.count || p.req.count <= a.short_most) return p;
  const int64_t c = slot - chunk_base(p.req.first, r);
  if (c < 0 || c * kChunk >= p.req.count) return p;
  p.first = p.req.first + c * kChunk, p.n = (int)min((int64_t)kChunk, p.req.count - c * kChunk);
  return p;
}

// A grid `beside` the one launched before it does not wait for it.  What keeps that safe:
//  - The grid before it is one of these kernels, and all of its CTAs triggered.  Each did so after its own wait, or is a grid beside
//    one that did: what grids before those wrote had been written and made visible by then.  So it may read that, the caller's inputs
//    and tiles of two launches back, and nothing that the grid before it, or the one that it ran beside, still writes.
//  - It writes what neither of these reads or writes: rows and tasks other chunks' slots, runs other requests' states and outputs.
//  - It ends after the grid before it, because its last CTA waits for that one; so whoever waits for it has waited for both.
// A trigger before a wait, a launch in between, or rows, tasks and walks in another order break this.  That a grid sees what was
// visible to the grid that triggered it, without a wait of its own, is how launches behave, not what PTX promises: waits there, where
// the walk is to be overlapped, would end the overlap (8192 tokens of 48 heads: 407 us in parts, 503 without).
__device__ __forceinline__ void end_beside(const PromptArgs& p) {
  if (p.beside && blockIdx.x == gridDim.x - 1) grid_dependency_wait();
}
__device__ __forceinline__ int64_t first_slot(const PromptArgs& p) {
  return p.tasks_from < 0 ? 0 : p.tasks_from + chunk_base(max(p.r.s.q_start[0], 0), 0);
}

// One chunk and key head: the tile of its keys and queries, each row brought to [1, 2) by a power of two and then fp16 (the
// rows' values stay what they are), and the rows' norms.
template <typename T>
__global__ void __launch_bounds__(256) gdn_rows_kernel(const PromptArgs p) {
  if (!p.beside) grid_dependency_wait();
  allow_dependent_launch();
  const RuleArgs& a = p.r;
  const int hk = blockIdx.x % a.k_heads;
  const int64_t slot = first_slot(p) + blockIdx.x / a.k_heads;
  const Place at = place_of(a, slot);
  if (!at.n) return end_beside(p);
  uint8_t* kq = p.kq + (slot * a.k_heads + hk) * kKqTile<T>;
  float* norms = p.norms + (slot * a.k_heads + hk) * 2 * kChunk;
  kv::Raw<T, 8> raw[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int e = threadIdx.x + x * 256, row = e / 16, i = row % kChunk;
    raw[x].clear();
    if (i < at.n) raw[x].load(reinterpret_cast<const T*>((row < kChunk ? a.k : a.q).at(at.first + i, hk)) + 8 * (e % 16));
  }
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int e = threadIdx.x + x * 256, row = e / 16, vec = e % 16, i = row % kChunk;
    uint32_t top = pattern_max(raw[x]);
#pragma unroll
    for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
    const float most = pattern_value<T>(top);
    const int power = (int)(__float_as_uint(most) >> 23);
    const float f = power == 255 || most == 0.f ? 1.f : __uint_as_float((uint32_t)max(254 - power, 1) << 23);
    float v[8], sum = 0.f;
    raw[x].get(v);
#pragma unroll
    for (int y = 0; y < 8; ++y) v[y] *= f, sum = fmaf(v[y], v[y], sum);
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    uint4 hi, lo;
    split2(v[0], v[1], hi.x, lo.x), split2(v[2], v[3], hi.y, lo.y), split2(v[4], v[5], hi.z, lo.z), split2(v[6], v[7], hi.w, lo.w);
    uint8_t* to = kq + vec / 8 * 16384 + swizzled(row, vec % 8);
    *reinterpret_cast<uint4*>(to) = hi;
    if (kParts<T> == 2) *reinterpret_cast<uint4*>(to + kTile) = lo;  // of 16-bit types it is zero
    // 0 for a row of zeros (and one of subnormal numbers) as well: its 1 / sqrt(eps) would pass fp16's range in w U, and a zero of K
    // times that is no number
    if (vec == 0) norms[row] = i < at.n && power > 0 ? 1.0f / sqrtf(sum + (a.eps * f) * f) : 0.f;
  }
  end_beside(p);
}

// -L in fp32 over the tile's rows 64.., which the queries leave and X takes: rows of 256 bytes, 32 in each half of the tile,
// in words of 16 bytes that lie apart for eight successive rows.
__device__ __forceinline__ uint32_t lower_at(int i, int j) {
  return i / 32 * 16384 + 8192 + i % 32 * 256 + (((j / 4) ^ ((i & 7) << 1)) << 4) + j % 4 * 4;
}
template <typename T>
constexpr int kChunkSmem = kKqTile<T>;

// One chunk and value head: T and X, the rows' factors.
//
// T is solved by blocks of 16: the four on the diagonal column by column, a warp each, then what lies below two of them, and
// below two such pairs, by two products with the tensor cores, T21 = T22 (-L21) T11.  (Diagonal blocks of 32 took two of the
// warps 9200 of a task's 31000 cycles.)  X = P T follows from the products' own layout: what a warp's mma leaves of
// its queries' rows is, times the decays, the operand of the next.  (Solving all of T and X in threads' registers took twice
// the instructions: 382 us for 129 chunks of 48 heads.)
template <typename T>
__global__ void __launch_bounds__(128, sizeof(T) == 4 ? 3 : 5) gdn_chunk_kernel(const PromptArgs p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(16) float s_fk[kChunk], s_fq[kChunk], s_beta[kChunk], s_hi[kChunk], s_lo[kChunk];
  __shared__ __align__(8) uint64_t s_full;
  __shared__ double s_first;
  __shared__ uint32_t s_vmax[4];
  if (!p.beside) grid_dependency_wait();
  allow_dependent_launch();
  const RuleArgs& a = p.r;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, h = blockIdx.x % a.v_heads;
  const int64_t slot = first_slot(p) + blockIdx.x / a.v_heads;
  const Place place = place_of(a, slot);
  if (!place.n) return end_beside(p);
  const int n = place.n, hk = h / (a.v_heads / a.k_heads);
  const int64_t first = place.first;
  if (tid == 0) {
    mbar_init(&s_full, 1);
    fence_barrier_init();
    mbar_arrive_expect_tx(&s_full, kKqTile<T>);
    bulk_g2s(smem, p.kq + (slot * a.k_heads + hk) * kKqTile<T>, kKqTile<T>, &s_full, l2_policy_evict_first());
  }
  // what is read comes at once: a wait for each after the other took 5000 of a task's 31000 cycles
  kv::Raw<T, 8> raw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int t = tid / 16 + e * 8;
    raw[e].clear();
    if (t < n) raw[e].load(reinterpret_cast<const T*>(a.v.at(first + t, h)) + 8 * (tid % 16));
  }
  const int64_t token = first + (tid < n ? tid : 0);
  const T gate = reinterpret_cast<const T*>(a.a + token * a.a_stride)[h], strength = reinterpret_cast<const T*>(a.b + token * a.b_stride)[h];
  const float a_log = a.a_log[h], dt_bias = a.dt_bias[h], norm = p.norms[(slot * a.k_heads + hk) * 2 * kChunk + tid];
  {  // the largest value
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, pattern_max(raw[e]));
    top = __reduce_max_sync(~0u, top);
    if (lane == 0) s_vmax[warp] = top;
  }
  (tid < kChunk ? s_fk : s_fq)[tid % kChunk] = norm;

  // decays: running sums of their base-2 logarithms in 64 bits, kept as two floats, for what counts is the difference of two
  // that may be large
  double g = 0.0;
  float beta = 0.f;
  if (tid < kChunk) {
    if (tid < n) {
      // e^-200 is nothing in fp32, and sums of 64 such keep 2^-38 of what follows them
      g = 1.4426950408889634 * (double)fmaxf(log_decay(kv::to_float(gate), a_log, dt_bias), -200.f);
      beta = sigmoid(kv::to_float(strength));
    }
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const double x = __shfl_up_sync(~0u, g, o);
      if (lane >= o) g += x;
    }
    if (tid == 31) s_first = g;
  }
  __syncthreads();
  if (tid < kChunk) {
    if (tid >= 32) g += s_first;
    const float hi = (float)g;
    s_hi[tid] = hi, s_lo[tid] = (float)(g - (double)hi);
    s_beta[tid] = beta;
  }

  __syncthreads();
  if (!mbar_wait_bounded(&s_full, 0)) {
    prompt_flag(KQ_ERR_TIMEOUT);
    mbar_wait_bounded(&s_full, 0);  // the copy gets the same time again, for the memory goes to another task
  }

  // products of 16 rows of queries and of keys a warp with the keys that they look back on, together, for these and the decays
  // are theirs in common (3600 tasks: 72 us one after the other, 68 so, although 48 bytes spill; with four CTAs an SM none do: 73)
  const uint32_t base = smem_u32(smem);
  float acc_p[8][4], acc_l[8][4];
#pragma unroll
  for (int b = 0; b < 8; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc_p[b][e] = acc_l[b][e] = 0.f;
  // the products with low parts first: a sum is cut off at each addition (fp32 outputs off by 3.1e-7, with all parts of a k
  // at once 5.6e-7)
#pragma unroll
  for (int low = kParts<T> - 1; low >= 0; --low)
#pragma unroll
    for (int k = 0; k < kD / 16; ++k) {
      const uint32_t half = base + k / 4 * 16384;
      const uint32_t mine = half + swizzled(warp * 16 + lane % 16, k % 4 * 2 + lane / 16), queries = mine + kChunk * 128;
      uint32_t fk[4], fq[4], fk_low[4], fq_low[4];
      ldmatrix4(fk, mine);
      ldmatrix4(fq, queries);
      if (low) ldmatrix4(fk_low, mine + kTile), ldmatrix4(fq_low, queries + kTile);
#pragma unroll
      for (int b = 0; b < 4; ++b) {  // 16 tokens: the matrices of tokens 0-7 and 8-15, low and high half of the 16 dimensions
        if (b > warp) continue;
        const uint32_t keys = half + swizzled(b * 16 + lane % 8 + lane / 16 * 8, k % 4 * 2 + lane / 8 % 2);
        uint32_t fb[4], fb_low[4];
        ldmatrix4(fb, keys);
        if (low) ldmatrix4(fb_low, keys + kTile);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (low) {
            mma_f16(acc_p[2 * b + e], fq, fb_low[2 * e], fb_low[2 * e + 1]);
            mma_f16(acc_l[2 * b + e], fk, fb_low[2 * e], fb_low[2 * e + 1]);
            mma_f16(acc_p[2 * b + e], fq_low, fb[2 * e], fb[2 * e + 1]);
            mma_f16(acc_l[2 * b + e], fk_low, fb[2 * e], fb[2 * e + 1]);
          } else {
            mma_f16(acc_p[2 * b + e], fq, fb[2 * e], fb[2 * e + 1]);
            mma_f16(acc_l[2 * b + e], fk, fb[2 * e], fb[2 * e + 1]);
          }
        }
      }
    }
  // of row i and the two columns from j on: the decays between, times the keys' norms
  auto decays = [&](int i, int j) {
    const float hi = s_hi[i], lo = s_lo[i];
    const float2 hj = *reinterpret_cast<const float2*>(s_hi + j), lj = *reinterpret_cast<const float2*>(s_lo + j);
    const float2 fj = *reinterpret_cast<const float2*>(s_fk + j);
    return make_float2(fj.x * exp2_fast((hi - hj.x) + (lo - lj.x)), fj.y * exp2_fast((hi - hj.y) + (lo - lj.y)));
  };
  uint32_t ph[4][4], pl[4][4];  // P as operands of 16 x 16
  __syncthreads();  // the tile is read: -L goes over its queries, T over its keys
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = warp * 16 + lane / 4 + e * 8;
    // the scale, which no fp16 part may have to hold, comes with the outputs
    const float of_p = kUp * s_fq[i], of_l = -s_beta[i] * s_fk[i];
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      if (b / 2 > warp) continue;
      const int j = b * 8 + lane % 4 * 2;
      const float2 r = decays(i, j);
      split2(j <= i ? acc_p[b][2 * e] * r.x * of_p : 0.f, j + 1 <= i ? acc_p[b][2 * e + 1] * r.y * of_p : 0.f, ph[b / 2][b % 2 * 2 + e],
             pl[b / 2][b % 2 * 2 + e]);
      *reinterpret_cast<float2*>(smem + lower_at(i, j)) =
          make_float2(j < i ? acc_l[b][2 * e] * r.x * of_l : 0.f, j + 1 < i ? acc_l[b][2 * e + 1] * r.y * of_l : 0.f);
    }
  }
  __syncthreads();

  uint8_t* lowpart = smem + kTile / 2;
  {  // column j of a diagonal block, from the first row down: t_i = [i = j] - sum_m L_im t_m; half the lanes keep the low parts
    const int j = lane % 16, at0 = 16 * warp;
    const uint32_t turn = warp * 64, from = warp / 2 * 16384 + warp % 2 * 4096;  // of row 16 warp + i, column 16 warp + m
    uint8_t* to = lane < 16 ? smem : lowpart;
    float2 t[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) t[m] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float2 s0 = make_float2(i == j ? 1.f : 0.f, 0.f), s1 = make_float2(0.f, 0.f);
#pragma unroll
      for (int m = 0; m < i; m += 4) {  // what lies at and past i is zero
        const float4 l = *reinterpret_cast<const float4*>(smem + ((lower_at(i, m) ^ turn) + from));
        s0 = fma2(make_float2(l.x, l.y), t[m / 2], s0);
        s1 = fma2(make_float2(l.z, l.w), t[m / 2 + 1], s1);
      }
      const float x = (s0.x + s1.x) + (s0.y + s1.y);
      (i % 2 ? t[i / 2].y : t[i / 2].x) = x;
      const float y = x * kUp;
      const __half hi = __float2half_rn(y);
      *reinterpret_cast<__half*>(to + swizzled(at0 + i, (at0 + j) / 8) + j % 8 * 2) = lane < 16 ? hi : __float2half_rn(y - __half2float(hi));
    }
  }
  __syncthreads();
  // Eight columns of T21 = T22 (-L21) T11 a warp, from row and column `at0` on, blocks of 16 * N: what the first product leaves
  // is turned into the second's right operand in registers.
  const uint32_t low = base + kTile / 2;
  auto below = [&](auto blocks, int at0, int col) {
    constexpr int N = decltype(blocks)::value;
    auto product = [&](float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], const uint32_t (&b)[4]) {
      mma_f16(c, ah, b[2], b[3]);
      mma_f16(c, al, b[0], b[1]);
      mma_f16(c, ah, b[0], b[1]);
    };
    uint32_t ah[4], al[4], b[N][4];  // of right operands: two registers of high parts, two of low ones
#pragma unroll
    for (int k = 0; k < N; ++k) ldmatrix4_t(b[k], (lane < 16 ? base : low) + swizzled(at0 + k * 16 + lane % 16, (at0 + col) / 8));
    float y[N][4] = {}, z[N][4] = {};
#pragma unroll
    for (int m = 0; m < N; ++m)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (16 * k + 16 <= col) continue;  // above T11's diagonal
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = at0 + 16 * (N + m) + lane / 4 + e % 2 * 8;
          const float2 l = *reinterpret_cast<const float2*>(smem + lower_at(row, at0 + k * 16 + lane % 4 * 2 + e / 2 * 8));
          split2(l.x * kUp, l.y * kUp, ah[e], al[e]);
        }
        product(y[m], ah, al, b[k]);
      }
#pragma unroll
    for (int m = 0; m < N; ++m) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        split2(y[m][2 * e] * kDown, y[m][2 * e + 1] * kDown, b[m][e], b[m][2 + e]);
        b[m][e] = turned(b[m][e]), b[m][2 + e] = turned(b[m][2 + e]);
      }
#pragma unroll
      for (int k = 0; k <= m; ++k) {
        const uint32_t at = swizzled(at0 + 16 * (N + m) + lane % 16, (at0 + 16 * (N + k)) / 8 + lane / 16);
        ldmatrix4(ah, base + at);
        ldmatrix4(al, low + at);
        product(z[m], ah, al, b[k]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t hi, lo;
        const uint32_t at = swizzled(at0 + 16 * (N + m) + lane / 4 + e * 8, (at0 + col) / 8) + lane % 4 * 4;
        split2(z[m][2 * e] * kDown, z[m][2 * e + 1] * kDown, hi, lo);
        *reinterpret_cast<uint32_t*>(smem + at) = hi, *reinterpret_cast<uint32_t*>(lowpart + at) = lo;
      }
    }
  };
  below(std::integral_constant<int, 1>{}, warp / 2 * 32, warp % 2 * 8);
  __syncthreads();
  below(std::integral_constant<int, 2>{}, 0, warp * 8);
  __syncthreads();

  // X = P T
  float x[8][4] = {};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k > warp) continue;
#pragma unroll
    for (int b = 0; b <= k; ++b) {
      uint32_t bh[4], bl[4];
      const uint32_t at = swizzled(k * 16 + lane % 16, b * 2 + lane / 16);
      ldmatrix4_t(bh, base + at);
      ldmatrix4_t(bl, low + at);
      mma_parts(x[2 * b], x[2 * b + 1], ph[k], pl[k], bh, bl);
    }
  }
#pragma unroll
  for (int b = 0; b < 8; ++b)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t hi, lo;
      const uint32_t at = swizzled(kChunk + warp * 16 + lane / 4 + e * 8, b) + lane % 4 * 4;
      split2(x[b][2 * e] * kDown, x[b][2 * e + 1] * kDown, hi, lo);
      *reinterpret_cast<uint32_t*>(smem + at) = hi, *reinterpret_cast<uint32_t*>(lowpart + at) = lo;
    }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p.tx + (slot * a.v_heads + h) * kTile),
                 "r"(base), "r"(kTile)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  if (tid < kChunk) {
    float* f = p.factors + (slot * a.v_heads + h) * kRowFactors;
    const float decay = exp2_fast(s_hi[tid]) * fmaf(s_lo[tid], 0.69314718f, 1.f), beta_i = s_beta[tid], fk = s_fk[tid];
    f[tid] = beta_i * decay * fk;
    f[kChunk + tid] = beta_i;
    f[2 * kChunk + tid] = kDown * fk * exp2_fast((s_hi[kChunk - 1] - s_hi[tid]) + (s_lo[kChunk - 1] - s_lo[tid]));
    f[3 * kChunk + tid] = kUp * decay * s_fq[tid];
    if (tid == 0) {
      f[4 * kChunk] = exp2_fast(s_hi[kChunk - 1]) * fmaf(s_lo[kChunk - 1], 0.69314718f, 1.f);
      f[4 * kChunk + 1] = pattern_value<T>(max(max(s_vmax[0], s_vmax[1]), max(s_vmax[2], s_vmax[3])));
    }
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  end_beside(p);
}

// ---- the walk down the chunks --------------------------------------------------------

// Everything is turned over here: a lane of tensor memory is a value dimension, so that S^T, R^T and (w U)^T are left
// operands, which tensor memory holds, straight from the registers that made them, and the chunk's tiles are right ones
// (128 value dimensions by 128, 128 and 128 columns, K = 128, 64 and 64):
//
//   D1 = S^T [K; Q]^T    D2 = R^T [T; X]^T    D3 = (w U)^T K
//
// A warp has 32 value dimensions (lanes) and a quarter of the columns (32 of S's rows, 16 tokens), and what a quarter made is
// one or two steps of K of the next product: products begin with the first quarter, and T's being triangular lets a quarter
// have its U when the quarters up to it have their R.  The queries' part of D1 and X's of D2 fill the gaps.
//
// With S, R and U as right operands in shared memory (64 value dimensions a CTA) each product read its left one, 4 KB, anew
// for 64 columns: 80 cycles each where the tensor core needs 32, and half a head took 6900 cycles a chunk.
//
// Sixteen warps compute, one issues products, one copies tiles, one fetches values' rows, one writes outputs' rows (as bulk
// copies of 256 bytes these two took 60 cycles a row, 7700 a chunk).

constexpr int kWorkWarps = 16, kWorkers = 32 * kWorkWarps;
constexpr int kRows = kD / 4, kToks = kChunk / 4;  // a thread's key dimensions of S, and its tokens
constexpr int kFactorBytes = kRowFactors * 4;
constexpr int kSlots = 3;  // of values and then outputs, and factors
// Two stages of tiles; one where [K; Q] has two parts, for shared memory holds no more.
template <typename T>
struct Walk {
  static constexpr int kStages = kParts<T> == 2 ? 1 : 2, kStage = kKqTile<T> + kTile;  // [K; Q], [T; X]
  static constexpr int kFactorsAt = kChunk * kD * (int)sizeof(T), kSlot = kFactorsAt + 2048;
  static constexpr int kSlotsAt = kStages * kStage;
  static constexpr int kSmem = kSlotsAt + kSlots * kSlot + 1024;  // and room to align
  static_assert(kSmem <= 232448 - 1024, "shared memory");
};
// tensor memory: S^T K, and over each 16 tokens' columns of it, once they are read, these tokens' U in two parts; S^T Q; U and
// then X's part of O; R's parts; D3; S's parts
constexpr int kDk = 0, kU = 0, kDq = 64, kDu = 128, kR = 192, kD3 = 256, kS = 384, kColumns = 512;

// Barriers that are waited on with a limit; after one ran out all waits return at once, and the warps run through.
struct Gate {
  volatile int* abort;
  __device__ __forceinline__ bool gone() const { return *abort != 0; }
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return;
    const long long start = clock64();
    while (!mbar_try_wait(bar, parity)) {
      if (gone()) return;
      if (clock64() - start > kWaitLimitCycles) {
        *abort = 1;
        prompt_flag(KQ_ERR_TIMEOUT);
        return;
      }
    }
  }
};

// Descriptor of an operand whose rows (128 bytes, 128-byte swizzle) run along K and whose N lies along the row: groups of 64
// of N `wide` bytes apart, of eight K 1024.
__device__ __forceinline__ uint64_t across_desc(const void* at, uint32_t wide) {
  const uint64_t start = (uint64_t)((smem_u32(at) >> 4) & 0x3FFF);
  return start | ((uint64_t)(wide >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
constexpr uint32_t kAcross = 1u << 16;  // of an instruction whose right operand lies so

// 16 bytes to shared memory, or as many zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// 2 N numbers of a lane as two fp16 parts, in N columns each.
template <int N>
__device__ __forceinline__ void put_parts(uint32_t hi_at, uint32_t lo_at, const float2 (&v)[N]) {
  static_assert(N % 8 == 0, "stores of eight columns");
#pragma unroll
  for (int c = 0; c < N; c += 8) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) split2(v[c + e].x, v[c + e].y, hi[e], lo[e]);
    tmem_st8(hi_at + c, hi);
    tmem_st8(lo_at + c, lo);
  }
  tmem_st_wait();
}

template <int N>
__device__ __forceinline__ void read_columns(uint32_t taddr, float2 (&v)[N]) {
  static_assert(N == 8 || N == 16, "one load");
  if constexpr (N == 8) {
    float f[16];
    tmem_ld16(taddr, f);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
  } else {
    uint32_t f[32];
    tmem_ld32(taddr, f);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float2(__uint_as_float(f[2 * i]), __uint_as_float(f[2 * i + 1]));
  }
}

template <typename T>
__global__ void __launch_bounds__(kWorkers + 128, 1) gdn_prompt_kernel(const PromptArgs p) {
  using W = Walk<T>;
  constexpr int kStages = W::kStages, kStage = W::kStage, kSlotsAt = W::kSlotsAt, kSlot = W::kSlot, kFactorsAt = W::kFactorsAt;
  constexpr int kRowWords = kD * (int)sizeof(T) / 16;  // of 16 bytes, of a row of values
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], tiles_free[kStages], slot_full[kSlots], slot_out[kSlots], slot_free[kSlots], s_ready[4], r_ready[4], u_ready[4],
      u_done[4], o_read, k_done, s_done[2], x_done, drained;
  __shared__ uint32_t s_tmem, s_most[2][kWorkWarps];
  __shared__ int s_abort;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  grid_dependency_wait();
  allow_dependent_launch();
  const RuleArgs& a = p.r;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int h = blockIdx.x % a.v_heads;
  // The longest first, of 32 requests at a time (six ragged ones of 48 heads, two rounds of CTAs: 103 us as they come,
  // 82 so).
  int64_t r = blockIdx.x / a.v_heads;
  if (a.s.requests > 1) {
    const int64_t mine = r / 32 * 32 + lane;
    const int count = mine < a.s.requests ? read_request(a.s, mine, a.max_new).count : -1;
    int before = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int other = __shfl_sync(~0u, count, i);
      before += other > count || (other == count && i < lane);
    }
    r = r / 32 * 32 + __ffs(__ballot_sync(~0u, before == r % 32)) - 1;
  }
  Request req = read_request(a.s, r, a.max_new);
  if (req.status && tid == 0) prompt_flag(req.status);
  if (!req.count || req.count <= a.short_most || p.from * kChunk >= req.count) return;
  const int64_t slot0 = chunk_base(req.first, r) + p.from;
  // from here on the request is the part of it that is walked down
  req.fresh = req.fresh && p.from == 0;
  req.first += (int32_t)(p.from * kChunk), req.count = (int32_t)(min((int64_t)req.count, p.to * kChunk) - p.from * kChunk);
  const int chunks = (req.count + kChunk - 1) / kChunk;
  const int hk = h / (a.v_heads / a.k_heads);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1), mbar_init(&tiles_free[i], 1);
    for (int i = 0; i < kSlots; ++i) mbar_init(&slot_full[i], 32), mbar_init(&slot_out[i], kWorkers), mbar_init(&slot_free[i], 32);
    for (int i = 0; i < 4; ++i)
      mbar_init(&s_ready[i], kWorkers / 4), mbar_init(&r_ready[i], kWorkers / 4), mbar_init(&u_ready[i], kWorkers / 4), mbar_init(&u_done[i], 1);
    mbar_init(&o_read, kWorkers);
    for (uint64_t* b : {&k_done, &s_done[0], &s_done[1], &x_done, &drained}) mbar_init(b, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == kWorkWarps) {
    tmem_alloc(&s_tmem, kColumns);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const Gate gate{&s_abort};

  if (warp == kWorkWarps + 1) {  // tiles
    if (elect_one()) {
      const uint64_t policy = l2_policy_evict_first();
      int c = 0;
      for (; c < chunks; ++c) {
        uint8_t* at = smem + c % kStages * kStage;
        uint64_t* bar = &full[c % kStages];
        if (c >= kStages) gate.wait(&tiles_free[c % kStages], c / kStages - 1 & 1);
        if (gate.gone()) break;
        mbar_arrive_expect_tx(bar, kStage);
        bulk_g2s(at, p.kq + ((slot0 + c) * a.k_heads + hk) * kKqTile<T>, kKqTile<T>, bar, policy);
        bulk_g2s(at + kKqTile<T>, p.tx + ((slot0 + c) * a.v_heads + h) * kTile, kTile, bar, policy);
      }
      // the copies that nobody waits for after a wait ran out
      for (int i = max(0, c - kStages); i < c; ++i) mbar_wait_bounded(&full[i % kStages], i / kStages & 1);
    }
    __syncwarp();
  } else if (warp == kWorkWarps + 2) {  // values, none past the last token, and factors
    for (int c = 0; c < chunks; ++c) {
      if (c >= kSlots) gate.wait(&slot_free[c % kSlots], c / kSlots - 1 & 1);
      const uint32_t at = smem_u32(smem + kSlotsAt + c % kSlots * kSlot);
      const int count = req.count - c * kChunk;
      const char* from = a.v.at(req.first + (int64_t)c * kChunk, h) + lane % kRowWords * 16;
#pragma unroll 8
      for (int t = lane / kRowWords; t < kChunk; t += 32 / kRowWords)
        copy16(at + (t * kRowWords + lane % kRowWords) * 16, t < count ? from + t * a.v.token_stride : from, t < count ? 16 : 0);
      const float* f = p.factors + ((slot0 + c) * a.v_heads + h) * kRowFactors;
      for (int t = lane; t < kFactorBytes / 16; t += 32) copy16(at + kFactorsAt + t * 16, f + t * 4, 16);
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&slot_full[c % kSlots])) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kWorkWarps + 3) {  // outputs, which lie where the values were
    for (int c = 0; c < chunks; ++c) {
      gate.wait(&slot_out[c % kSlots], c / kSlots & 1);
      const uint8_t* from = smem + kSlotsAt + c % kSlots * kSlot + lane % kRowWords * 16;
      const int count = min(kChunk, req.count - c * kChunk);
      char* to = a.out.at(req.first + (int64_t)c * kChunk, h) + lane % kRowWords * 16;
#pragma unroll 8
      for (int t = lane / kRowWords; t < count; t += 32 / kRowWords)
        *reinterpret_cast<uint4*>(to + t * a.out.token_stride) = *reinterpret_cast<const uint4*>(from + t * kRowWords * 16);
      mbar_arrive(&slot_free[c % kSlots]);
    }
  } else if (warp == kWorkWarps) {  // products
    if (elect_one()) {
      const uint32_t narrow = idesc_f16(128, kChunk), wide = idesc_f16(128, kD / 2) | kAcross;
      constexpr uint64_t kLower = (kChunk * 128) >> 4, kLowPart = (kTile / 2) >> 4;  // a tile's rows 64.., its low parts
      for (int c = 0; c < chunks; ++c) {
        const uint8_t* at = smem + c % kStages * kStage;
        const uint64_t kd = sw128_desc(at), td = sw128_desc(at + kKqTile<T>), kt = across_desc(at, 16384);
        // A sum on the tensor cores is cut off, not rounded, at each addition: what is small comes first where nothing waits.
        constexpr int kPasses = kParts<T> + 1;
        auto state = [&](uint32_t to, uint64_t rows, int k, int pass, bool more) {  // 16 of S's key dimensions
          // low x whole, then high x low of K or Q where it has a low part, then high x high
          const bool low = pass == 0, low_rows = kPasses == 3 && pass == 1;
          tc_mma_ts(tmem + to, tmem + kS + low * (kD / 2) + k * 8,
                    rows + (uint64_t)((k / 4 * 16384 + k % 4 * 32 + low_rows * kTile) >> 4), narrow, more);
        };
        auto solved = [&](uint32_t to, uint64_t rows, int k, int pass, bool more) {  // 16 tokens' R, and the tokens from there on
          // low x high, high x low, high x high
          tc_mma_ts(tmem + to + 16 * k, tmem + kR + (pass == 0 ? kChunk / 2 : 0) + k * 8,
                    rows + (pass == 1 ? kLowPart : 0) + (uint64_t)((k * 16 * 128 + k * 32) >> 4), idesc_f16(128, kChunk - 16 * k), more);
        };
        auto update = [&](int half, int k) {  // 16 tokens' U, 64 of S's key dimensions
          const uint64_t keys = kt + (uint64_t)((half * 16384 + k * 2048) >> 4);
          const uint32_t to = tmem + kD3 + half * (kD / 2), u = tmem + kU + k * 16;
          tc_mma_ts(to, u + 8, keys, wide, k);
          if (kParts<T> == 2) tc_mma_ts(to, u, keys + (kTile >> 4), wide, 1);
          tc_mma_ts(to, u, keys, wide, 1);
        };
        if (gate.gone()) break;
        gate.wait(&full[c % kStages], c / kStages & 1);
        if (c) gate.wait(&s_done[1], c - 1 & 1);  // the last chunk's U, which the first product goes over, is read
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          gate.wait(&s_ready[j], c & 1);
          tc_fence_after();
#pragma unroll
          for (int k = 2 * j; k < 2 * j + 2; ++k)
#pragma unroll
            for (int pass = 0; pass < kPasses; ++pass) state(kDk, kd, k, pass, k || pass);
        }
        tc_commit(&k_done);
        if (c) {  // the last chunk's outputs are in registers
          gate.wait(&o_read, c - 1 & 1);
          tc_fence_after();
        }
#pragma unroll
        for (int pass = 0; pass < kPasses; ++pass)
#pragma unroll
          for (int k = 0; k < kD / 16; ++k) state(kDq, kd + kLower, k, pass, k || pass);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          gate.wait(&r_ready[j], c & 1);
          tc_fence_after();
#pragma unroll
          for (int pass = 0; pass < 3; ++pass) solved(kDu, td, j, pass, j || pass);
          tc_commit(&u_done[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          gate.wait(&u_ready[j], c & 1);
          tc_fence_after();
          update(0, j);
        }
        tc_commit(&s_done[0]);  // half of S goes on while the other half is made
#pragma unroll
        for (int j = 0; j < 4; ++j) update(1, j);
        tc_commit(&s_done[1]);
#pragma unroll
        for (int pass = 0; pass < 3; ++pass)
#pragma unroll
          for (int j = 0; j < 4; ++j) solved(kDu, td + kLower, j, pass, j || pass);
        if (c + kStages < chunks) tc_commit(&tiles_free[c % kStages]);  // only where it is waited for
        tc_commit(&x_done);
      }
      if (!gate.gone()) gate.wait(&x_done, chunks - 1 & 1);  // nothing is in flight when the memory goes
      if (gate.gone()) {  // a wait ran out, here or elsewhere: the products get the same time again
        tc_commit(&drained);
        mbar_wait_bounded(&drained, 0);
      }
    }
    __syncwarp();
  } else {
    const int quarter = warp % 4, sub = warp / 4, dim = quarter * 32 + lane;  // a value dimension; which quarter of the columns
    const uint32_t mine = tmem + (quarter << 21);
    float* state = a.state + (((int64_t)req.slot * a.v_heads + h) * kD + sub * kRows) * kD + dim;
    float2 S[kRows / 2];  // rows of two successive key dimensions, times 2^power
#pragma unroll
    for (int e = 0; e < kRows / 2; ++e)
      S[e] = req.fresh ? make_float2(0.f, 0.f) : make_float2(state[2 * e * kD], state[(2 * e + 1) * kD]);
    auto factors = [&](int c, int which) {  // of this warp's tokens
      return reinterpret_cast<const float*>(smem + kSlotsAt + c % kSlots * kSlot + kFactorsAt) + which * kChunk + sub * kToks;
    };
    auto values = [&](int c) {  // of this thread's tokens, and then their outputs
      return reinterpret_cast<T*>(smem + kSlotsAt + c % kSlots * kSlot) + sub * kToks * kD + dim;
    };
    auto largest = [&]() {
      uint32_t most = 0;
#pragma unroll
      for (int e = 0; e < kRows / 2; ++e) most = max(most, max(__float_as_uint(fabsf(S[e].x)), __float_as_uint(fabsf(S[e].y))));
      return __reduce_max_sync(~0u, most);
    };
    float down = 1.f;
    auto outputs = [&](int c) {  // of a chunk whose S was taken at scale / down
      float2 q[kToks / 2], x[kToks / 2];
      gate.wait(&x_done, c & 1);
      tc_fence_after();
      read_columns(mine + kDq + sub * kToks, q);
      read_columns(mine + kDu + sub * kToks, x);
      tc_fence_before();
      mbar_arrive(&o_read);
      const float* f3 = factors(c, 3);
#pragma unroll
      for (int e = 0; e < kToks / 2; e += 2) {
        const float4 w = *reinterpret_cast<const float4*>(f3 + 2 * e);
        x[e] = mul2(fma2(q[e], make_float2(w.x, w.y), x[e]), both(down));
        x[e + 1] = mul2(fma2(q[e + 1], make_float2(w.z, w.w), x[e + 1]), both(down));
      }
      T* out = values(c);
#pragma unroll
      for (int e = 0; e < kToks; ++e) out[e * kD] = kv::from_float<T>(e % 2 ? x[e / 2].y : x[e / 2].x);
      mbar_arrive(&slot_out[c % kSlots]);  // factors and values are read, outputs written
    };
    // A chunk's values times their strengths, made while the chunk before is waited for; returns the largest value.
    float2 strong[kToks / 2];
    auto strengthen = [&](int c) {
      gate.wait(&slot_full[c % kSlots], c / kSlots & 1);
      const float* f1 = factors(c, 1);
      const T* value = values(c);
      auto v = [&](int t) { return kv::to_float(value[t * kD]); };
#pragma unroll
      for (int e = 0; e < kToks / 2; e += 2) {
        const float4 y = *reinterpret_cast<const float4*>(f1 + 2 * e);
        strong[e] = mul2(make_float2(v(2 * e), v(2 * e + 1)), make_float2(y.x, y.y));
        strong[e + 1] = mul2(make_float2(v(2 * e + 2), v(2 * e + 3)), make_float2(y.z, y.w));
      }
      return factors(c, 0)[4 * kChunk + 1 - sub * kToks];
    };
    int power = 0;  // S is kept times 2^power, so that it, R and U stay within 2^15
    float reach = 0.f;  // no column of S is longer (a column has 128 entries, so 12 times the largest at most)
    auto measure = [&](int turn) {  // reach from S as it is; all warps together
      const uint32_t most = largest();
      if (lane == 0) s_most[turn][warp] = most;
      named_barrier(1, kWorkers);
      reach = 12.f * __uint_as_float(__reduce_max_sync(~0u, lane < kWorkWarps ? s_most[turn][lane] : 0u)) * power_of_two(-power);
    };
    auto rescale = [&](float vmax) {  // |R| and |U| of a chunk are at most 64 max|v| + the longest column
      const int bound = (int)(__float_as_uint(fmaf(64.f, vmax, reach)) >> 23) - 126;  // 2^bound is more
      const int want = min(max(15 - bound, -120), 120);
      if (want >= power && want <= power + 3) return;
      const int half = (want - power) / 2;  // in two steps, for the whole may be no number
      const float2 by = both(power_of_two(half)), on = both(power_of_two(want - power - half));
#pragma unroll
      for (int e = 0; e < kRows / 2; ++e) S[e] = mul2(mul2(S[e], by), on);
      power = want;
    };
    measure(0);
    rescale(strengthen(0));
    for (int c = 0; c < chunks; ++c) {
      put_parts(mine + kS + sub * (kRows / 2), mine + kS + kD / 2 + sub * (kRows / 2), S);
      tc_fence_before();
      mbar_arrive(&s_ready[sub]);
      if (c) outputs(c - 1);
      down = kDown * a.scale * power_of_two(-power);
      float2 d[kToks / 2];
      gate.wait(&k_done, c & 1);
      tc_fence_after();
      read_columns(mine + kDk + sub * kToks, d);
      {
        const float* f0 = factors(c, 0);
        const float2 up = both(power_of_two(power));
#pragma unroll
        for (int e = 0; e < kToks / 2; e += 2) {
          const float4 x = *reinterpret_cast<const float4*>(f0 + 2 * e);
          d[e] = fma2(d[e], make_float2(-x.x, -x.y), mul2(strong[e], up));
          d[e + 1] = fma2(d[e + 1], make_float2(-x.z, -x.w), mul2(strong[e + 1], up));
        }
      }
      put_parts(mine + kR + sub * (kToks / 2), mine + kR + kChunk / 2 + sub * (kToks / 2), d);
      tc_fence_before();
      mbar_arrive(&r_ready[sub]);
      gate.wait(&u_done[sub], c & 1);
      tc_fence_after();
      read_columns(mine + kDu + sub * kToks, d);
      {
        const float* f2 = factors(c, 2);
#pragma unroll
        for (int e = 0; e < kToks / 2; e += 2) {
          const float4 x = *reinterpret_cast<const float4*>(f2 + 2 * e);
          d[e] = mul2(d[e], make_float2(x.x, x.y)), d[e + 1] = mul2(d[e + 1], make_float2(x.z, x.w));
        }
      }
      put_parts(mine + kU + sub * kToks, mine + kU + sub * kToks + kToks / 2, d);
      tc_fence_before();
      mbar_arrive(&u_ready[sub]);
      const float decay = factors(c, 0)[4 * kChunk - sub * kToks], vmax = factors(c, 0)[4 * kChunk + 1 - sub * kToks];
      const float vnext = c + 1 < chunks ? strengthen(c + 1) : vmax;
      gate.wait(&s_done[sub / 2], c & 1);
      tc_fence_after();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        read_columns(mine + kD3 + sub * kRows + half * 16, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) S[8 * half + e] = fma2(S[8 * half + e], both(decay), d[e]);
      }
      tc_fence_before();
      // S's columns have grown by 64 max|v| at most; what they came to is looked at now and then
      reach = fmaf(64.f, vmax, reach);
      if (c % 8 == 7 && c + 1 < chunks) measure(c / 8 & 1);
      rescale(vnext);
    }
    outputs(chunks - 1);
    const float back = power_of_two(-power);
#pragma unroll
    for (int e = 0; e < kRows / 2; ++e) state[2 * e * kD] = S[e].x * back, state[(2 * e + 1) * kD] = S[e].y * back;
  }
  __syncthreads();
  if (warp == kWorkWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, kColumns);
  }
}

constexpr int kFirstPart = 12;  // chunks

static int64_t prompt_slots(int64_t requests, int64_t tokens) { return tokens / kChunk + requests; }
static int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

int64_t prompt_workspace(int k_heads, int v_heads, int64_t requests, int64_t tokens, int dtype) {
  const int64_t slots = prompt_slots(requests, tokens), kq = dtype == KQ_F32 ? kKqTile<float> : kKqTile<__half>;
  return slots * (k_heads * kq + v_heads * (int64_t)kTile) + align256(slots * k_heads * 2 * kChunk * 4) +
         align256(slots * v_heads * kRowFactors * 4);
}

template <typename T>
static cudaError_t launch(const RuleArgs& a, void* ws, cudaStream_t st) {
  const int64_t slots = prompt_slots(a.s.requests, a.s.tokens);
  PromptArgs p{};
  p.r = a;
  p.kq = static_cast<uint8_t*>(ws);
  p.tx = p.kq + slots * a.k_heads * kKqTile<T>;
  p.norms = reinterpret_cast<float*>(p.tx + slots * a.v_heads * kTile);
  p.factors = p.norms + align256(slots * a.k_heads * 2 * kChunk * 4) / 4;
  if (cudaError_t e = cudaFuncSetAttribute(gdn_chunk_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kChunkSmem<T>)) return e;
  if (cudaError_t e = cudaFuncSetAttribute(gdn_prompt_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Walk<T>::kSmem)) return e;
  const auto rows = [&](int64_t chunks) {
    return launch_dependent(gdn_rows_kernel<T>, dim3((unsigned)(chunks * a.k_heads)), dim3(256), 0, st, p);
  };
  const auto tasks = [&](int64_t chunks) {
    return launch_dependent(gdn_chunk_kernel<T>, dim3((unsigned)(chunks * a.v_heads)), dim3(128), kChunkSmem<T>, st, p);
  };
  const auto walk = [&]() {
    return launch_dependent(gdn_prompt_kernel<T>, dim3((unsigned)(a.s.requests * a.v_heads)), dim3(kWorkers + 128), Walk<T>::kSmem, st, p);
  };
  // One request's heads leave SMs idle: its chunks go in parts, and while one part is walked down, the next one's chunk tasks
  // and the rows of the one after run on the other SMs (1.4 us a chunk on what 48 heads leave, against 2.6 of walking, so
  // parts may grow).  8192 tokens of 48 heads: 503 us at once, 439 in parts; tasks and walk as CTAs of one kernel, which then
  // held the registers of the larger, 500.
  const int64_t chunks = (std::min(a.max_new, a.s.tokens) + kChunk - 1) / kChunk;
  if (a.s.requests == 1 && 2 * a.v_heads <= 152 && chunks >= 2 * kFirstPart) {
    const auto part_after = [&](int64_t to, int64_t size) {  // what follows chunk `to`, the end of a part of that size
      const int64_t left = chunks - to;
      return left < 2 * size ? left : size * 3 / 2;
    };
    int64_t from = 0, size = kFirstPart, next = part_after(size, size);
    p.tasks_from = 0;
    if (cudaError_t e = rows(size)) return e;
    if (cudaError_t e = tasks(size)) return e;
    p.beside = 1;
    p.tasks_from = size;
    if (cudaError_t e = rows(next)) return e;
    while (true) {
      p.from = from, p.to = from + size;
      if (cudaError_t e = walk()) return e;
      if (!next) return cudaSuccess;
      p.tasks_from = p.to;
      if (cudaError_t e = tasks(next)) return e;
      from += size, size = next, next = part_after(from + size, size);
      p.tasks_from = from + size;
      if (next)
        if (cudaError_t e = rows(next)) return e;
    }
  }
  p.to = INT64_MAX / kChunk, p.tasks_from = -1;
  if (cudaError_t e = rows(slots)) return e;
  if (cudaError_t e = tasks(slots)) return e;
  return walk();
}

cudaError_t launch_prompt(const RuleArgs& a, int dtype, void* ws, cudaStream_t st) {
  return dtype == KQ_F32 ? launch<float>(a, ws, st) : dtype == KQ_F16 ? launch<__half>(a, ws, st) : launch<__nv_bfloat16>(a, ws, st);
}

int prompt_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_prompt_status, sizeof(v)) != cudaSuccess) return -1;
  if (clear && v) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(g_prompt_status, &z, sizeof(z)) != cudaSuccess) return -1;
  }
  return (int)v;
}

}  // namespace gdn
}  // namespace kq
