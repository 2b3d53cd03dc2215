// The gated-delta layers' operators beside their projections: the short causal
// convolution with its rolling state, and the gated delta rule token by token.
// (kq_gdn_prompt.cu has the runs of more than kShortRun tokens.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kq_device.cuh"
#include "kq_gdn.cuh"
#include "kq_internal.h"
#include "kq_kv.cuh"

namespace kq {
namespace gdn {

__device__ unsigned int g_gdn_status = 0;
__device__ __forceinline__ void gdn_flag(int status) { atomicOr(&g_gdn_status, 1u << status); }

// ---- the causal convolution -----------------------------------------------------
//
// y[t] = silu(bias + sum_j w[j] x[t - W + 1 + j]), channel by channel: two flops a
// byte or less, so memory bounds it.  A warp takes four channels a lane and
// walks down a piece of a request's tokens with the last W - 1 inputs in registers:
// each input is read once but for the W - 1 before a piece.  Pieces begin at the
// request's first token and every kPiece tokens from there, so only a request's
// first piece reads its state, and the same lanes write the new one: nothing is
// read after another CTA wrote it.  Each request has a warp for its first piece,
// which finds it without a search (a decode step is all such); the pieces after it
// belong to the window of kPiece token rows they begin in, one at most in each,
// whose warp finds the request by a 32-way search of q_start.
//
// Measured: 64 requests' tokens of 10240 f16 channels 6.5 us (1.6 of bytes, the rest
// three loads that wait for one another, the last the state's behind the request's length, and a
// launch); in fp32 6.7; 7 ragged requests of 5900 tokens together, bf16, 49 us, 4.9 TB/s, in fp32 83,
// 5.8 TB/s.  Eight channels a lane, or eight tokens' loads ahead, took
// more registers and as long.

constexpr int kConvWarps = 4, kConvAhead = 4, kConvWide = 4;

struct ConvArgs {
  Rows x, out;
  Requests s;
  char* state;
  const float* weight;
  const float* bias;
  int32_t channels, silu;
  int32_t piece;
  int64_t windows;
};

template <typename T, int W>
__global__ void __launch_bounds__(32 * kConvWarps) conv_kernel(const ConvArgs a) {
  constexpr int V = kConvWide;  // channels of a lane
  const int lane = threadIdx.x % 32;
  const int64_t unit = (int64_t)blockIdx.x * kConvWarps + threadIdx.x / 32;
  const int channel = (blockIdx.y * 32 + lane) * V;
  const bool here = channel < a.channels;
  grid_dependency_wait();
  allow_dependent_launch();
  float w[W][V], bias[V];
  if (here) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float* from = a.weight + (int64_t)(channel + e) * W;
      if constexpr (W == 4) {
        const float4 x = *reinterpret_cast<const float4*>(from);
        w[0][e] = x.x, w[1][e] = x.y, w[2][e] = x.z, w[3][e] = x.w;
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = from[j];
      }
      bias[e] = a.bias ? a.bias[channel + e] : 0.f;
    }
  }
  int64_t r = unit, begin = 0;
  if (unit >= a.s.requests) {  // the last request that begins at or before the window
    const int64_t window = unit - a.s.requests, lo = window * a.piece;
    if (window >= a.windows) return;
    if (window == 0 && lane == 0 && (a.s.q_start[0] < 0 || a.s.q_start[0] > a.s.tokens)) gdn_flag(KQ_ERR_RANGE);
    r = 0;
    for (int64_t span = a.s.requests;;) {
      const int64_t step = (span + 31) / 32, at = r + lane * step;
      const unsigned some = __ballot_sync(~0u, lane * step < span && a.s.q_start[at] <= lo);
      if (!some) return;
      const int last = 31 - __clz(some);
      r += last * step;
      if (step == 1) break;
      span = min(step, span - last * step);
    }
    begin = (lo - a.s.q_start[r] + a.piece - 1) / a.piece * a.piece;
    if (begin <= 0) return;  // that is its first piece
  }
  const Request q = read_request(a.s, r, a.s.tokens);
  if (q.status && lane == 0) gdn_flag(q.status);
  if (begin >= q.count || !here) return;
  const int32_t from = (int32_t)begin, end = min(q.count, from + a.piece);
  const char* x = a.x.at(q.first, 0) + channel * sizeof(T);
  char* out = a.out.at(q.first, 0) + channel * sizeof(T);
  T* kept = reinterpret_cast<T*>(a.state) + (int64_t)q.slot * (W - 1) * a.channels + channel;
  kv::Raw<T, V> raw[kConvAhead];
  auto load = [&](int32_t t) {
#pragma unroll
    for (int i = 0; i < kConvAhead; ++i)
      if (t + i < end) raw[i].load(reinterpret_cast<const T*>(x + (t + i) * a.x.token_stride));
  };
  load(from);
  kv::Raw<T, V> old[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    old[j].clear();
    if (from > 0) old[j].load(reinterpret_cast<const T*>(x + (from - (W - 1) + j) * a.x.token_stride));
    else if (!q.fresh) old[j].load(kept + (int64_t)j * a.channels);
  }
  if (from == 0) {  // the new state: the last inputs, those of the old one among them where there are fewer
    kv::Raw<T, V> next[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int32_t at = q.count - (W - 1) + j;
      if (at >= 0) next[j].load(reinterpret_cast<const T*>(x + at * a.x.token_stride));
      else if (q.count == 1) next[j] = old[j + 1 < W - 1 ? j + 1 : W - 2];
      else next[j] = old[j + 2 < W - 1 ? j + 2 : W - 2];  // fewer than W - 1 are one or two
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      next[j].store(kept + (int64_t)j * a.channels);
  }
  float past[W - 1][V];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) old[j].get(past[j]);
  for (int32_t t = from; t < end; t += kConvAhead) {
    kv::Raw<T, V> now[kConvAhead];
#pragma unroll
    for (int i = 0; i < kConvAhead; ++i) now[i] = raw[i];
    load(t + kConvAhead);
#pragma unroll
    for (int i = 0; i < kConvAhead; ++i) {
      float v[V], y[V];
      now[i].get(v);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float s = bias[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) s = fmaf(w[j][e], past[j][e], s);
        s = fmaf(w[W - 1][e], v[e], s);
        y[e] = a.silu ? silu<T>(s) : s;
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) past[j][e] = past[j + 1][e];
        past[W - 2][e] = v[e];
      }
      if (t + i >= end) continue;
      kv::store4(reinterpret_cast<T*>(out + (t + i) * a.out.token_stride), y);
    }
  }
}

template <typename T>
static cudaError_t launch_conv(const ConvArgs& a, int width, cudaStream_t st) {
  const int wide = 32 * kConvWide;
  const dim3 grid((unsigned)((a.s.requests + a.windows + kConvWarps - 1) / kConvWarps), (unsigned)((a.channels + wide - 1) / wide));
  const auto k = width == 2 ? conv_kernel<T, 2> : width == 3 ? conv_kernel<T, 3> : conv_kernel<T, 4>;
  return launch_dependent(k, grid, dim3(32 * kConvWarps), 0, st, a);
}

// ---- the gated delta rule, token by token ------------------------------------------
//
// A state's columns do not know of one another: u_c = beta (v_c - g S_c . k),
// S_c <- g S_c + k u_c, out_c = S_c . q = g S_c . q + (k . q) u_c with S before.  So
// a CTA keeps 32 columns of one state in registers, eight rows of four columns a
// thread, from the first token of its request to the last: the state is read and
// written once however many tokens there are.
//
// A decode step (gdn_step_kernel, one token a request) is bound by the states' bytes
// (128 KB a value head read and written at D = 128); both products with S are made in
// one pass over the registers, and one barrier joins the four warps' sums.  Measured:
// 128 requests of 48 heads (806 MB) 120 us, 6.7 TB/s, what a copy reaches.

constexpr int kStepThreads = 128, kStepCols = 32;

template <typename T, int D>
__global__ void __launch_bounds__(kStepThreads) gdn_step_kernel(const RuleArgs p) {
  constexpr int kSlices = D / kStepCols, kRows = D / 16;
  __shared__ __align__(16) float s_k[D], s_q[D];
  __shared__ __align__(16) float s_part[4][2][kStepCols];
  __shared__ float s_kq;
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int slice = blockIdx.x % kSlices, h = blockIdx.x / kSlices % p.v_heads;
  const int64_t r = blockIdx.x / kSlices / p.v_heads;
  const Request req = read_request(p.s, r, p.max_new);
  if (req.status && tid == 0) gdn_flag(req.status);
  if (!req.count) return;
  const int hk = h / (p.v_heads / p.k_heads);
  const int64_t token = req.first;
  const int row0 = (warp * 4 + lane / 8) * kRows, col = (lane % 8) * 4, col0 = slice * kStepCols;
  float* state = p.state + ((int64_t)req.slot * p.v_heads + h) * D * D + (int64_t)row0 * D + col0 + col;
  float4 S[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    S[i] = req.fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(state + (int64_t)i * D);
  if (warp == 0) {
    float kk[8], qq[8], k2 = 0.f, q2 = 0.f, kq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) kk[i] = qq[i] = 0.f;
    if (lane < D / 8) {
      kv::load8(reinterpret_cast<const T*>(p.k.at(token, hk)) + 8 * lane, kk);
      kv::load8(reinterpret_cast<const T*>(p.q.at(token, hk)) + 8 * lane, qq);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) k2 = fmaf(kk[i], kk[i], k2), q2 = fmaf(qq[i], qq[i], q2), kq = fmaf(kk[i], qq[i], kq);
#pragma unroll
    for (int o = D / 16; o; o >>= 1) {
      k2 += __shfl_xor_sync(~0u, k2, o);
      q2 += __shfl_xor_sync(~0u, q2, o);
      kq += __shfl_xor_sync(~0u, kq, o);
    }
    const float fk = p.unit ? 1.0f / sqrtf(k2 + p.eps) : 1.f, fq = p.unit ? p.scale / sqrtf(q2 + p.eps) : p.scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) kk[i] *= fk, qq[i] *= fq;
    if (lane < D / 8) kv::store8(&s_k[8 * lane], kk), kv::store8(&s_q[8 * lane], qq);
    if (lane == 0) s_kq = kq * fk * fq;
  }
  const float a = kv::to_float(reinterpret_cast<const T*>(p.a + token * p.a_stride)[h]);
  const float b = kv::to_float(reinterpret_cast<const T*>(p.b + token * p.b_stride)[h]);
  float v[4];
  kv::load4(reinterpret_cast<const T*>(p.v.at(token, h)) + col0 + col, v);
  const float g = expf(p.gates ? log_decay(a, p.a_log[h], p.dt_bias[h]) : a), beta = p.gates ? sigmoid(b) : b;
  __syncthreads();
  float kr[kRows], qr[kRows];
#pragma unroll
  for (int i = 0; i < kRows; i += 4) kv::load4(&s_k[row0 + i], kr + i), kv::load4(&s_q[row0 + i], qr + i);
  float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), qs = ks;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    ks.x = fmaf(kr[i], S[i].x, ks.x), ks.y = fmaf(kr[i], S[i].y, ks.y);
    ks.z = fmaf(kr[i], S[i].z, ks.z), ks.w = fmaf(kr[i], S[i].w, ks.w);
    qs.x = fmaf(qr[i], S[i].x, qs.x), qs.y = fmaf(qr[i], S[i].y, qs.y);
    qs.z = fmaf(qr[i], S[i].z, qs.z), qs.w = fmaf(qr[i], S[i].w, qs.w);
  }
#pragma unroll
  for (int o = 8; o < 32; o *= 2) {
    ks.x += __shfl_xor_sync(~0u, ks.x, o), ks.y += __shfl_xor_sync(~0u, ks.y, o);
    ks.z += __shfl_xor_sync(~0u, ks.z, o), ks.w += __shfl_xor_sync(~0u, ks.w, o);
    qs.x += __shfl_xor_sync(~0u, qs.x, o), qs.y += __shfl_xor_sync(~0u, qs.y, o);
    qs.z += __shfl_xor_sync(~0u, qs.z, o), qs.w += __shfl_xor_sync(~0u, qs.w, o);
  }
  if (lane < 8) {
    *reinterpret_cast<float4*>(&s_part[warp][0][col]) = ks;
    *reinterpret_cast<float4*>(&s_part[warp][1][col]) = qs;
  }
  __syncthreads();
  ks = qs = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float4 x = *reinterpret_cast<const float4*>(&s_part[w][0][col]);
    const float4 y = *reinterpret_cast<const float4*>(&s_part[w][1][col]);
    ks.x += x.x, ks.y += x.y, ks.z += x.z, ks.w += x.w;
    qs.x += y.x, qs.y += y.y, qs.z += y.z, qs.w += y.w;
  }
  const float4 u = make_float4(beta * fmaf(-g, ks.x, v[0]), beta * fmaf(-g, ks.y, v[1]), beta * fmaf(-g, ks.z, v[2]),
                               beta * fmaf(-g, ks.w, v[3]));
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    *reinterpret_cast<float4*>(state + (int64_t)i * D) = make_float4(fmaf(kr[i], u.x, g * S[i].x), fmaf(kr[i], u.y, g * S[i].y),
                                                                      fmaf(kr[i], u.z, g * S[i].z), fmaf(kr[i], u.w, g * S[i].w));
  if (tid < 8) {
    const float kq = s_kq;
    const float o[4] = {fmaf(kq, u.x, g * qs.x), fmaf(kq, u.y, g * qs.y), fmaf(kq, u.z, g * qs.z), fmaf(kq, u.w, g * qs.w)};
    kv::store4(reinterpret_cast<T*>(p.out.at(token, h)) + col0 + col, o);
  }
}

// Runs of tokens, one after the other, eight staged at a time; one barrier a token.  (Four tokens a pass, with their u from
// one another's products, took fewer instructions and barriers but twice the registers: eight runs of up to 5 fp32 tokens
// 20 us against 14, 16 runs of 33 154 against 129.)

constexpr int kStepTokens = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kStepThreads) gdn_run_kernel(const RuleArgs p) {
  constexpr int kSlices = D / kStepCols, kRows = D / 16;
  __shared__ __align__(16) float s_k[kStepTokens][D], s_q[kStepTokens][D], s_v[kStepTokens][kStepCols];
  __shared__ float s_g[kStepTokens], s_beta[kStepTokens], s_kq[kStepTokens];
  __shared__ __align__(16) float s_part[2][4][2][kStepCols];
  const bool last = p.beside && blockIdx.x == gridDim.x - 1;
  if (!p.beside) grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int slice = blockIdx.x % kSlices, h = blockIdx.x / kSlices % p.v_heads;
  const int64_t r = blockIdx.x / kSlices / p.v_heads;
  const Request req = read_request(p.s, r, p.max_new);
  if (req.status && tid == 0) gdn_flag(req.status);
  if (!req.count || req.count > p.short_most) {
    if (last) grid_dependency_wait();
    return;
  }
  const int hk = h / (p.v_heads / p.k_heads);
  const int row0 = (warp * 4 + lane / 8) * kRows, col = (lane % 8) * 4, col0 = slice * kStepCols;
  float* state = p.state + ((int64_t)req.slot * p.v_heads + h) * D * D + (int64_t)row0 * D + col0 + col;
  float4 S[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    S[i] = req.fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(state + (int64_t)i * D);
  int turn = 0;
  for (int32_t t0 = 0; t0 < req.count; t0 += kStepTokens) {
    const int n = min(kStepTokens, req.count - t0);
    __syncthreads();  // the tokens before are done with
    for (int e = tid; e < kStepTokens * (D / 8); e += kStepThreads) {
      const int t = e / (D / 8), vec = e % (D / 8);
      const int64_t token = (int64_t)req.first + t0 + t;
      float kk[8], qq[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) kk[i] = qq[i] = 0.f;
      if (t < n) {
        kv::load8(reinterpret_cast<const T*>(p.k.at(token, hk)) + 8 * vec, kk);
        kv::load8(reinterpret_cast<const T*>(p.q.at(token, hk)) + 8 * vec, qq);
      }
      float k2 = 0.f, q2 = 0.f, kq = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) k2 = fmaf(kk[i], kk[i], k2), q2 = fmaf(qq[i], qq[i], q2), kq = fmaf(kk[i], qq[i], kq);
#pragma unroll
      for (int o = D / 16; o; o >>= 1) {
        k2 += __shfl_xor_sync(~0u, k2, o);
        q2 += __shfl_xor_sync(~0u, q2, o);
        kq += __shfl_xor_sync(~0u, kq, o);
      }
      const float fk = p.unit ? 1.0f / sqrtf(k2 + p.eps) : 1.f, fq = p.unit ? p.scale / sqrtf(q2 + p.eps) : p.scale;
#pragma unroll
      for (int i = 0; i < 8; ++i) kk[i] *= fk, qq[i] *= fq;
      kv::store8(&s_k[t][8 * vec], kk);
      kv::store8(&s_q[t][8 * vec], qq);
      if (vec == 0) s_kq[t] = kq * fk * fq;
    }
    for (int e = tid; e < kStepTokens * kStepCols; e += kStepThreads) {
      const int t = e / kStepCols, c = e % kStepCols;
      if (t < n)
        s_v[t][c] = kv::to_float(reinterpret_cast<const T*>(p.v.at((int64_t)req.first + t0 + t, h))[col0 + c]);
    }
    if (tid < n) {
      const int64_t token = (int64_t)req.first + t0 + tid;
      const float a = kv::to_float(reinterpret_cast<const T*>(p.a + token * p.a_stride)[h]);
      const float b = kv::to_float(reinterpret_cast<const T*>(p.b + token * p.b_stride)[h]);
      s_g[tid] = expf(p.gates ? log_decay(a, p.a_log[h], p.dt_bias[h]) : a);
      s_beta[tid] = p.gates ? sigmoid(b) : b;
    }
    __syncthreads();
    for (int t = 0; t < n; ++t, turn ^= 1) {
      float kr[kRows], qr[kRows];
#pragma unroll
      for (int i = 0; i < kRows; i += 4) kv::load4(&s_k[t][row0 + i], kr + i), kv::load4(&s_q[t][row0 + i], qr + i);
      float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), qs = ks;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        ks.x = fmaf(kr[i], S[i].x, ks.x), ks.y = fmaf(kr[i], S[i].y, ks.y);
        ks.z = fmaf(kr[i], S[i].z, ks.z), ks.w = fmaf(kr[i], S[i].w, ks.w);
        qs.x = fmaf(qr[i], S[i].x, qs.x), qs.y = fmaf(qr[i], S[i].y, qs.y);
        qs.z = fmaf(qr[i], S[i].z, qs.z), qs.w = fmaf(qr[i], S[i].w, qs.w);
      }
#pragma unroll
      for (int o = 8; o < 32; o *= 2) {
        ks.x += __shfl_xor_sync(~0u, ks.x, o), ks.y += __shfl_xor_sync(~0u, ks.y, o);
        ks.z += __shfl_xor_sync(~0u, ks.z, o), ks.w += __shfl_xor_sync(~0u, ks.w, o);
        qs.x += __shfl_xor_sync(~0u, qs.x, o), qs.y += __shfl_xor_sync(~0u, qs.y, o);
        qs.z += __shfl_xor_sync(~0u, qs.z, o), qs.w += __shfl_xor_sync(~0u, qs.w, o);
      }
      if (lane < 8) {
        *reinterpret_cast<float4*>(&s_part[turn][warp][0][col]) = ks;
        *reinterpret_cast<float4*>(&s_part[turn][warp][1][col]) = qs;
      }
      __syncthreads();
      ks = qs = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&s_part[turn][w][0][col]);
        const float4 y = *reinterpret_cast<const float4*>(&s_part[turn][w][1][col]);
        ks.x += x.x, ks.y += x.y, ks.z += x.z, ks.w += x.w;
        qs.x += y.x, qs.y += y.y, qs.z += y.z, qs.w += y.w;
      }
      const float g = s_g[t], beta = s_beta[t], kq = s_kq[t];
      float4 u = *reinterpret_cast<const float4*>(&s_v[t][col]);
      u.x = beta * fmaf(-g, ks.x, u.x), u.y = beta * fmaf(-g, ks.y, u.y);
      u.z = beta * fmaf(-g, ks.z, u.z), u.w = beta * fmaf(-g, ks.w, u.w);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        S[i].x = fmaf(kr[i], u.x, g * S[i].x), S[i].y = fmaf(kr[i], u.y, g * S[i].y);
        S[i].z = fmaf(kr[i], u.z, g * S[i].z), S[i].w = fmaf(kr[i], u.w, g * S[i].w);
      }
      if (tid < 8) {
        const float o[4] = {fmaf(kq, u.x, g * qs.x), fmaf(kq, u.y, g * qs.y), fmaf(kq, u.z, g * qs.z),
                            fmaf(kq, u.w, g * qs.w)};
        kv::store4(reinterpret_cast<T*>(p.out.at((int64_t)req.first + t0 + t, h)) + col0 + col, o);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) *reinterpret_cast<float4*>(state + (int64_t)i * D) = S[i];
  if (last) grid_dependency_wait();
}

template <typename T>
static cudaError_t launch_step(const RuleArgs& a, int head_dim, cudaStream_t st) {
  const int64_t grid = a.s.requests * a.v_heads * (head_dim / kStepCols);
  const auto k = a.max_new <= 1 ? (head_dim == 64 ? gdn_step_kernel<T, 64> : gdn_step_kernel<T, 128>)
                                : (head_dim == 64 ? gdn_run_kernel<T, 64> : gdn_run_kernel<T, 128>);
  return launch_dependent(k, dim3((unsigned)grid), dim3(kStepThreads), 0, st, a);
}

}  // namespace gdn

int read_gdn_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, gdn::g_gdn_status, sizeof(v)) != cudaSuccess) return -1;
  if (clear && v) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(gdn::g_gdn_status, &z, sizeof(z)) != cudaSuccess) return -1;
  }
  const int w = gdn::prompt_status(clear);
  return w < 0 ? -1 : (int)v | w;
}

static int check_requests(const int32_t* q_start, const int32_t* kv_len, const int32_t* slot, int64_t requests,
                          int64_t tokens, const void* state, int64_t slots) {
  // (a token's index, and that of a few past the last, fits 32 bits)
  if (requests < 1 || requests > 0x7fffffffll - 1 || tokens < 0 || tokens > 0x7fffffffll - gdn::kChunk || slots < 1 ||
      slots > 0x7fffffffll)
    return fail(KQ_ERR_SHAPE, "requests = %lld, tokens = %lld, slots = %lld", (long long)requests, (long long)tokens,
                (long long)slots);
  if (!q_start || !slot || !state) return fail(KQ_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned16(q_start) || !aligned16(kv_len) || !aligned16(slot) || !aligned16(state))
    return fail(KQ_ERR_ALIGNMENT, "q_start, kv_len, slot or state not 16-byte aligned");
  return KQ_OK;
}

// Whether rows of `wide` bytes of the two views share a byte; side by side in rows of one stride they do not.
static bool overlap(const gdn::Rows& x, const gdn::Rows& y, int64_t rows, int64_t wide) {
  const char* x1 = x.data + (rows - 1) * x.token_stride + wide;
  const char* y1 = y.data + (rows - 1) * y.token_stride + wide;
  if (x.data >= y1 || y.data >= x1) return false;
  const int64_t stride = x.token_stride;
  if (rows == 1 || stride != y.token_stride || stride == 0) return true;
  const int64_t off = ((y.data - x.data) % stride + stride) % stride;
  return off < wide || off + wide > stride;
}

static int check_rule(const kq_gdn_rule* p) {
  if (!p) return fail(KQ_ERR_INVALID_ARG, "p is NULL");
  if (p->reserved != 0 || (p->unit != 0 && p->unit != 1) || (p->gates != 0 && p->gates != 1))
    return fail(KQ_ERR_INVALID_ARG, "unit and gates are 0 or 1, reserved is 0");
  if (p->head_dim != 64 && p->head_dim != 128) return fail(KQ_ERR_SHAPE, "head_dim = %d (64 or 128)", p->head_dim);
  if (p->k_heads < 1 || p->v_heads < 1 || p->v_heads > 4096 || p->v_heads % p->k_heads)
    return fail(KQ_ERR_SHAPE, "%d value heads on %d key heads", p->v_heads, p->k_heads);
  if (!(p->eps >= 0.f && std::isfinite(p->eps)) || !std::isfinite(p->scale))
    return fail(KQ_ERR_INVALID_ARG, "eps is negative, or eps or scale not finite");
  if (p->gates != (p->a_log != nullptr) || p->gates != (p->dt_bias != nullptr))
    return fail(KQ_ERR_INVALID_ARG, "a_log and dt_bias come with gates = 1, and only then");
  if ((p->a_log && !aligned16(p->a_log)) || (p->dt_bias && !aligned16(p->dt_bias)))
    return fail(KQ_ERR_ALIGNMENT, "a_log or dt_bias not 16-byte aligned");
  return KQ_OK;
}

static int check_sizes(const kq_gdn_rule* p, int64_t requests, int64_t tokens, int64_t max_new) {
  const int64_t most = 0x7fffffffll / (4 * p->v_heads);  // CTAs
  if (requests < 1 || requests > most / 2 || tokens < 0 || tokens / gdn::kChunk > most / 2 || max_new < 0)
    return fail(KQ_ERR_SHAPE, "%lld requests, %lld tokens, max_new = %lld, %d heads", (long long)requests, (long long)tokens,
                (long long)max_new, p->v_heads);
  return KQ_OK;
}

// Whether runs longer than kShortRun tokens go in chunks on the tensor cores: what is solved and summed in fp16 parts is
// bounded where keys have unit length and strengths and decays are at most 1.  (A prompt of 6000 tokens of 16/48 heads of 128 f16 in
// chunks 0.30 ms, with unit = 0 or gates = 0 token by token 3.6; of 4/12 heads of 128 0.26, of 64 2.8.)
static bool in_chunks(const kq_gdn_rule* p, int64_t max_new) {
  return p->head_dim == 128 && p->unit && p->gates && max_new > gdn::kShortRun;
}

}  // namespace kq

using namespace kq;

extern "C" {

int kq_causal_conv(const kq_conv* p, int dtype, const kq_heads* x, const int32_t* d_q_start, const int32_t* d_kv_len,
                   const int32_t* d_slot, int64_t requests, int64_t tokens, void* d_state, int64_t slots,
                   const kq_heads* out, void* stream) {
  clear_error();
  if (int s = check_dtype(dtype)) return s;
  if (!p || !p->weight) return fail(KQ_ERR_INVALID_ARG, "p or its weight is NULL");
  if (p->reserved != 0 || (p->silu != 0 && p->silu != 1)) return fail(KQ_ERR_INVALID_ARG, "silu is 0 or 1, reserved is 0");
  if (p->channels < 8 || p->channels % 8 || p->channels > (1 << 20) || p->width < 2 || p->width > 4)
    return fail(KQ_ERR_SHAPE, "%d channels (a multiple of 8 up to 2^20), width %d (2 to 4)", p->channels, p->width);
  if (!aligned16(p->weight) || !aligned16(p->bias)) return fail(KQ_ERR_ALIGNMENT, "weight or bias not 16-byte aligned");
  if (int s = check_requests(d_q_start, d_kv_len, d_slot, requests, tokens, d_state, slots)) return s;
  if (tokens == 0) return KQ_OK;
  if (int s = check_heads(x, "x", dtype)) return s;
  if (int s = check_out_rows(out, "out", dtype, tokens, 1, p->channels)) return s;
  const int size = dtype == KQ_F32 ? 4 : 2;
  gdn::ConvArgs a{};
  a.x = gdn::rows_of(x, size), a.out = gdn::rows_of(out, size);
  if (overlap(a.x, a.out, tokens, (int64_t)p->channels * size)) return fail(KQ_ERR_INVALID_ARG, "out overlaps x");
  a.s = gdn::Requests{d_q_start, d_kv_len, d_slot, requests, tokens, slots};
  a.state = static_cast<char*>(d_state), a.weight = p->weight, a.bias = p->bias;
  a.channels = p->channels, a.silu = p->silu;
  // Pieces as short as keep the warps (4256 are resident) to a wave or so, for the inputs before a piece are read again; longer
  // ones where there are many waves (one request's tokens of 10240 bf16 channels with pieces of 8, 16, 32, 64: 1000 13, 12, 14,
  // 13 us; 2000 25, 21, 21, 26; 4000 49, 39, 37, 40; 8000 93, 74, 66, 66; 20000 -, 173, 154, 147).
  const int64_t groups = (p->channels + 32 * gdn::kConvWide - 1) / (32 * gdn::kConvWide);
  const auto warps = [&](int piece) { return (requests + (tokens + piece - 1) / piece) * groups; };
  a.piece = 8;
  while (a.piece < 32 && warps(a.piece) > 6000) a.piece *= 2;
  if (a.piece == 32 && warps(32) > 14000) a.piece = 64;
  a.windows = (tokens + a.piece - 1) / a.piece;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  KQ_CUDA_TRY(dtype == KQ_F32   ? gdn::launch_conv<float>(a, p->width, st)
              : dtype == KQ_F16 ? gdn::launch_conv<__half>(a, p->width, st)
                                : gdn::launch_conv<__nv_bfloat16>(a, p->width, st));
  return KQ_OK;
}

size_t kq_gdn_workspace_bytes(const kq_gdn_rule* p, int dtype, int64_t requests, int64_t tokens, int64_t max_new) {
  clear_error();
  if (check_dtype(dtype) || check_rule(p) || check_sizes(p, requests, tokens, max_new)) return 0;
  return in_chunks(p, max_new) ? (size_t)gdn::prompt_workspace(p->k_heads, p->v_heads, requests, tokens, dtype) : 0;
}

int kq_gdn(const kq_gdn_rule* p, int dtype, const kq_heads* q, const kq_heads* k, const kq_heads* v, const void* d_a,
           int64_t a_stride, const void* d_b, int64_t b_stride, const int32_t* d_q_start, const int32_t* d_kv_len,
           const int32_t* d_slot, int64_t requests, int64_t tokens, int64_t max_new, float* d_state, int64_t slots,
           const kq_heads* out, void* d_ws, size_t ws_bytes, void* stream) {
  clear_error();
  if (int s = check_dtype(dtype)) return s;
  if (int s = check_rule(p)) return s;
  if (int s = check_requests(d_q_start, d_kv_len, d_slot, requests, tokens, d_state, slots)) return s;
  if (int s = check_sizes(p, requests, tokens, max_new)) return s;
  if (a_stride < 0 || b_stride < 0)
    return fail(KQ_ERR_SHAPE, "a_stride = %lld, b_stride = %lld", (long long)a_stride, (long long)b_stride);
  if (tokens == 0) return KQ_OK;
  if (!d_a || !d_b) return fail(KQ_ERR_INVALID_ARG, "a or b is NULL");
  const int size = dtype == KQ_F32 ? 4 : 2;
  if ((uintptr_t)d_a % size || (uintptr_t)d_b % size) return fail(KQ_ERR_ALIGNMENT, "a or b not aligned to its type");
  if (int s = check_heads(q, "q", dtype)) return s;
  if (int s = check_heads(k, "k", dtype)) return s;
  if (int s = check_heads(v, "v", dtype)) return s;
  if (int s = check_out_rows(out, "out", dtype, tokens, p->v_heads, p->head_dim)) return s;
  gdn::RuleArgs a{};
  a.q = gdn::rows_of(q, size), a.k = gdn::rows_of(k, size), a.v = gdn::rows_of(v, size), a.out = gdn::rows_of(out, size);
  a.a = static_cast<const char*>(d_a), a.b = static_cast<const char*>(d_b);
  a.a_stride = a_stride * size, a.b_stride = b_stride * size;
  a.s = gdn::Requests{d_q_start, d_kv_len, d_slot, requests, tokens, slots};
  a.state = d_state, a.a_log = p->a_log, a.dt_bias = p->dt_bias, a.max_new = max_new;
  a.k_heads = p->k_heads, a.v_heads = p->v_heads, a.unit = p->unit, a.gates = p->gates, a.eps = p->eps, a.scale = p->scale;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  a.short_most = 0x7fffffff;
  const bool chunks = in_chunks(p, max_new);
  if (chunks) {
    const size_t need = gdn::prompt_workspace(p->k_heads, p->v_heads, requests, tokens, dtype);
    if (!d_ws || ws_bytes < need)
      return fail(KQ_ERR_WORKSPACE, "workspace of %zu bytes, %zu are needed", d_ws ? ws_bytes : (size_t)0, need);
    if (!aligned16(d_ws)) return fail(KQ_ERR_ALIGNMENT, "workspace not 16-byte aligned");
  }
  // a head's CTAs read q and k when others may have put their outputs away
  for (const kq_heads* from : {q, k})
    if (rows_overlap(from, p->k_heads, out, p->v_heads, tokens, p->head_dim, dtype)) return fail(KQ_ERR_INVALID_ARG, "out overlaps q or k");
  if (!same_view(v, out, tokens, p->v_heads) && rows_overlap(v, p->v_heads, out, p->v_heads, tokens, p->head_dim, dtype))
    return fail(KQ_ERR_INVALID_ARG, "out overlaps v without being its view");
  if (chunks) {
    a.short_most = requests == 1 ? 0 : gdn::kShortRun;
    KQ_CUDA_TRY(gdn::launch_prompt(a, dtype, d_ws, st));
    if (requests == 1) return KQ_OK;
    a.beside = 1;
  }
  KQ_CUDA_TRY(dtype == KQ_F32   ? gdn::launch_step<float>(a, p->head_dim, st)
              : dtype == KQ_F16 ? gdn::launch_step<__half>(a, p->head_dim, st)
                                : gdn::launch_step<__nv_bfloat16>(a, p->head_dim, st));
  return KQ_OK;
}

}  // extern "C"
