// What a step does around its attention: slot maps from the requests' lengths,
// the norms and rotation of query and key heads, and the cache write in 4 bits.
// (The cache's layout: kq_kv.cuh; "Kipp Benchmarks": quantized KV rows,
// block-table indirection.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_kv.cuh"

namespace kq {
namespace kv {

__device__ unsigned int g_kv_status = 0;
__device__ __forceinline__ void kv_flag(int status) { atomicOr(&g_kv_status, 1u << status); }

// ---------------------------------------------------------------------------
// Slot maps
// ---------------------------------------------------------------------------

// A token's page needs the number of pages that earlier requests take from the
// free list: an exclusive sum over the requests.  Every CTA owns a range of
// tokens and runs the sum itself, kScan requests at a time, up to the chunk that
// ends its range (CTA 0 runs it to the end and writes the per-request outputs),
// so the whole map is one launch with no pass over intermediate sums.  A page
// is entered in the table by the one token that opens it.  Bound by latency: 90k
// tokens of 61 requests take 3.4 us beyond an empty launch (2048 tokens a CTA
// instead of 512 took 9.5), 256 requests of one token 1.4.
constexpr int kScanThreads = 256;
constexpr int kScan = 4 * kScanThreads;
constexpr int kMapTokens = 512;  // tokens of a CTA

struct SlotArgs {
  const int32_t *cached, *fresh, *free_pages;
  int32_t *table, *q_start, *kv_len, *positions, *slots, *used;
  int64_t requests, free_count, table_stride, tokens;
  int32_t page_size;
};

// Sum of counts, held at 2^31 - 1: lengths that no cache holds then pass the capacity instead of wrapping around it.
__device__ __forceinline__ int32_t sum_held(int32_t a, int32_t b) {
  return (int32_t)min((uint32_t)a + (uint32_t)b, 0x7fffffffu);
}

__global__ void __launch_bounds__(kScanThreads) slot_map_kernel(SlotArgs a) {
  __shared__ int32_t s_first[kScan + 1];  // first token of each request of the chunk
  __shared__ int32_t s_pages[kScan];      // pages taken before it
  __shared__ int32_t s_cached[kScan];
  __shared__ int2 s_warp[kScanThreads / 32];
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * kMapTokens, t1 = min(a.tokens, t0 + kMapTokens);
  const bool writer = blockIdx.x == 0;
  const int P = a.page_size;
  int32_t run_tokens = 0, run_pages = 0;
  bool range = false;
  for (int64_t base = 0; base < a.requests; base += kScan) {
    // four successive requests a thread
    int32_t c[4], n[4], need[4];
    int2 sum = make_int2(0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = base + 4 * tid + i;
      c[i] = r < a.requests ? a.cached[r] : 0;
      n[i] = r < a.requests ? a.fresh[r] : 0;
      if (c[i] < 0 || n[i] < 0 || c[i] > 0x7fffffff - n[i]) range = true;
      c[i] = max(c[i], 0);
      n[i] = min(max(n[i], 0), 0x7fffffff - c[i]);
      const int64_t end = (int64_t)c[i] + n[i];
      need[i] = (int32_t)((end + P - 1) / P - ((int64_t)c[i] + P - 1) / P);
      sum.x = sum_held(sum.x, n[i]);
      sum.y = sum_held(sum.y, need[i]);
    }
    int2 inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(~0u, inc.x, o), y = __shfl_up_sync(~0u, inc.y, o);
      if (lane >= o) inc.x = sum_held(inc.x, x), inc.y = sum_held(inc.y, y);
    }
    int2 earlier = make_int2(__shfl_up_sync(~0u, inc.x, 1), __shfl_up_sync(~0u, inc.y, 1));  // the warp's lanes before
    if (lane == 0) earlier = make_int2(0, 0);
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int2 before = make_int2(run_tokens, run_pages), total = before;
#pragma unroll
    for (int w = 0; w < kScanThreads / 32; ++w) {
      total.x = sum_held(total.x, s_warp[w].x), total.y = sum_held(total.y, s_warp[w].y);
      if (w + 1 == warp) before = total;
    }
    before.x = sum_held(before.x, earlier.x);
    before.y = sum_held(before.y, earlier.y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 4 * tid + i;
      s_first[j] = before.x;
      s_pages[j] = before.y;
      s_cached[j] = c[i];
      if (writer && base + j < a.requests) {
        a.q_start[base + j] = before.x;
        a.kv_len[base + j] = c[i] + n[i];
      }
      before.x = sum_held(before.x, n[i]);
      before.y = sum_held(before.y, need[i]);
    }
    if (tid == kScanThreads - 1) s_first[kScan] = before.x;
    __syncthreads();
    const int in_chunk = (int)min((int64_t)kScan, a.requests - base);
    // the CTA's tokens that belong to this chunk's requests
    const int64_t lo = max(t0, (int64_t)run_tokens), hi = min(t1, (int64_t)total.x);
    for (int64_t t = lo + tid; t < hi; t += kScanThreads) {
      int l = 0, h = in_chunk;  // the last request whose first token is not after t
      while (h - l > 1) {
        const int m = (l + h) >> 1;
        if (s_first[m] <= t) l = m; else h = m;
      }
      const int32_t pos = s_cached[l] + (int32_t)(t - s_first[l]);
      const int32_t old = (int32_t)(((int64_t)s_cached[l] + P - 1) / P), at = pos / P;
      int32_t* row = a.table + (base + l) * a.table_stride;
      int32_t page = -1;
      if (at >= a.table_stride) {
        range = true;
      } else if (at < old) {
        page = row[at];
      } else {
        const int64_t f = (int64_t)s_pages[l] + (at - old);
        if (f < a.free_count) page = a.free_pages[f]; else range = true;
        if (pos % P == 0) row[at] = page;
      }
      const int64_t slot = page < 0 ? -1 : (int64_t)page * P + pos % P;
      if (slot > 0x7fffffff) range = true;
      a.positions[t] = pos;
      a.slots[t] = slot > 0x7fffffff ? -1 : (int32_t)slot;
    }
    run_tokens = total.x;
    run_pages = total.y;
    if (!writer && run_tokens >= t1) break;
    __syncthreads();
  }
  if (writer && tid == 0) {
    a.q_start[a.requests] = run_tokens;
    a.used[0] = run_pages;
    if (run_tokens > a.tokens || run_tokens == 0x7fffffff) range = true;
  }
  for (int64_t t = max(t0, (int64_t)run_tokens) + tid; t < t1; t += kScanThreads) {
    a.positions[t] = 0;
    a.slots[t] = -1;
  }
  if (range) kv_flag(KQ_ERR_RANGE);
}

// ---------------------------------------------------------------------------
// Norm, rotation, cache write
// ---------------------------------------------------------------------------

struct View {
  void* data;
  int64_t token, head;  // strides in elements
};

struct QkArgs {
  View q, k, v, q_out, k_out;
  const float *q_weight, *k_weight, *rope;
  const int32_t *positions, *slots;
  int64_t rope_positions, tokens;
  int32_t q_heads, kv_heads, rope_dim, interleaved, norm;
  float eps;
  Cache cache;
};

// n with |n - a/d| <= 1/2, halves up: round-half-away(a / d) for a >= 0, d > 0.
// d is an fp16 value, so (n + 1/2) d is exact in fp32 for n < 16 and the two
// comparisons decide what the quotient's own rounding cannot.
__device__ __forceinline__ int round_ratio(float a, float d, float inv) {
  float n = floorf(fminf(a * inv, 15.f) + 0.5f);
  if (a >= (n + 0.5f) * d) n += 1.f;
  if (a < (n - 0.5f) * d) n -= 1.f;
  return (int)n;
}

// The four lanes of a 32-dimension group hold 8 values each: the group's scale
// (SCALE4: the first value of largest magnitude over -8, rounded to fp16) and
// this lane's eight codes, nibble j the j-th value.  The whole warp takes part.
//
// The codes come from the product with 1/d, rounded by adding 1.5 2^23 (+ 8:
// the low bits are then the code).  x - n d, exact but for its own rounding,
// shows whether n is beyond doubt, |x - n d| < |d| / 2; where it is not for
// some value of the warp (a tie, or a quotient that its rounding moved), all
// are decided by comparisons.  (Comparisons for every value made a prompt's
// cache write bound by instructions: 230 a lane against 90.)
__device__ __forceinline__ uint32_t quantize_group(const float (&x)[8], __half& scale) {
  float hi = x[0], lo = x[0];
  float2 none = make_float2(0.f, 0.f);  // 0 x: not 0 where x is not finite
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    hi = fmaxf(hi, fmaxf(x[i], x[i + 1]));
    lo = fminf(lo, fminf(x[i], x[i + 1]));
    none = fma2(make_float2(x[i], x[i + 1]), make_float2(0.f, 0.f), none);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
    lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
  }
  const uint32_t strange = __ballot_sync(~0u, !(none.x + none.y == 0.f));
  const bool bad = strange >> (threadIdx.x & 28) & 15u;
  float m = hi > -lo ? hi : lo;
  const bool tie = hi == -lo && hi > 0.f;
  if (__any_sync(~0u, tie)) {  // both signs: the first one's counts
    int at = 64;
    float v = 0.f;
#pragma unroll
    for (int i = 7; i >= 0; --i)
      if (fabsf(x[i]) == hi) at = (threadIdx.x & 3) * 8 + i, v = x[i];
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const int b = __shfl_xor_sync(~0u, at, o);
      const float w = __shfl_xor_sync(~0u, v, o);
      if (b < at) at = b, v = w;
    }
    if (tie) m = v;
  }
  scale = __float2half_rn(m * -0.125f);
  if (bad) scale = __ushort_as_half((unsigned short)0x7FFF);
  const float d = __half2float(scale), mag = fabsf(d);
  const bool plain = mag > 0.f && mag <= 65504.f;
  const float inv = plain ? __fdividef(1.f, d) : 0.f, half = plain ? 0.5f * mag : 1.f, by = plain ? -d : 0.f;
  constexpr float kMagic = 12582912.f + 8.f;
  uint32_t w = 0;
  bool doubt = mag < 6.104e-5f;  // a subnormal scale may leave quotients beyond -8
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {
    const float2 v = plain ? make_float2(x[i], x[i + 1]) : make_float2(0.f, 0.f);
    const float2 t = fma2(v, make_float2(inv, inv), make_float2(kMagic, kMagic));
    const float2 e = fma2(add2(t, make_float2(-kMagic, -kMagic)), make_float2(by, by), v);
    doubt |= !(fabsf(e.x) < half) || !(fabsf(e.y) < half);
    const uint32_t q0 = min(__float_as_uint(t.x) & 31u, 15u), q1 = min(__float_as_uint(t.y) & 31u, 15u);
    w = w << 8 | q1 << 4 | q0;
  }
  if (__any_sync(~0u, doubt) && plain) {
    const float up = fabsf(inv);
    w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = round_ratio(fabsf(x[i]), mag, up);
      const int q = (x[i] < 0.f) != (d < 0.f) ? 8 - n : 8 + n;
      w |= (uint32_t)min(max(q, 0), 15) << (4 * i);
    }
  }
  if (!plain && mag != 0.f) kv_flag(bad ? KQ_ERR_NONFINITE : KQ_ERR_RANGE);
  return w;
}

// A head row is spread over D / 8 lanes ("row group"), eight dimensions a lane.
constexpr int kQkThreads = 256;
enum Mode { kNorm, kAppendEach, kAppendGranules };

// The whole warp takes part; lanes without a row pass zeros.
template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o, kLanes);
  return v;
}
__device__ __forceinline__ void set2(float* p, float2 v) { p[0] = v.x, p[1] = v.y; }
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float u = a;
  a = fmaf(u, c, -b * s);
  b = fmaf(b, c, u * s);
}
// Whether the token's position lies in the table; `entry` is its row.
__device__ __forceinline__ bool rope_row(const QkArgs& a, int64_t t, bool report, const float*& entry) {
  const int32_t pos = a.positions[t];
  if (pos < 0 || pos >= a.rope_positions) {
    if (report) kv_flag(KQ_ERR_RANGE);
    return false;
  }
  entry = a.rope + (int64_t)pos * a.rope_dim;
  return true;
}

// Query rows (and key rows that are not quantized): kHeads heads of one token a
// row group, all loaded before the first is reduced and held as they came: bound
// by the bytes of the rows, so what counts is how many are on their way (four
// heads, held in fp32 by 24 warps an SM, moved 3.4 TB/s).  A lane holds four
// dimensions and their four partners in the rotation (what is not rotated:
// eight in a row), so that rotating takes no shuffles and half the table loads.
// 4099 tokens of 28 heads of 256 in bf16: 24 us, 4.9 TB/s (35 us with eight
// dimensions in a row, shuffles and rows held in fp32).
template <typename T, int D, int kHeads>
__device__ __forceinline__ void norm_rows(const QkArgs& a, const View& in, const View& out, const float* weight, int heads,
                                          int64_t t0, int h0) {
  constexpr int kLanes = D / 8;
  const int row = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const int64_t t = t0 + row;
  const bool live = t < a.tokens;
  const int turning = a.rope_dim / 8, n = live ? min(kHeads, heads - h0) : 0;
  const bool turns = l < turning, split = turns && !a.interleaved;
  const int ea = split ? 4 * l : 8 * l, eb = split ? a.rope_dim / 2 + 4 * l : 8 * l + 4;
  const T* src = static_cast<const T*>(in.data) + t * in.token + h0 * in.head;
  Raw<T, 4> xa[kHeads], xb[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    xa[i].clear(), xb[i].clear();
    if (i < n) xa[i].load(src + i * in.head + ea), xb[i].load(src + i * in.head + eb);
  }
  float w[8], c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {};
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = 1.f;
  if (weight) load4(weight + ea, &w[0]), load4(weight + eb, &w[4]);
  bool held = true;
  if (a.rope_dim && live) {
    const float* entry = nullptr;
    held = rope_row(a, t, l == 0, entry);
    if (held && turns) load4(entry + 4 * l, c), load4(entry + a.rope_dim / 2 + 4 * l, s);
  }
  // the rows' sums side by side: their shuffles overlap
  float r[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    float v[8];
    xa[i].get(v), xb[i].get(v + 4);
    float2 ss = mul2(make_float2(v[0], v[1]), make_float2(v[0], v[1]));
#pragma unroll
    for (int j = 2; j < 8; j += 2) ss = fma2(make_float2(v[j], v[j + 1]), make_float2(v[j], v[j + 1]), ss);
    r[i] = ss.x + ss.y;
  }
  if (a.norm) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < kHeads; ++i) r[i] += __shfl_xor_sync(~0u, r[i], o, kLanes);
    }
  }
  T* dst = static_cast<T*>(out.data) + t * out.token + h0 * out.head;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (i >= n) break;
    const float f = a.norm ? rsqrtf(r[i] * (1.f / D) + a.eps) : 1.f;
    float v[8];
    xa[i].get(v), xb[i].get(v + 4);
    // weight, rotation, and the norm's factor last: it is common to a row
#pragma unroll
    for (int j = 0; j < 8; j += 2) set2(v + j, mul2(make_float2(v[j], v[j + 1]), make_float2(w[j], w[j + 1])));
    if (split) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float2 p = make_float2(v[j], v[j + 1]), q = make_float2(v[4 + j], v[5 + j]);
        const float2 cc = make_float2(c[j], c[j + 1]), sn = make_float2(s[j], s[j + 1]);
        set2(v + j, fma2(p, cc, mul2(make_float2(-q.x, -q.y), sn)));
        set2(v + 4 + j, fma2(q, cc, mul2(p, sn)));
      }
    } else if (turns) {
#pragma unroll
      for (int j = 0; j < 4; ++j) turn(v[2 * j], v[2 * j + 1], c[j], s[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) set2(v + j, mul2(make_float2(v[j], v[j + 1]), make_float2(f, f)));
    if (!held) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
    store4(dst + i * out.head + ea, v), store4(dst + i * out.head + eb, v + 4);
  }
}

// Eight successive dimensions a lane of a key row (normed and rotated) or a value row (as it is) in fp32, for quantizing.
template <typename T, int D>
__device__ __forceinline__ Raw<T, 8> load_row(const QkArgs& a, bool key, int64_t t, int h, bool live) {
  const View& in = key ? a.k : a.v;
  Raw<T, 8> raw;
  raw.clear();
  if (live) raw.load(static_cast<const T*>(in.data) + t * in.token + h * in.head + 8 * (threadIdx.x % (D / 8)));
  return raw;
}
// entry: the token's row of the rotation table; NULL: outside the table (or no rotation).
template <typename T, int D>
__device__ __forceinline__ void cache_row(const QkArgs& a, bool key, const float* entry, const Raw<T, 8>& raw, float (&x)[8]) {
  constexpr int kLanes = D / 8;
  const int l = threadIdx.x % kLanes, e0 = 8 * l, half_dim = a.rope_dim / 2;
  raw.get(x);
  if (!key) return;  // the same for the whole warp
  float r = 1.f;
  if (a.norm) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    r = rsqrtf(row_sum<kLanes>(ss) * (1.f / D) + a.eps);
  }
  if (a.k_weight) {
    float w[8];
    load8(a.k_weight + e0, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= w[j];
  }
  const bool held = entry || !a.rope_dim;
  if (a.rope_dim) {
    const bool turns = e0 < a.rope_dim, reads = entry && turns;
    if (a.interleaved) {
      if (reads) {
        float c[4], s[4];
        load4(entry + 4 * l, c), load4(entry + half_dim + 4 * l, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) turn(x[2 * j], x[2 * j + 1], c[j], s[j]);
      }
    } else {
      const bool low = e0 < half_dim;
      const int i0 = low ? e0 : e0 - half_dim, partner = turns ? (low ? l + half_dim / 8 : l - half_dim / 8) : l;
      float c[8], s[8];
      if (reads) load8(entry + i0, c), load8(entry + half_dim + i0, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float other = __shfl_sync(~0u, x[j], partner, kLanes);
        if (reads) x[j] = low ? fmaf(x[j], c[j], -other * s[j]) : fmaf(x[j], c[j], other * s[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = held ? x[j] * r : 0.f;
}

// A lane's codes and (one lane of four) its group's scale, at `granule`.
template <int D>
__device__ __forceinline__ void put_row(uint8_t* granule, int token, bool key, uint32_t codes, __half scale) {
  using L = Layout<D>;
  const int l = threadIdx.x % (D / 8);
  if (key) {
    *reinterpret_cast<uint32_t*>(granule + L::key_word(token, l)) = codes;
  } else {
    *reinterpret_cast<uint16_t*>(granule + L::value_unit(token, 2 * l)) = (uint16_t)codes;
    *reinterpret_cast<uint16_t*>(granule + L::value_unit(token, 2 * l + 1)) = (uint16_t)(codes >> 16);
  }
  if (l % 4 == 0) *reinterpret_cast<__half*>(granule + L::key_scale(token, l / 4) + (key ? 0 : D)) = scale;
}
template <int D>
__device__ __forceinline__ uint8_t* granule_of(const Cache& c, int32_t slot, int h) {
  const int32_t page = slot / c.page_size, in_page = slot - page * c.page_size;
  return c.data + ((int64_t)page * c.kv_heads + h) * c.block_bytes +
         (int64_t)(in_page / kGranule) * Layout<D>::kBytes;
}
__device__ __forceinline__ int32_t slot_of(const QkArgs& a, int64_t t) {
  const int32_t slot = a.slots[t];
  if (slot < a.cache.pages * a.cache.page_size) return slot;
  kv_flag(KQ_ERR_RANGE);
  return -1;
}

// Keys and values of a window of 32 (or 16) tokens of one head.  Where the tokens are
// runs of successive slots (prompts), the rows are put together in shared memory
// as the granules that they fill and go out word by word in memory order; a word
// of two tokens' values of which one is not in the window, as half words.
// Straight to the cache a token's values are 32 two-byte stores.  8192 tokens of
// 8 key and 32 query heads of 128 in bf16: 58 us (3.0 TB/s; 86 before, straight
// and with 230 instructions to quantize a lane's values); what bounds it is the
// issue of instructions, 70% of the slots.
constexpr int kWindowGranules = 4;
template <int D>
constexpr int kWindow = D == 256 ? 16 : 32;

template <typename T, int D>
__device__ __forceinline__ void append_window(const QkArgs& a, int64_t t0, int h) {
  using L = Layout<D>;
  constexpr int kLanes = D / 8, kRows = kQkThreads / kLanes, W = kWindow<D>;
  constexpr int kEach = W / kRows;  // key rows, and value rows, of a row group
  __shared__ __align__(16) uint8_t image[kWindowGranules * L::kBytes];
  __shared__ __align__(16) float s_table[W * D];
  __shared__ int32_t s_slot[W], s_index[W], s_pos[W], s_first[kWindowGranules], s_count;
  __shared__ uint32_t s_mask[kWindowGranules];
  const int tid = threadIdx.x, row = tid / kLanes;
  // all that the window reads is on its way before any of it is used
  Raw<T, 8> keys[kEach], values[kEach];
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    const int64_t t = t0 + row + n * kRows;
    keys[n] = load_row<T, D>(a, true, t, h, t < a.tokens);
    values[n] = load_row<T, D>(a, false, t, h, t < a.tokens);
  }
  if (tid < kWindowGranules) s_mask[tid] = 0;
  __syncthreads();
  if (tid < 32) {
    const bool in = tid < W && t0 + tid < a.tokens;
    int32_t pos = in && a.rope_dim ? a.positions[t0 + tid] : -1;
    const int32_t slot = in ? slot_of(a, t0 + tid) : -1;
    if (pos >= a.rope_positions) pos = -1;
    if (slot >= 0 && a.rope_dim && pos < 0) kv_flag(KQ_ERR_RANGE);
    const int32_t granule = slot < 0 ? -1 : slot / kGranule;
    const int32_t before = __shfl_up_sync(~0u, granule, 1);
    const uint32_t starts = __ballot_sync(~0u, granule >= 0 && (tid == 0 || before != granule));
    const int index = __popc(starts & (0xFFFFFFFFu >> (31 - tid))) - 1;
    if (tid < W) s_slot[tid] = slot, s_index[tid] = index, s_pos[tid] = pos;
    if (tid == 0) s_count = __popc(starts);
    if (granule >= 0 && index < kWindowGranules) {
      atomicOr(&s_mask[index], 1u << (slot % kGranule));
      if (starts >> tid & 1u) s_first[index] = slot;
    }
  }
  __syncthreads();
  const int quarter = a.rope_dim / 4;  // of a table row, 16 bytes each
  for (int i = tid; i < W * quarter; i += kQkThreads) {
    const int in = i / quarter, at = i - in * quarter;
    if (s_pos[in] >= 0)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&s_table[in * a.rope_dim + 4 * at])),
                   "l"(a.rope + (int64_t)s_pos[in] * a.rope_dim + 4 * at)
                   : "memory");
  }
  const bool together = s_count <= kWindowGranules;
  auto put = [&](int n, bool key, const float* entry, const Raw<T, 8>& raw) {
    const int in = row + n * kRows;
    const int32_t slot = s_slot[in];
    float x[8];
    cache_row<T, D>(a, key, entry, raw, x);
    if (slot < 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;  // a skipped token's values ask nothing
    }
    __half scale;
    const uint32_t codes = quantize_group(x, scale);
    if (slot >= 0)
      put_row<D>(together ? image + s_index[in] * L::kBytes : granule_of<D>(a.cache, slot, h), slot % kGranule, key, codes,
                 scale);
  };
#pragma unroll
  for (int n = 0; n < kEach; ++n) put(n, false, nullptr, values[n]);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    const int in = row + n * kRows;
    put(n, true, s_pos[in] >= 0 ? &s_table[in * a.rope_dim] : nullptr, keys[n]);
  }
  if (!together) return;
  __syncthreads();
  for (int g = 0; g < s_count; ++g) {
    const uint32_t mask = s_mask[g];
    const uint8_t* src = image + g * L::kBytes;
    uint8_t* dst = granule_of<D>(a.cache, s_first[g], h);
    if (mask == 0xFFFFu) {
      for (int i = tid; i < L::kBytes / 16; i += kQkThreads)
        reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(src)[i];
      continue;
    }
    for (int i = tid; i < L::kBytes / 4; i += kQkThreads) {
      const uint32_t word = reinterpret_cast<const uint32_t*>(src)[i];
      const int byte = 4 * i;
      uint32_t have;  // bit 0: the low half's token is there, bit 1: the high half's
      if (byte < L::kValues) {
        have = (mask >> (byte % L::kKeySlab / (L::kSlabDim / 2)) & 1u) * 3u;
      } else if (byte < L::kKeyScales) {
        const int in = (byte - L::kValues) % L::kKeySlab;
        have = mask >> (in / L::kBlock * 8 + in % L::kBlock / (4 * L::kGroups) % 4 * 2) & 3u;
      } else {
        have = (mask >> ((byte - L::kKeyScales) % L::kScaleSlab / (2 * L::kGroups)) & 1u) * 3u;
      }
      if (have == 3u) {
        reinterpret_cast<uint32_t*>(dst)[i] = word;
      } else if (have) {
        reinterpret_cast<uint16_t*>(dst)[2 * i + (have >> 1)] = (uint16_t)(have & 2u ? word >> 16 : word);
      }
    }
  }
}

// CTAs [0, row_ctas): query rows (and, without a cache, key rows), kRows tokens
// of one chunk of kHeads heads each.  The others: keys and values into the
// cache, a row a row group or a window of tokens a CTA.
template <typename T, int D, int kHeads, Mode kMode>
__global__ void __launch_bounds__(kQkThreads) qk_kernel(QkArgs a, uint32_t row_ctas) {
  constexpr int kLanes = D / 8, kRows = kQkThreads / kLanes;
  grid_dependency_wait();
  allow_dependent_launch();
  const uint32_t along = (uint32_t)((a.tokens + kRows - 1) / kRows);
  uint32_t b = blockIdx.x;
  if (b < row_ctas) {
    const int chunk = b / along, q_chunks = (a.q_heads + kHeads - 1) / kHeads;
    const int64_t t0 = (int64_t)(b % along) * kRows;
    if (kMode != kNorm || chunk < q_chunks)
      norm_rows<T, D, kHeads>(a, a.q, a.q_out, a.q_weight, a.q_heads, t0, chunk * kHeads);
    else
      norm_rows<T, D, kHeads>(a, a.k, a.k_out, a.k_weight, a.kv_heads, t0, (chunk - q_chunks) * kHeads);
    return;
  }
  b -= row_ctas;
  if constexpr (kMode == kAppendEach) {
    const int y = b / along, h = y % a.kv_heads;
    const bool key = y < a.kv_heads;
    const int64_t t = (int64_t)(b % along) * kRows + threadIdx.x / kLanes;
    const int32_t slot = t < a.tokens ? slot_of(a, t) : -1;
    const float* entry = nullptr;
    if (key && slot >= 0 && a.rope_dim) rope_row(a, t, threadIdx.x % kLanes == 0, entry);
    float x[8];
    cache_row<T, D>(a, key, entry, load_row<T, D>(a, key, t, h, slot >= 0), x);
    if (slot < 0) {  // nothing is asked of a lane without a row (a norm with eps = 0 makes NaN of its zeros)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
    }
    __half scale;
    const uint32_t codes = quantize_group(x, scale);
    if (slot >= 0) put_row<D>(granule_of<D>(a.cache, slot, h), slot % kGranule, key, codes, scale);
  } else if constexpr (kMode == kAppendGranules) {
    const uint32_t windows = (uint32_t)((a.tokens + kWindow<D> - 1) / kWindow<D>);
    append_window<T, D>(a, (int64_t)(b % windows) * kWindow<D>, b / windows);
  }
}

// One row of one slot a row group: its codes' values in `T`.  8192 tokens of 8
// heads of 128 to fp16: 12 us, 3.5 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(kQkThreads) read_kernel(Cache c, const int32_t* slots, int64_t count, View k, View v) {
  using L = Layout<D>;
  constexpr int kLanes = D / 8, kRows = kQkThreads / kLanes;
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t item = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes;
  const int l = threadIdx.x % kLanes;
  if (item >= count * c.kv_heads) return;
  const int64_t t = item / c.kv_heads;
  const int h = (int)(item % c.kv_heads);
  int32_t slot = slots[t];
  if (slot >= c.pages * c.page_size) {
    if (l == 0) kv_flag(KQ_ERR_RANGE);
    slot = -1;
  }
  float kx[8] = {}, vx[8] = {};
  if (slot >= 0) {
    const int page = slot / c.page_size, in_page = slot - page * c.page_size, tok = in_page % kGranule;
    const uint8_t* g =
        c.data + ((int64_t)page * c.kv_heads + h) * c.block_bytes + (int64_t)(in_page / kGranule) * L::kBytes;
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(g + L::key_word(tok, l));
    const uint32_t vw = *reinterpret_cast<const uint16_t*>(g + L::value_unit(tok, 2 * l)) |
                        (uint32_t)*reinterpret_cast<const uint16_t*>(g + L::value_unit(tok, 2 * l + 1)) << 16;
    const float ks = __half2float(*reinterpret_cast<const __half*>(g + L::key_scale(tok, l / 4)));
    const float vs = __half2float(*reinterpret_cast<const __half*>(g + L::key_scale(tok, l / 4) + D));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      kx[j] = (float)((int)(kw >> (4 * j) & 15u) - 8) * ks;
      vx[j] = (float)((int)(vw >> (4 * j) & 15u) - 8) * vs;
    }
  }
  store8(static_cast<T*>(k.data) + t * k.token + h * k.head + 8 * l, kx);
  store8(static_cast<T*>(v.data) + t * v.token + h * v.head + 8 * l, vx);
}

template <typename T, int D, bool kAppend>
static cudaError_t launch_qk(const QkArgs& a, cudaStream_t st) {
  constexpr int kRows = kQkThreads / (D / 8);
  const int64_t along = (a.tokens + kRows - 1) / kRows;
  // Four heads a row group once that still fills the GPU, one below: 1024 tokens of 28 heads of 256 take 9.0 us with
  // four, 12.3 with one; 64 tokens 5.5 and 4.8.  (Eight held too many registers: 35 us against 29 for 4099 tokens.)
  constexpr int kMany = 4;
  const int64_t rows = a.tokens * (a.q_heads + (kAppend ? 0 : 1) * (int64_t)a.kv_heads);
  const int heads = rows >= kMany * 152 * 2 * kRows ? kMany : 1;
  const int64_t chunks = (a.q_heads + heads - 1) / heads + (kAppend ? 0 : (a.kv_heads + heads - 1) / heads);
  const int64_t row_ctas = along * chunks;
  // Windows from four CTAs an SM of them on: 2432 tokens of 8 heads of 128 take 28.8 us with their queries against 30.8 a
  // row a row group, 4096 tokens 43.0 against 47.2, but 1024 tokens 18.5 against 16.5 and 64 tokens 12.3 against 8.2.
  const int64_t windows = (a.tokens + kWindow<D> - 1) / kWindow<D> * a.kv_heads;
  const bool granules = kAppend && windows >= 4 * 152;
  const int64_t ctas = row_ctas + (kAppend ? (granules ? windows : along * 2 * a.kv_heads) : 0);
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  void (*k)(QkArgs, uint32_t);
  if constexpr (kAppend) {
    k = granules ? (heads > 1 ? qk_kernel<T, D, kMany, kAppendGranules> : qk_kernel<T, D, 1, kAppendGranules>)
                 : (heads > 1 ? qk_kernel<T, D, kMany, kAppendEach> : qk_kernel<T, D, 1, kAppendEach>);
  } else {
    k = heads > 1 ? qk_kernel<T, D, kMany, kNorm> : qk_kernel<T, D, 1, kNorm>;
  }
  return launch_dependent(k, dim3((unsigned)ctas), dim3(kQkThreads), 0, st, a, (uint32_t)row_ctas);
}

template <typename T, bool kAppend>
static cudaError_t launch_qk(int d, const QkArgs& a, cudaStream_t st) {
  return d == 64 ? launch_qk<T, 64, kAppend>(a, st)
                 : (d == 128 ? launch_qk<T, 128, kAppend>(a, st) : launch_qk<T, 256, kAppend>(a, st));
}

template <bool kAppend>
static cudaError_t launch_qk(int dtype, int d, const QkArgs& a, cudaStream_t st) {
  return dtype == KQ_F32 ? launch_qk<float, kAppend>(d, a, st)
                         : (dtype == KQ_F16 ? launch_qk<__half, kAppend>(d, a, st)
                                            : launch_qk<__nv_bfloat16, kAppend>(d, a, st));
}

template <typename T>
static cudaError_t launch_read(const Cache& c, int d, const int32_t* slots, int64_t n, View k, View v, cudaStream_t st) {
  const int64_t rows = kQkThreads / (d / 8), grid = (n * c.kv_heads + rows - 1) / rows;
  auto f = d == 64 ? read_kernel<T, 64> : (d == 128 ? read_kernel<T, 128> : read_kernel<T, 256>);
  return launch_dependent(f, dim3((unsigned)grid), dim3(kQkThreads), 0, st, c, slots, n, k, v);
}

static View view(const kq_heads* h) { return h ? View{h->data, h->token_stride, h->head_stride} : View{nullptr, 0, 0}; }

}  // namespace kv

int check_cache(const kq_kv_cache* c) {
  if (!c) return fail(KQ_ERR_INVALID_ARG, "cache is NULL");
  if (!c->data) return fail(KQ_ERR_INVALID_ARG, "NULL cache data");
  if (c->reserved != 0) return fail(KQ_ERR_INVALID_ARG, "reserved field of the cache is not 0");
  if (c->pages < 1 || c->kv_heads < 1 || kq_kv_block_bytes(c->page_size, c->head_dim) == 0)
    return fail(KQ_ERR_SHAPE, "cache of %lld pages of %d tokens, %d heads of %d (pages, heads >= 1, page_size a multiple of 16, head_dim 64, 128 or 256)",
                (long long)c->pages, c->page_size, c->kv_heads, c->head_dim);
  if (c->pages > 0x7fffffffll / c->page_size)
    return fail(KQ_ERR_SHAPE, "cache of %lld pages of %d tokens: slots pass 31 bits", (long long)c->pages, c->page_size);
  if (!aligned16(c->data)) return fail(KQ_ERR_ALIGNMENT, "cache not 16-byte aligned");
  return KQ_OK;
}

int check_heads(const kq_heads* h, const char* name, int dtype) {
  if (!h || !h->data) return fail(KQ_ERR_INVALID_ARG, "%s is NULL", name);
  const int64_t per = dtype == KQ_F32 ? 4 : 8;
  if (!aligned16(h->data)) return fail(KQ_ERR_ALIGNMENT, "%s not 16-byte aligned", name);
  if (h->token_stride < 0 || h->head_stride < 0) return fail(KQ_ERR_SHAPE, "negative stride of %s", name);
  if (h->token_stride % per || h->head_stride % per)
    return fail(KQ_ERR_ALIGNMENT, "strides of %s are not multiples of 16 bytes", name);
  return KQ_OK;
}

kv::Cache cache_view(const kq_kv_cache* c) {
  return kv::Cache{static_cast<uint8_t*>(c->data), kq_kv_block_bytes(c->page_size, c->head_dim), c->pages, c->page_size,
                   c->kv_heads};
}

int check_dtype(int dtype) {
  if (dtype != KQ_F32 && dtype != KQ_F16 && dtype != KQ_BF16) return fail(KQ_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  return KQ_OK;
}

static int check_qk(const kq_qk_norm* p, const int32_t* pos, int64_t tokens) {
  if (!p) return fail(KQ_ERR_INVALID_ARG, "p is NULL");
  if (p->reserved != 0 || (p->norm != 0 && p->norm != 1) || (p->interleaved != 0 && p->interleaved != 1))
    return fail(KQ_ERR_INVALID_ARG, "norm and interleaved are 0 or 1, reserved is 0");
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256)
    return fail(KQ_ERR_SHAPE, "head_dim = %d (64, 128 or 256)", p->head_dim);
  if (p->q_heads < 1 || p->kv_heads < 1 || p->q_heads > 4096 || p->kv_heads > 4096)
    return fail(KQ_ERR_SHAPE, "%d query and %d key heads (1 to 4096)", p->q_heads, p->kv_heads);
  if (p->rope_dim < 0 || p->rope_dim > p->head_dim || p->rope_dim % 16)
    return fail(KQ_ERR_SHAPE, "rope_dim = %d (a multiple of 16 up to head_dim)", p->rope_dim);
  if (p->norm && !(p->eps >= 0.f && std::isfinite(p->eps))) return fail(KQ_ERR_INVALID_ARG, "eps is negative or not finite");
  if (!p->norm && (p->q_weight || p->k_weight)) return fail(KQ_ERR_INVALID_ARG, "weights given without the norm");
  if (p->rope_dim) {
    if (!p->d_rope || !pos) return fail(KQ_ERR_INVALID_ARG, "rotation without a table or positions");
    if (p->rope_positions < 1) return fail(KQ_ERR_SHAPE, "rope_positions = %lld", (long long)p->rope_positions);
  }
  if ((p->q_weight && !aligned16(p->q_weight)) || (p->k_weight && !aligned16(p->k_weight)) ||
      (p->d_rope && !aligned16(p->d_rope)) || (pos && !aligned16(pos)))
    return fail(KQ_ERR_ALIGNMENT, "weights, table or positions not 16-byte aligned");
  if (tokens < 0 || tokens > 0x7fffffffll / 8192) return fail(KQ_ERR_SHAPE, "tokens = %lld", (long long)tokens);
  return KQ_OK;
}

static kv::QkArgs qk_args(const kq_qk_norm* p, const int32_t* pos, int64_t tokens) {
  kv::QkArgs a{};
  a.q_weight = p->q_weight, a.k_weight = p->k_weight, a.rope = p->d_rope;
  a.positions = pos, a.rope_positions = p->rope_positions, a.tokens = tokens;
  a.q_heads = p->q_heads, a.kv_heads = p->kv_heads, a.rope_dim = p->rope_dim, a.interleaved = p->interleaved;
  a.norm = p->norm, a.eps = p->eps;
  return a;
}

int read_kv_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, kv::g_kv_status, sizeof(v)) != cudaSuccess) return -1;
  if (clear && v) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(kv::g_kv_status, &z, sizeof(z)) != cudaSuccess) return -1;
  }
  return (int)v;
}

}  // namespace kq

using namespace kq;

extern "C" {

int64_t kq_kv_block_bytes(int32_t page_size, int32_t head_dim) {
  if (page_size < 16 || page_size % 16 || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return 0;
  return (int64_t)page_size * head_dim * 9 / 8;
}

int kq_slot_map(const int32_t* d_cached, const int32_t* d_new, int64_t requests, int32_t page_size,
                const int32_t* d_free_pages, int64_t free_count, int32_t* d_block_table, int64_t table_stride,
                int32_t* d_q_start, int32_t* d_kv_len, int32_t* d_positions, int32_t* d_slots, int64_t tokens,
                int32_t* d_pages_used, void* stream) {
  clear_error();
  if (!d_cached || !d_new || !d_block_table || !d_q_start || !d_kv_len || !d_pages_used ||
      (free_count != 0 && !d_free_pages) || (tokens != 0 && (!d_positions || !d_slots)))
    return fail(KQ_ERR_INVALID_ARG, "NULL pointer");
  if (requests < 1 || requests > 0x7fffffffll || table_stride < 1 || free_count < 0 || tokens < 0 || tokens > 0x7fffffffll)
    return fail(KQ_ERR_SHAPE, "requests = %lld, table_stride = %lld, free_count = %lld, tokens = %lld",
                (long long)requests, (long long)table_stride, (long long)free_count, (long long)tokens);
  if (page_size < 16 || page_size % 16) return fail(KQ_ERR_SHAPE, "page_size = %d (a positive multiple of 16)", page_size);
  for (const void* p : {(const void*)d_cached, (const void*)d_new, (const void*)d_free_pages, (const void*)d_block_table,
                        (const void*)d_q_start, (const void*)d_kv_len, (const void*)d_positions, (const void*)d_slots,
                        (const void*)d_pages_used})
    if (!aligned16(p)) return fail(KQ_ERR_ALIGNMENT, "an array is not 16-byte aligned");
  kv::SlotArgs a{d_cached, d_new, d_free_pages, d_block_table, d_q_start, d_kv_len, d_positions, d_slots, d_pages_used,
                 requests, free_count, table_stride, tokens, page_size};
  const int64_t grid = std::max<int64_t>(1, (tokens + kv::kMapTokens - 1) / kv::kMapTokens);
  KQ_CUDA_TRY(launch_dependent(kv::slot_map_kernel, dim3((unsigned)grid), dim3(kv::kScanThreads), 0,
                               static_cast<cudaStream_t>(stream), a));
  return KQ_OK;
}

int kq_rope_table_host(float* out, int64_t positions, int32_t rope_dim, double base) {
  clear_error();
  if (!out) return fail(KQ_ERR_INVALID_ARG, "NULL pointer");
  if (positions < 1 || rope_dim < 2 || rope_dim % 2)
    return fail(KQ_ERR_SHAPE, "positions = %lld, rope_dim = %d", (long long)positions, rope_dim);
  if (!(base > 0) || !std::isfinite(base)) return fail(KQ_ERR_INVALID_ARG, "base must be positive and finite");
  for (int i = 0; i < rope_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rope_dim);
    for (int64_t p = 0; p < positions; ++p) {
      out[p * rope_dim + i] = (float)std::cos((double)p * f);
      out[p * rope_dim + rope_dim / 2 + i] = (float)std::sin((double)p * f);
    }
  }
  return KQ_OK;
}

int kq_qk_norm_rope(const kq_qk_norm* p, int dtype, const kq_heads* q, const kq_heads* k, const int32_t* d_positions,
                    int64_t tokens, const kq_heads* q_out, const kq_heads* k_out, void* stream) {
  clear_error();
  if (int s = check_dtype(dtype)) return s;
  if (int s = check_qk(p, d_positions, tokens)) return s;
  if (tokens == 0) return KQ_OK;
  if (int s = check_heads(q, "q", dtype)) return s;
  if (int s = check_heads(k, "k", dtype)) return s;
  if (int s = check_heads(q_out, "q_out", dtype)) return s;
  if (int s = check_heads(k_out, "k_out", dtype)) return s;
  kv::QkArgs a = qk_args(p, d_positions, tokens);
  a.q = kv::view(q), a.k = kv::view(k), a.q_out = kv::view(q_out), a.k_out = kv::view(k_out);
  KQ_CUDA_TRY(kv::launch_qk<false>(dtype, p->head_dim, a, static_cast<cudaStream_t>(stream)));
  return KQ_OK;
}

int kq_kv_append(const kq_qk_norm* p, const kq_kv_cache* cache, int dtype, const kq_heads* q, const kq_heads* k,
                 const kq_heads* v, const int32_t* d_positions, const int32_t* d_slots, int64_t tokens,
                 const kq_heads* q_out, void* stream) {
  clear_error();
  if (int s = check_dtype(dtype)) return s;
  if (int s = check_qk(p, d_positions, tokens)) return s;
  if (int s = check_cache(cache)) return s;
  if (cache->kv_heads != p->kv_heads || cache->head_dim != p->head_dim)
    return fail(KQ_ERR_SHAPE, "cache of %d heads of %d, keys of %d heads of %d", cache->kv_heads, cache->head_dim,
                p->kv_heads, p->head_dim);
  if (tokens == 0) return KQ_OK;
  if (!q != !q_out) return fail(KQ_ERR_INVALID_ARG, "q and q_out come together");
  if (q) {
    if (int s = check_heads(q, "q", dtype)) return s;
    if (int s = check_heads(q_out, "q_out", dtype)) return s;
  }
  if (int s = check_heads(k, "k", dtype)) return s;
  if (int s = check_heads(v, "v", dtype)) return s;
  if (!d_slots) return fail(KQ_ERR_INVALID_ARG, "d_slots is NULL");
  if (!aligned16(d_slots)) return fail(KQ_ERR_ALIGNMENT, "d_slots not 16-byte aligned");
  kv::QkArgs a = qk_args(p, d_positions, tokens);
  if (!q) a.q_heads = 0;
  a.q = kv::view(q), a.k = kv::view(k), a.v = kv::view(v), a.q_out = kv::view(q_out);
  a.slots = d_slots;
  a.cache = cache_view(cache);
  KQ_CUDA_TRY(kv::launch_qk<true>(dtype, p->head_dim, a, static_cast<cudaStream_t>(stream)));
  return KQ_OK;
}

int kq_kv_read(const kq_kv_cache* cache, const int32_t* d_slots, int64_t count, int dtype, const kq_heads* k_out,
               const kq_heads* v_out, void* stream) {
  clear_error();
  if (int s = check_dtype(dtype)) return s;
  if (int s = check_cache(cache)) return s;
  if (count == 0) return KQ_OK;
  if (int s = check_heads(k_out, "k_out", dtype)) return s;
  if (int s = check_heads(v_out, "v_out", dtype)) return s;
  if (!d_slots) return fail(KQ_ERR_INVALID_ARG, "d_slots is NULL");
  if (!aligned16(d_slots)) return fail(KQ_ERR_ALIGNMENT, "d_slots not 16-byte aligned");
  if (count < 0 || count > 0x7fffffffll / cache->kv_heads) return fail(KQ_ERR_SHAPE, "count = %lld", (long long)count);
  const kv::Cache c = cache_view(cache);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const kv::View k = kv::view(k_out), v = kv::view(v_out);
  KQ_CUDA_TRY(dtype == KQ_F32 ? kv::launch_read<float>(c, cache->head_dim, d_slots, count, k, v, st)
                              : (dtype == KQ_F16 ? kv::launch_read<__half>(c, cache->head_dim, d_slots, count, k, v, st)
                                                 : kv::launch_read<__nv_bfloat16>(c, cache->head_dim, d_slots, count, k, v, st)));
  return KQ_OK;
}

}  // extern "C"
