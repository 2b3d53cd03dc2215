// What the attention kernels share: arguments, a request's extent, the cut of
// the work into runs, small arithmetic.  kq_attn.cu: one to a few query rows a
// request (and fp32 queries); kq_attn_prompt.cu: 16-bit prompts.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kq.h"
#include "kq_device.cuh"
#include "kq_kv.cuh"

namespace kq {
namespace attn {

using kv::Cache;
using kv::kGranule;
using kv::Layout;

constexpr int kSms = 152;

// Where a run of the prompt kernel begins: in unit `at` of row block k of request r and key head h, which looks at
// `tiles` key tiles and whose first unit is work unit `lo`.
struct RunStart {
  int64_t r, lo;
  int32_t k, h, at, tiles;
};

// The row tile that a run of attend_kernel begins in: the runs from .. to hold it, `from` as its first or a later row.  (A
// run without work: from = to.)
struct alignas(16) TileStart {
  int32_t from, to, later;
  int32_t first, x0, rows, h;  // the request's first token, the row tile's first row and all rows of the key head
  int32_t reserved;
};

struct Args {
  Cache cache;
  const void* q;
  void* out;
  int64_t q_token, q_head, out_token, out_head;
  const int32_t *q_start, *kv_len, *table;
  int64_t table_stride, requests, tokens, max_new;
  int32_t window;  // 0: none
  int32_t q_heads, group;
  float scale;
  // requests with more query rows than this are the prompt kernel's
  int32_t few_rows;
  int32_t by_runs;  // how cut rows are found again (combine_kernel)
  // workspace
  int64_t* base;             // first work unit of each request, and the total (with by_runs: not written)
  TileStart* starts;         // of each run of attend_kernel (with by_runs alone)
  float* partials;           // two slots per run of kRows x D sums, kRows references, kRows weights
  int64_t* prompt_total;     // work units of the prompt kernel
  RunStart* prompt_starts;   // of each of its runs
  float* prompt_partials;
};

// What a request asks for.  Tiles of `tile` keys from tile0 on cover every key
// that one of its tokens sees.
struct Request {
  int32_t first, n;      // its new tokens
  int32_t len, pos0;     // keys held; position of its first new token (negative: that token sees nothing)
  int32_t lo;            // first key that one of its tokens sees
  int32_t tile0, tiles;
  int32_t rows;          // query rows of one key head
};

// First key that a token at `pos` sees.  (pos - (window - 1) would pass -2^31 for a negative position and the longest window.)
__device__ __forceinline__ int32_t first_key(const Args& a, int32_t pos) {
  return a.window ? max(0, max(pos, 0) - (a.window - 1)) : 0;
}

// kFromL2: read past the SM's own cache.
template <bool kFromL2 = false>
__device__ __forceinline__ Request request_of(const Args& a, int64_t r, int tile, bool* out_of_range = nullptr) {
  auto load = [](const int32_t* p) { return kFromL2 ? __ldcg(p) : *p; };
  Request q;
  q.first = load(a.q_start + r);
  const int32_t end = load(a.q_start + r + 1);
  int32_t len = load(a.kv_len + r);
  const int64_t room = a.table_stride * a.cache.page_size;
  bool bad = len < 0 || len > room;
  q.n = end - q.first;
  if (q.first < 0 || end < q.first || end > a.tokens || q.n > a.max_new) bad = true, q.n = 0;
  len = max(len, 0);
  q.pos0 = len - q.n;
  q.len = (int32_t)min((int64_t)len, room);
  q.lo = first_key(a, q.pos0);
  q.tile0 = q.lo / tile;
  q.tiles = q.n > 0 && q.len > q.lo ? (q.len - 1) / tile - q.tile0 + 1 : 0;
  q.rows = (int32_t)min((int64_t)0x7fffffff, (int64_t)q.n * a.group);
  if (bad && out_of_range) *out_of_range = true;
  return q;
}

// Pages of `len` keys.  (Lengths go up to 2^31 - 1: neither this sum nor the end of the last key tile fits 32 bits, so
// tiles are compared by their first key.)
__device__ __forceinline__ int32_t pages_of(int32_t len, int32_t page_size) { return len / page_size + (len % page_size != 0); }

// The prompt kernel's row blocks and key tiles (kq_attn_prompt.cu).
template <int D>
struct PromptShape {
  static constexpr int kTiles = D == 256 ? 1 : 2;     // 128 query rows each
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kKeys = 64;
  // A row (a block of query rows of one key head) counts as its key tiles and so many units before them: fetching the
  // queries and putting the rows away cost 15000 to 18000 cycles, a tile 1900.  (Counted by tiles alone, ragged prompts
  // left CTAs with nine short rows, 176000 cycles, beside others with two, 72000.  6 ragged prompts of up to 700 of 1500
  // tokens, 8 key heads of 128: 90.9 us with six units, 84.5 with ten, 89.2 with 14.)
  static constexpr int kRowCost = 10;
  // Units that a run is worth: two tiles of a row.  (Runs share the units evenly, so one more than this many make two
  // runs of half as many, of which the first may hold no tile.)  The last 300 of 2000 tokens: 43.2 us; with twelve more
  // units a run 9 us more.
  static constexpr int kLeastRun = kRowCost + 2;
  __device__ static int32_t units(int32_t tiles) { return tiles ? tiles + kRowCost : 0; }
  static constexpr int64_t kPartial = kRows * (int64_t)(D + 2);
};

// A block of query rows and the key tiles it looks at.
struct RowBlock {
  int32_t rows, lo, hi;  // keys lo .. hi - 1 are seen by some row
  int32_t tile0, tiles;
};
template <int D>
__device__ __forceinline__ RowBlock row_block(const Args& a, const Request& q, int32_t k) {
  using S = PromptShape<D>;
  RowBlock b;
  const int32_t x0 = k * S::kRows;
  b.rows = min(S::kRows, q.rows - x0);
  const int32_t i0 = x0 / a.group, i1 = (x0 + b.rows - 1) / a.group;
  b.hi = min(q.len, q.pos0 + i1 + 1);
  b.lo = first_key(a, q.pos0 + i0);
  b.tile0 = b.lo / S::kKeys;
  b.tiles = b.hi > b.lo ? (b.hi - 1) / S::kKeys - b.tile0 + 1 : 0;
  return b;
}

// The work units cut into runs: the first `extra` of them per + 1 long, the others per.  No run is empty.
struct Runs {
  int64_t per, extra, count;
  __device__ __forceinline__ Runs(int64_t total, int64_t most, int least) {
    count = min(most, (total + least - 1) / least);
    per = count ? total / count : 0;
    extra = total - per * count;
  }
  __device__ __forceinline__ int64_t start(int64_t i) const { return i * per + min(i, extra); }
  __device__ __forceinline__ int64_t of(int64_t unit) const {
    const int64_t cut = extra * (per + 1);
    return unit < cut ? unit / (per + 1) : extra + (unit - cut) / per;
  }
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t u) { return __half22float2(*reinterpret_cast<__half2*>(&u)); }

// Launches the prompt kernel for `dtype` KQ_F16 or KQ_BF16 (kq_attn_prompt.cu).
cudaError_t launch_prompt(int dtype, int head_dim, const Args& a, cudaStream_t st);

}  // namespace attn
}  // namespace kq
