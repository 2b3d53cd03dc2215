// Attention of prompts (16-bit queries, more than a few query rows a request)
// over the paged 4-bit cache, on the 5th-generation tensor cores.
//
// With many query rows per key the work is a dense contraction: 4 D flops per
// (query, key) pair against 4.5 bits per key value, so the tensor cores bound
// it.  A CTA takes blocks of 256 query rows of one key head (two M tiles of
// 128; at D = 256 one tile, for tensor memory holds 512 columns) and walks over
// tiles of 64 keys:
//
//   S = Q K^T   tcgen05.mma, both operands in shared memory
//   P = 2^(f S - m)  one thread per row, from and to tensor memory (fp16)
//   O += P V    tcgen05.mma, P from tensor memory
//
// Keys and values become fp16 as they are unpacked (code - 8, exact, times the
// scale, one rounding: the two roundings of K and V and that of P are each
// 2^-11 at most, as the one of a 16-bit output, and independent); sums, maxima
// and weights stay fp32.  Queries are scaled by a power of two per row, so bf16
// loses nothing either.  Where a scale passes 8188 (the value would leave fp16)
// the tile's keys or values are divided by 8, and scores or probabilities
// multiplied by it.
//
// Roles: warp 0 copies granules into raw stages; warps 1 and 3 issue the MMAs
// of an M tile each; warp 2 looks at a stage's scales; warps 4-7 and 8-11 are
// the softmax of the two M tiles; warps 12-15 and 16-19 unpack every other key
// tile, into a ring of buffers that keys and values take in turn (one group of
// four warps bound the kernel: 507 us, 309 without it; eight warps on every
// tile spent 750 of their 2600 cycles a tile at barriers and had one chain of
// work at a time).  Each M tile has two S buffers (P replaces S in place), and
// QK of the next key tile is issued before PV of this one, so that a softmax
// finds its next scores waiting: with one S buffer of 128 keys per M tile the
// chain QK, softmax, PV bound the kernel (382 us).  The reference m of a row is
// the largest score of the first tile it sees; it moves when a tile's sum of p
// passes 2^12, and then its warp rescales O in tensor memory.  The loops are
// unrolled no further than the instruction cache takes with five roles running
// (378 us with the unpacking loops unrolled, 266 without).
//
// Measured: the last 2048 of 8192 tokens, 32 query and 8 key heads of 128,
// bf16: 249 to 255 us, 945 to 966 TFLOP/s of what the mask leaves.  Issue slots
// bound it (63% taken; tensor pipe 42%): unpacking, which each row block does
// anew, and the softmax.  Rounding K, V and P to fp16 costs rows of fp16 output
// an error of 3.6e-4 to 3.8e-4 where rounding the output alone costs 2.1e-4.  (P
// as two fp16 parts left 3.2e-4 and took 300 us instead of 255 in fp16.)  The
// scores' rounding goes into the exponent: it grows with their size.
//
// Row blocks in order, each head's key tiles end to end, are cut into one run
// of tiles per CTA, whatever the prompts' lengths and masks; a block cut
// between CTAs leaves partial sums, which kq_attn.cu's combine kernel joins.
#include <cuda_runtime.h>

#include <cmath>

#include "kq_attn.cuh"
#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_kv.cuh"
#include "kq_tcgen05.cuh"

namespace kq {
namespace attn {

using namespace tc;

__device__ unsigned int g_prompt_status = 0;
__device__ __forceinline__ void prompt_flag(int status) { atomicOr(&g_prompt_status, 1u << status); }

// Five warpgroups of 96 registers a thread at launch: two that keep scores in registers take 144, the others give 32
// back (2 x 144 + 3 x 64 = 5 x 96).
constexpr int kPromptWarps = 20, kPromptThreads = 32 * kPromptWarps;
constexpr int kUnpackFirst = 12, kUnpackWarps = 4;  // two groups of them, a key tile in turn each
constexpr float kPromptMost = 4096.f;  // times 8 (see above) still fits fp16
constexpr float kCoarse = 16777216.f;  // 2^24: numbers from here on lie two or more apart
constexpr int kInfos = 8;            // key tiles between unpacking and softmax, and more

template <int D>
struct PromptConfig : PromptShape<D> {
  using S = PromptShape<D>;
  using L = Layout<D>;
  static constexpr int kGranules = S::kKeys / kGranule;          // of a key tile
  static constexpr int kQBytes = 128 * D * 2;                    // one M tile
  static constexpr int kBuffer = S::kKeys * D * 2;               // a tile of keys or values in fp16
  static constexpr int kRaw = kGranules * L::kBytes;
  static constexpr int kBuffers = D == 256 ? 3 : 6;
  static constexpr int kStages = D == 256 ? 2 : 4;               // raw
  static constexpr int kRing = S::kTiles * kQBytes;              // offsets
  static constexpr int kRawAt = kRing + kBuffers * kBuffer;
  static constexpr int kSmem = kRawAt + kStages * kRaw + 1024;   // and room to align to 1024
  // tensor memory columns: two S buffers of each M tile (P over them), then O
  static constexpr int kO = 2 * S::kTiles * S::kKeys;
  static constexpr int kColumns = 512;
  static_assert(kO + S::kTiles * D <= kColumns, "tensor memory");
};

struct TileInfo {
  float key_scale, value_scale;  // 1, or 8 where the tile was divided by 8
  uint32_t nan;                  // a value scale of a visible key is not finite
  uint32_t hidden;               // bit per granule whose page is missing
  uint32_t special;              // values need a look: hidden or invisible keys, large or non-finite scales
};

// Barriers that every role waits on with a limit; after one ran out all waits return at once, and the roles run through.
struct Gate {
  volatile int* abort;
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return;
    const long long start = clock64();
    while (!mbar_try_wait_suspend(bar, parity)) {
      if (*abort) return;
      if (clock64() - start > kWaitLimitCycles) {
        *abort = 1;
        prompt_flag(KQ_ERR_TIMEOUT);
        return;
      }
    }
  }
};

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

template <int N>
__device__ __forceinline__ void load_raw(uint32_t (&w)[N], const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}

// A pair of codes (low nibble of each half of v) minus 8, times d.
__device__ __forceinline__ uint32_t value_pair(uint32_t v, __half2 d) {
  const uint32_t magic = (v & 0x000F000Fu) | 0x64006400u;  // 1024 + q
  return as_u32(__hmul2(__hsub2(as_h2(magic), as_h2(0x64086408u)), d));
}

// The same of the second nibble of each half.
__device__ __forceinline__ uint32_t value_pair_up(uint32_t v, __half2 d) {
  const uint32_t magic = (v & 0x00F000F0u) | 0x64006400u;  // 1024 + 16 q
  return as_u32(__hmul2(__hfma2(as_h2(magic), as_h2(0x2C002C00u), as_h2(0xD480D480u)), d));
}

// Keys of tokens 8 b .. 8 b + 7, slab sl: each lane a quarter of one token's groups, one 16-byte chunk a group.  The
// eight dimensions of a chunk lie in the order 0 4 1 5 2 6 3 7, as the queries do.  Tokens of odd index take their
// groups in the other order, so that a store's eight lanes fall on different banks.
template <int D>
__device__ __forceinline__ void unpack_keys(const uint8_t* raw, uint8_t* buf, int b, int sl, bool shrink) {
  using C = PromptConfig<D>;
  using L = Layout<D>;
  constexpr int G = L::kGroups;
  const int lane = threadIdx.x & 31, r = lane / 4, c = lane & 3;
  const uint8_t* g0 = raw + (b / 2) * L::kBytes;
  uint32_t w[G], ks[G / 2];
  load_raw<G>(w, g0 + L::kKeys + sl * L::kKeySlab + (b % 2) * L::kBlock + lane * (L::kBlock / 32));
  const uint8_t* sp = g0 + L::kKeyScales + sl * L::kScaleSlab + ((b % 2) * 8 + r) * G * 2;
  if constexpr (G == 4) {
    load_raw<2>(ks, sp);
  } else {
    ks[0] = *reinterpret_cast<const uint32_t*>(sp);
  }
  if (shrink) {
#pragma unroll
    for (int i = 0; i < G / 2; ++i) ks[i] = as_u32(__hmul2(as_h2(ks[i]), __float2half2_rn(0.125f)));
  }
  const uint32_t pick = r & 1;
#pragma unroll
  for (int s = 0; s < G; ++s) {
    const uint32_t v = pick ? w[s ^ 1] : w[s];
    const __half2 d = as_h2(__byte_perm(ks[s / 2], 0, (s % 2) ^ pick ? 0x3232 : 0x1010));
    const uint32_t u = v >> 8;
    uint4 o;  // nibbles 1 and 3 stay 4 bits up: 1024 + 16 q, times 1/16, minus 72
    o.x = value_pair(v, d);
    o.y = value_pair_up(v, d);
    o.z = value_pair(u, d);
    o.w = value_pair_up(u, d);
    const int dim = sl * L::kSlabDim + 32 * (s ^ (r & 1));
    const int chunk = (dim % 64) / 8 + c;
    *reinterpret_cast<uint4*>(buf + (dim / 64) * (C::kKeys * 128) + (8 * b + r) * 128 + ((chunk ^ r) << 4)) = o;
  }
}

// Values of tokens 8 b .. 8 b + 7, slab sl, transposed: row = dimension, the tile's keys along it.  A lane holds four
// dimensions of two successive tokens and stores a pair of tokens a dimension; the lanes take their dimensions in
// rotated order, so that a store's rows fall on different banks.
template <int D>
__device__ __forceinline__ void unpack_values(const uint8_t* raw, uint8_t* buf, int b, int sl, bool special, bool shrink,
                                              uint32_t valid) {
  using L = Layout<D>;
  constexpr int G = L::kGroups;
  const int lane = threadIdx.x & 31, r = lane / 4, c = lane & 3;
  const uint8_t* g0 = raw + (b / 2) * L::kBytes;
  uint32_t w[G], vs[G];
  load_raw<G>(w, g0 + L::kValues + sl * L::kKeySlab + (b % 2) * L::kBlock + lane * (L::kBlock / 32));
  load_raw<G>(vs, g0 + L::kValueScales + sl * L::kScaleSlab + ((b % 2) * 8 + 2 * c) * G * 2);
  __half2 d[G];
#pragma unroll
  for (int g = 0; g < G; ++g) d[g] = as_h2(__byte_perm(vs[g / 2], vs[G / 2 + g / 2], g % 2 ? 0x7632 : 0x5410));
  if (special) {
    // hidden keys and scales that are not finite count as zero (those keys' rows are marked by the softmax)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      d[g] = as_h2(as_u32(d[g]) & __hle2_mask(__habs2(d[g]), as_h2(0x7BFF7BFFu)) & valid);
      if (shrink) d[g] = __hmul2(d[g], __float2half2_rn(0.125f));
    }
  }
  uint8_t* base = buf + (b / 8) * (D * 128) + (sl * L::kSlabDim + 4 * r) * 128 + 4 * c;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = (j + (r >> 1)) & 3, row = (4 * r + e) & 7;
    uint8_t* at = base + e * 128 + (((b % 8) ^ row) << 4);
#pragma unroll
    for (int g = 0; g < G; ++g) *reinterpret_cast<uint32_t*>(at + g * 32 * 128) = value_pair(w[g] >> (4 * e), d[g]);
  }
}

// Bits lo .. hi - 1 of 32.
__device__ __forceinline__ uint32_t visible(int lo, int hi) {
  const uint32_t below = hi <= 0 ? 0u : (hi >= 32 ? ~0u : (1u << hi) - 1);
  const uint32_t skipped = lo <= 0 ? 0u : (lo >= 32 ? ~0u : (1u << lo) - 1);
  return below & ~skipped;
}
// Keys c .. c + 31 of a tile whose granules (16 keys) are missing.
__device__ __forceinline__ uint32_t hidden_keys(uint32_t hidden, int c) {
  const uint32_t h = hidden >> (c / kGranule);
  return (h & 1u ? 0xFFFFu : 0u) | (h & 2u ? 0xFFFF0000u : 0u);
}

// A query row of a block: its token, and its head among those of the key head.
struct RowAt {
  int32_t token, head;
};

// The run's position: request, row block, key head, unit of that row.
struct Place {
  int64_t r;
  int32_t k, h, at;
};

// A run's segments: row by row (request, row block, key head), the key tiles of it that the run holds.  Each warp's lies
// in shared memory: within a segment a role holds what it uses of it, and no more, in its registers (kept there whole it
// was spilled in the unpacking loops: 374 us against 325 for 2048 tokens on 8192).
template <int D>
struct Walk {
  using S = PromptShape<D>;
  Place at;
  int64_t unit, end;
  Request q;
  RowBlock blk;
  int32_t from, to, tiles, nm;   // key tiles of the segment, its M tiles
  int32_t upto;                  // unit of the row that the segment ends before
  uint32_t bufs;                 // buffers of keys and values used so far
  uint32_t queries;              // bit m: how many segments M tile m has been part of, modulo 2
  uint32_t uses;                 // bit 2 m + b: how often S buffer b of M tile m has been used, modulo 2
  bool first;

  __device__ __forceinline__ void begin(const Args& a, const Place& p, int64_t u, int64_t e) {
    at = p, unit = u, end = e, bufs = queries = uses = 0, first = true;
    if (unit < end) {
      q = request_of(a, at.r, S::kKeys);
      blk = row_block<D>(a, q, at.k);
    }
  }
  // Parity of the barrier phase of M tile m's j-th score tile of the segment.
  __device__ __forceinline__ uint32_t phase(int m, int j) const { return ((uses >> (2 * m + (j & 1))) + j / 2) & 1; }
  __device__ __forceinline__ bool next(const Args& a) {
    while (unit < end) {
      if (at.at == S::units(blk.tiles)) {  // heads, then blocks, then requests
        at.at = 0;
        if (++at.h == a.cache.kv_heads) {
          at.h = 0;
          do {
            if (++at.k >= (q.rows + S::kRows - 1) / S::kRows) {
              at.k = 0;
              do q = request_of(a, ++at.r, S::kKeys);
              while (q.rows <= a.few_rows);  // a unit remains, so some request has it
            }
            blk = row_block<D>(a, q, at.k);
          } while (blk.tiles == 0);
        }
      }
      upto = (int32_t)min((int64_t)S::units(blk.tiles), at.at + (end - unit));
      from = max(0, at.at - S::kRowCost), to = max(0, upto - S::kRowCost);
      tiles = to - from;
      nm = blk.rows > 128 ? 2 : 1;
      if (tiles) return true;
      advance();  // the run ends before the row's first tile
    }
    return false;
  }
  __device__ __forceinline__ void advance() {
    unit += upto - at.at;
    at.at = upto;
  }
  __device__ __forceinline__ void done() {
    bufs += 2 * tiles;
    uses ^= ((((tiles + 1) / 2) & 1u) | ((tiles / 2) & 1u) << 1) * (nm == 2 ? 5u : 1u);
    queries ^= nm == 2 ? 3u : 1u;
    first = false;
    advance();
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kPromptThreads, 1) prompt_kernel(Args a) {
  using C = PromptConfig<D>;
  using L = Layout<D>;
  constexpr int N = C::kKeys;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t raw_full[C::kStages], raw_seen[C::kStages], raw_empty[C::kStages], buf_full[C::kBuffers], buf_empty[C::kBuffers];
  __shared__ uint64_t s_full[C::kTiles][2], p_full[C::kTiles][2], pv_done[C::kTiles][2], q_full[C::kTiles];
  __shared__ TileInfo s_info[kInfos];
  __shared__ uint8_t s_nan[kInfos][N];        // groups of a key whose value scale is not finite
  __shared__ uint32_t s_hidden[C::kStages];   // of a raw stage
  __shared__ uint64_t s_drain[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int64_t s_entry[kPromptThreads];  // row blocks before each request of a chunk
  __shared__ int64_t s_sum[kPromptWarps];
  __shared__ Place s_place;
  __shared__ Walk<D> s_walk[kPromptWarps];
  // (an offset and not a rounded address: the compiler then still knows it for shared memory)
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_seen[i], 1);
      mbar_init(&raw_empty[i], kUnpackWarps);
    }
    for (int i = 0; i < 2 * C::kTiles; ++i) {
      mbar_init(&s_full[i / 2][i & 1], 1);
      mbar_init(&p_full[i / 2][i & 1], 128);
      mbar_init(&pv_done[i / 2][i & 1], 1);
    }
    for (int i = 0; i < C::kTiles; ++i) mbar_init(&q_full[i], 128);
    for (int i = 0; i < C::kBuffers; ++i) {
      mbar_init(&buf_full[i], kUnpackWarps);
      mbar_init(&buf_empty[i], C::kTiles);
    }
    mbar_init(&s_drain[0], 1);
    mbar_init(&s_drain[1], 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, C::kColumns);
    tmem_relinquish();
  }
  grid_dependency_wait();
  allow_dependent_launch();

  // ---- the work units before each row block, and where this CTA's run begins ----
  auto block_sum = [&](int64_t v, int64_t& before, int64_t& all) {  // exclusive sum over the CTA
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += x;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    before = inc - v, all = 0;
    for (int i = 0; i < kPromptWarps; ++i) {
      if (i < warp) before += s_sum[i];
      all += s_sum[i];
    }
  };
  int64_t unit = 0, end = 0;  // this CTA's run
  {
    int64_t total = 0;
    for (int pass = 0; pass < 2; ++pass) {
      // the thread's last row block, whose place starts the run if the run starts in it
      Place p{};
      int64_t u = 0, first_unit = 0;
      int32_t tiles = 0;
      auto found = [&]() {
        if (u > 0 && unit >= first_unit && unit < first_unit + u) {
          const int64_t in = unit - first_unit;
          p.h = (int32_t)(in / C::units(tiles)), p.at = (int32_t)(in % C::units(tiles));
          s_place = p;
          a.prompt_starts[blockIdx.x] = RunStart{p.r, unit - p.at, p.k, p.h, p.at, tiles};
        }
      };
      int64_t units = 0, entries = 0;
      for (int64_t r0 = 0; r0 < a.requests; r0 += kPromptThreads) {
        int64_t blocks = 0;
        if (r0 + tid < a.requests) {
          const Request q = request_of(a, r0 + tid, N);
          blocks = q.rows > a.few_rows ? (q.rows + C::kRows - 1) / C::kRows : 0;
        }
        int64_t before, all;
        block_sum(blocks, before, all);
        s_entry[tid] = before;
        __syncthreads();
        const int in_chunk = (int)min((int64_t)kPromptThreads, a.requests - r0);
        for (int64_t e0 = 0; e0 < all; e0 += kPromptThreads) {
          const int64_t e = e0 + tid;
          int64_t at, sum;
          u = 0;
          if (e < all) {
            int l = 0, h = in_chunk;
            while (h - l > 1) {  // the last request whose first row block is not after e
              const int m = (l + h) >> 1;
              if (s_entry[m] <= e) l = m; else h = m;
            }
            p.r = r0 + l, p.k = (int32_t)(e - s_entry[l]);
            tiles = row_block<D>(a, request_of(a, p.r, N), p.k).tiles;
            u = (int64_t)C::units(tiles) * a.cache.kv_heads;
          }
          block_sum(u, at, sum);
          first_unit = units + at;
          if (pass == 1) found();
          units += sum;
        }
        entries += all;
        __syncthreads();  // s_entry has been read
      }
      if (pass == 0) {
        total = units;
        if (blockIdx.x == 0 && tid == 0) *a.prompt_total = total;
        const Runs runs(total, kSms, C::kLeastRun);
        if (blockIdx.x < runs.count) unit = runs.start(blockIdx.x), end = runs.start(blockIdx.x + 1);
        if (unit == end) break;  // the same for the whole CTA
        if (a.requests <= kPromptThreads && entries <= kPromptThreads) {  // one look was enough
          found();
          break;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const Gate gate{&s_abort};
  {
    Walk<D> w;
    w.begin(a, s_place, unit, end);
    if (lane == 0) s_walk[warp] = w;
    __syncwarp();
  }
  auto next = [&]() {
    Walk<D> w = s_walk[warp];
    __syncwarp();
    const bool more = w.next(a);
    if (lane == 0) s_walk[warp] = w;
    __syncwarp();
    return more;
  };
  auto done = [&]() {
    Walk<D> w = s_walk[warp];
    __syncwarp();
    w.done();
    if (lane == 0) s_walk[warp] = w;
    __syncwarp();
  };
  uint32_t raws = 0;  // raw stages that a copying, looking or unpacking warp is through with
  // Each role walks over the run's segments by itself, copies and unpacking ahead into the next one as far as their
  // rings go.
  if (warp >= 4 && warp < 4 + 4 * C::kTiles) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    // n / group = umulhi(n, per_group) for n below 2^32 / group: here n < group + 256
    const uint32_t per_group = 0xFFFFFFFFu / (uint32_t)a.group + 1;
    while (next()) {
      const Walk<D> w = s_walk[warp];
      // ---- queries: one thread a row ----
      const int m_tile = (warp - 4) / 4;
      const int row = (warp & 3) * 32 + lane;       // tensor memory lane
      const int32_t x = w.at.k * C::kRows + m_tile * 128 + row, i = x / a.group;
      const bool live = m_tile * 128 + row < w.blk.rows;
      const int32_t pos = w.q.pos0 + i;
      const int32_t key_hi = live ? max(0, min(pos + 1, w.q.len)) : 0x7fffffff;
      const int32_t key_lo = live ? first_key(a, pos) : 0;
      // A row's D / 8 lanes load it, eight dimensions each; the factor then goes to the row's own thread.  (The scale's
      // sign goes with the queries, so that larger sums are larger scores.)
      const int32_t token0 = w.q.first + w.at.k * C::kRows / a.group, head0 = w.at.k * C::kRows % a.group;
      auto rows_at = [&](int in) {  // row `in` of the block
        const uint32_t n = head0 + in, d = a.group == 1 ? n : __umulhi(n, per_group);
        return RowAt{token0 + (int32_t)d, (int32_t)(n - d * a.group)};
      };
      float factor = 0.f;
      if (m_tile < w.nm) {
        // (Copied to their place first, then scaled there in a short loop: a segment runs this code once, so its
        // instructions come from far away, and 16 rows unrolled took 15000 cycles.)
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
        const int l = lane % kLanes, sub = lane / kLanes;
        uint8_t* tile = smem + m_tile * C::kQBytes + (l / 8) * (128 * 128);
        const float score = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
        const float sign = a.scale == 0.f ? 0.f : copysignf(1.f, a.scale);
        const T* src = static_cast<const T*>(a.q) + (int64_t)w.at.h * a.group * a.q_head + 8 * l;
#pragma unroll 1
        for (int it = 0; it < kLanes; ++it) {
          const int rr = (warp & 3) * 32 + it * kAtOnce + sub;
          const bool held = m_tile * 128 + rr < w.blk.rows;
          const RowAt y = rows_at(held ? m_tile * 128 + rr : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           smem_u32(tile + rr * 128 + (((l % 8) ^ (rr & 7)) << 4))),
                       "l"(src + (int64_t)y.token * a.q_token + (int64_t)y.head * a.q_head), "r"(held ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 2
        for (int it = 0; it < kLanes; ++it) {
          const int rr = (warp & 3) * 32 + it * kAtOnce + sub;
          uint4* place = reinterpret_cast<uint4*>(tile + rr * 128 + (((l % 8) ^ (rr & 7)) << 4));
          union { uint4 u; T t[8]; } in;
          in.u = *place;
          float v[8], top = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = kv::to_float(in.t[e]), top = fmaxf(top, fabsf(v[e]));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
          // 2^e2 brings the row's largest into [2^7, 2^8); an infinite row is left as it is
          const int exponent = (int)(__float_as_uint(top) >> 23);
          const int e2 = exponent == 255 ? 0 : min(max(134 - exponent, -110), 110);
          const float up = sign * __uint_as_float((uint32_t)(127 + e2) << 23);
          const float f = fmaxf(score * __uint_as_float((uint32_t)(127 - e2) << 23), 1e-37f);
          const float mine = __shfl_sync(~0u, f, (lane - it * kAtOnce) * kLanes);
          if (lane / kAtOnce == it) factor = mine;
          uint4 o;
          o.x = pack2(v[0] * up, v[4] * up), o.y = pack2(v[1] * up, v[5] * up);
          o.z = pack2(v[2] * up, v[6] * up), o.w = pack2(v[3] * up, v[7] * up);
          *place = o;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      // the segment's queries are in place, and what the last one left in O has been read
      if (m_tile < w.nm) mbar_arrive(&q_full[m_tile]);
      // ---- softmax ----
      if (m_tile < w.nm) {
        float ref = -INFINITY, weight = 0.f;
        uint32_t nan_groups = 0;
        const int32_t all_lo = __reduce_max_sync(~0u, key_lo), all_hi = __reduce_min_sync(~0u, key_hi);
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // tensor memory address of the warp's lanes
        for (int j = 0; j < w.tiles; ++j) {
          const int b = j & 1, slot = (w.bufs / 2 + j) % kInfos;
          const int32_t key0 = (w.blk.tile0 + w.from + j) * N;
          const uint32_t s_at = tmem + lanes + (2 * m_tile + b) * N;
          gate.wait(&s_full[m_tile][b], w.phase(m_tile, j));
          __syncwarp();
          tc_fence_after();
          uint32_t s[2][32];
          tmem_ld32(s_at, s[0]);
          tmem_ld32(s_at + 32, s[1]);
          const TileInfo info = s_info[slot];
          float f = factor * info.key_scale;
          const int32_t rel_lo = key_lo - key0, rel_hi = key_hi - key0;
          tmem_ld_wait();
          if (info.hidden || key0 < all_lo || key0 > all_hi - N) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t see = visible(rel_lo - 32 * c, rel_hi - 32 * c) & ~hidden_keys(info.hidden, 32 * c);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(see >> e & 1u)) s[c][e] = 0xFF800000u;  // -inf
            }
          }
          // Of the row's scores, log2.  (Needed in a row's first tile and when the reference moves: without the fence the
          // compiler worked it out before the branches, 61 of a tile's 430 instructions.)
          auto largest = [&]() {
            asm volatile("" : "+r"(s[0][0]));
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; ++e)
              top[e % 4] = fmaxf(top[e % 4], fmaxf(__uint_as_float(s[0][e]), __uint_as_float(s[1][e])));
            return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * f;
          };
          if (__any_sync(~0u, ref == -INFINITY)) {  // a row's first scores; nothing of it is in O yet
            const float top = largest();
            if (ref == -INFINITY) ref = top;
          }
          // p = 2^(f S - ref).  The reference stays while a tile's p add up to less than 2^12 (each then fits fp16): the
          // exponentials wait for no maximum.  f S - ref is rounded once, so a reference that is the row's own largest
          // score, rounded, leaves that one 2^r, r what its rounding took: a fraction, but from 2^28 on r passes 12
          // either way, and p overflows or the row's weight vanishes.  From 2^24 on the scores are therefore rounded as
          // the reference was, before the subtraction; the largest p is then 1.  After a move every p is 2 at most, so
          // there is no third round.
          uint32_t p[32];
          float2 acc;
#pragma unroll 1
          for (int round = 0;; ++round) {
            const float minus = ref == -INFINITY ? 0.f : -ref;
            if (fabsf(minus) >= kCoarse) {
#pragma unroll
              for (int e = 0; e < 64; ++e) s[e / 32][e % 32] = __float_as_uint(__uint_as_float(s[e / 32][e % 32]) * f);
              f = 1.f;
            }
            float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              const float2 v = make_float2(__uint_as_float(s[e / 32][e % 32]), __uint_as_float(s[e / 32][e % 32 + 1]));
              float2 y = fma2(v, make_float2(f, f), make_float2(minus, minus));
              y = make_float2(exp2_approx(y.x), exp2_approx(y.y));
              sums[e / 2 % 2] = add2(sums[e / 2 % 2], y);
              p[e / 2] = pack2(y.x, y.y);
            }
            acc = add2(sums[0], sums[1]);
            const bool moves = acc.x + acc.y > kPromptMost;
            if (round == 1 || !__any_sync(~0u, moves)) break;
            const float top = largest(), keep = moves ? exp2_approx(ref - top) : 1.f;
            if (moves) ref = top;
            weight *= keep;
            if (j > 0) {  // rescale what earlier tiles left in O, once the last of them is in
              gate.wait(&pv_done[m_tile][b ^ 1], w.phase(m_tile, j - 1));
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                float o[16];
                tmem_ld16(tmem + lanes + C::kO + m_tile * D + c, o);
                tmem_ld_wait();
                uint32_t u[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * keep);
                tmem_st16(tmem + lanes + C::kO + m_tile * D + c, u);
              }
            }
          }
          if (info.value_scale != 1.f) {
#pragma unroll
            for (int e = 0; e < 32; ++e) p[e] = as_u32(__hmul2(as_h2(p[e]), __float2half2_rn(8.f)));
          }
          tmem_st32(s_at, p);
          weight += acc.x + acc.y;
          if (info.nan) {
            for (int e = 0; e < N; ++e)
              if (e >= rel_lo && e < rel_hi) nan_groups |= s_nan[slot][e];
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[m_tile][b]);
        }
        // ---- the block's rows ----
        gate.wait(&pv_done[m_tile][(w.tiles - 1) & 1], w.phase(m_tile, w.tiles - 1));
        __syncwarp();
        tc_fence_after();
          const bool whole = w.from == 0 && w.to == w.blk.tiles;
          float* part = a.prompt_partials + (2 * (int64_t)blockIdx.x + (w.first ? 0 : 1)) * C::kPartial;
          const float scale = whole ? (weight == 0.f ? 0.f : 1.f / weight) : 1.f;
          if (!whole && live) {
            part[C::kRows * D + m_tile * 128 + row] = ref;
            part[C::kRows * D + C::kRows + m_tile * 128 + row] = weight;
          }
          // 32 dimensions at a time, turned in the warp's own part of the queries' place: a row's thread has its sums,
          // eight lanes store them side by side
          uint8_t* turn = smem + m_tile * C::kQBytes + (warp & 3) * 32 * 128;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(tmem + lanes + C::kO + m_tile * D + c, o);
            tmem_ld_wait();
            const float poison = nan_groups >> (c / 32) & 1u ? NAN : 0.f;
            uint8_t* mine = turn + lane * 128;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float4 v;
              v.x = __uint_as_float(o[4 * e]) * scale + poison, v.y = __uint_as_float(o[4 * e + 1]) * scale + poison;
              v.z = __uint_as_float(o[4 * e + 2]) * scale + poison, v.w = __uint_as_float(o[4 * e + 3]) * scale + poison;
              *reinterpret_cast<float4*>(mine + ((e ^ (lane & 7)) << 4)) = v;
            }
            __syncwarp();
#pragma unroll 8
            for (int it = 0; it < 8; ++it) {
              const int rr = 4 * it + lane / 8, in = m_tile * 128 + (warp & 3) * 32 + rr, e = lane & 7;
              const float4 v = *reinterpret_cast<const float4*>(turn + rr * 128 + ((e ^ (rr & 7)) << 4));
              if (in < w.blk.rows) {
                if (whole) {
                  const RowAt y = rows_at(in);
                  T* dst = static_cast<T*>(a.out) + (int64_t)y.token * a.out_token +
                           (int64_t)(w.at.h * a.group + y.head) * a.out_head + c + 4 * e;
                  union { uint2 u; T t[4]; } z;
                  z.t[0] = kv::from_float<T>(v.x), z.t[1] = kv::from_float<T>(v.y);
                  z.t[2] = kv::from_float<T>(v.z), z.t[3] = kv::from_float<T>(v.w);
                  *reinterpret_cast<uint2*>(dst) = z.u;
                } else {
                  *reinterpret_cast<float4*>(part + (int64_t)in * D + c + 4 * e) = v;
                }
              }
            }
            __syncwarp();
          }
        tc_fence_before();
      }
      done();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    while (next()) {
      const Walk<D> w = s_walk[warp];
      if (warp == 0) {
        // ---- copies ----
        const uint64_t policy = l2_policy_evict_first();
        const int per_page = a.cache.page_size / kGranule;
        const int32_t pages = pages_of(w.q.len, a.cache.page_size);
        const int32_t* table = a.table + w.at.r * a.table_stride;
        auto page_id = [&](int32_t t) -> int32_t {
          const int32_t page = ((w.blk.tile0 + t) * C::kGranules + lane) / per_page;
          return lane < C::kGranules && page < pages ? table[page] : -1;
        };
        int32_t next = page_id(w.from);
        for (int32_t t = w.from; t < w.to; ++t, ++raws) {
          const int st = raws % C::kStages;
          const int32_t id = next;
          if (t + 1 < w.to) next = page_id(t + 1);
          if (raws >= C::kStages) gate.wait(&raw_empty[st], (raws / C::kStages - 1) & 1);
          const int32_t granule = (w.blk.tile0 + t) * C::kGranules + lane, key = granule * kGranule;
          const bool here = lane < C::kGranules && id >= 0 && id < a.cache.pages;
          if (lane < C::kGranules && !here && key < w.blk.hi && key > w.blk.lo - kGranule) prompt_flag(KQ_ERR_RANGE);
          const uint32_t have = __ballot_sync(~0u, here);
          if (lane == 0) {
            s_hidden[st] = ~have & ((1u << C::kGranules) - 1);
            mbar_arrive_expect_tx(&raw_full[st], __popc(have) * L::kBytes);
          }
          __syncwarp();
          if (here)
            bulk_g2s(smem + C::kRawAt + st * C::kRaw + lane * L::kBytes,
                     a.cache.data + ((int64_t)id * a.cache.kv_heads + w.at.h) * a.cache.block_bytes +
                         (int64_t)(granule % per_page) * L::kBytes,
                     L::kBytes, &raw_full[st], policy);
        }
      } else if (warp == 1 || (warp == 3 && C::kTiles == 2)) {
        // ---- matrix products, an issuing warp per M tile ----
        const int m = warp / 2;
        if (elect_one()) {
          const bool busy = m < w.nm;  // else only the buffers' turns are taken
          if (busy) gate.wait(&q_full[m], (w.queries >> m) & 1);
          const uint32_t qk = idesc_f16(128, N), pv = idesc_f16(128, D);
          const uint64_t ad = sw128_desc(smem + m * C::kQBytes);
          for (int j = 0; j <= w.tiles; ++j) {
            if (j < w.tiles) {  // S = Q K^T of tile j
              const uint32_t kb = w.bufs + 2 * j;
              const int b = j & 1, buf = kb % C::kBuffers;
              // the buffer's last S and P are read
              if (busy && j >= 2) gate.wait(&pv_done[m][b], w.phase(m, j - 2));
              gate.wait(&buf_full[buf], (kb / C::kBuffers) & 1);
              if (busy) {
                tc_fence_after();
                const uint64_t bd = sw128_desc(smem + C::kRing + buf * C::kBuffer);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                  tc_mma_ss(tmem + (2 * m + b) * N, ad + (uint64_t)(((k / 4) * 128 * 128 + (k % 4) * 32) >> 4),
                            bd + (uint64_t)(((k / 4) * N * 128 + (k % 4) * 32) >> 4), qk, k > 0);
                tc_commit(&s_full[m][b]);
                tc_commit(&buf_empty[buf]);
              } else {
                mbar_arrive(&buf_empty[buf]);
              }
            }
            if (j > 0) {  // O += P V of tile j - 1
              const uint32_t vb = w.bufs + 2 * j - 1;
              const int b = (j - 1) & 1, buf = vb % C::kBuffers;
              gate.wait(&buf_full[buf], (vb / C::kBuffers) & 1);
              if (busy) {
                gate.wait(&p_full[m][b], w.phase(m, j - 1));
                tc_fence_after();
                const uint64_t bd = sw128_desc(smem + C::kRing + buf * C::kBuffer);
#pragma unroll
                for (int k = 0; k < N / 16; ++k)
                  tc_mma_ts(tmem + C::kO + m * D, tmem + (2 * m + b) * N + k * 8, bd + (uint64_t)((k * 32) >> 4), pv,
                            j > 1 || k > 0);
                tc_commit(&pv_done[m][b]);
                tc_commit(&buf_empty[buf]);
              } else {
                mbar_arrive(&buf_empty[buf]);
              }
            }
          }
        }
        __syncwarp();
      } else if (warp == 2) {
        // ---- a look at the scales ----
        for (int32_t t = w.from; t < w.to; ++t, ++raws) {
          const int st = raws % C::kStages, slot = (w.bufs / 2 + t - w.from) % kInfos;
          const uint8_t* raw = smem + C::kRawAt + st * C::kRaw;
          gate.wait(&raw_full[st], (raws / C::kStages) & 1);
          __syncwarp();
          const uint32_t hidden = s_hidden[st];
          const int32_t key0 = (w.blk.tile0 + t) * N;
          const bool dirty = hidden || key0 < w.blk.lo || key0 > w.blk.hi - N;
          uint32_t top[2] = {0, 0};  // the largest of the keys', of the values', as bits: NaN above infinity above the numbers
#pragma unroll
          for (int e = 0; e < C::kGranules * 2 * D / 128; ++e) {
            const int byte = 128 * e + 4 * lane, g = byte / (2 * D), in = byte % (2 * D);
            uint32_t u = *reinterpret_cast<const uint32_t*>(raw + g * L::kBytes + L::kKeyScales + in) & 0x7FFF7FFFu;
            if (dirty) {  // hidden keys' scales may be anything; a word holds two groups of one token
              const int32_t key = key0 + g * kGranule + in % D % L::kScaleSlab / (2 * L::kGroups);
              if (key < w.blk.lo || key >= w.blk.hi || (hidden >> g & 1u)) u = 0;
            }
            top[in >= D] = __vmaxu2(top[in >= D], u);
          }
          const uint32_t top_k = __reduce_max_sync(~0u, max(top[0] & 0xFFFFu, top[0] >> 16));
          const uint32_t top_v = __reduce_max_sync(~0u, max(top[1] & 0xFFFFu, top[1] >> 16));
          const bool k_down = top_k > 0x6FFFu, v_down = top_v > 0x6FFFu, nan = top_v >= 0x7C00u;
          if (nan) {
            for (int e = lane; e < N; e += 32) {
              uint32_t groups = 0;
              const int32_t key = key0 + e;
              if (key >= w.blk.lo && key < w.blk.hi && !(hidden >> (e / kGranule) & 1u)) {
                for (int gq = 0; gq < D / 32; ++gq) {
                  const uint16_t u = *reinterpret_cast<const uint16_t*>(raw + (e / kGranule) * L::kBytes + D +
                                                                        L::key_scale(e % kGranule, gq));
                  groups |= (uint32_t)((u & 0x7FFFu) >= 0x7C00u) << gq;
                }
              }
              s_nan[slot][e] = (uint8_t)groups;
            }
          }
          if (lane == 0) s_info[slot] = TileInfo{k_down ? 8.f : 1.f, v_down ? 8.f : 1.f, nan, hidden, dirty || v_down};
          __syncwarp();
          if (lane == 0) mbar_arrive(&raw_seen[st]);
        }
      } else if (warp >= kUnpackFirst) {
        // ---- unpacking ----
        const int me = (warp - kUnpackFirst) % kUnpackWarps;
        const uint32_t group = (warp - kUnpackFirst) / kUnpackWarps;
        for (int32_t t = w.from; t < w.to; ++t, ++raws) {
          if ((raws & 1) != group) continue;
          const int st = raws % C::kStages;
          const uint8_t* raw = smem + C::kRawAt + st * C::kRaw;
          gate.wait(&raw_seen[st], (raws / C::kStages) & 1);
          const TileInfo info = s_info[(w.bufs / 2 + t - w.from) % kInfos];
          const uint32_t kb = w.bufs + 2 * (t - w.from);
          if (kb >= C::kBuffers) gate.wait(&buf_empty[kb % C::kBuffers], (kb / C::kBuffers - 1) & 1);
          __syncwarp();
          uint8_t* buf = smem + C::kRing + (kb % C::kBuffers) * C::kBuffer;
#pragma unroll 1
          for (int task = me; task < N / 8 * L::kSlabs; task += kUnpackWarps)
            unpack_keys<D>(raw, buf, task / L::kSlabs, task % L::kSlabs, info.key_scale != 1.f);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&buf_full[kb % C::kBuffers]);
          const uint32_t vb = kb + 1;
          if (vb >= C::kBuffers) gate.wait(&buf_empty[vb % C::kBuffers], (vb / C::kBuffers - 1) & 1);
          __syncwarp();
          buf = smem + C::kRing + (vb % C::kBuffers) * C::kBuffer;
#pragma unroll 1
          for (int task = me; task < N / 8 * L::kSlabs; task += kUnpackWarps) {
            const int b = task / L::kSlabs;
            uint32_t valid = ~0u;
            if (info.special) {
              const int32_t key = (w.blk.tile0 + t) * N + 8 * b + 2 * (lane & 3);
              const bool held = !(info.hidden >> (b / 2) & 1u);
              valid = (held && key >= w.blk.lo && key < w.blk.hi ? 0xFFFFu : 0u) |
                      (held && key + 1 >= w.blk.lo && key + 1 < w.blk.hi ? 0xFFFF0000u : 0u);
            }
            unpack_values<D>(raw, buf, b, task % L::kSlabs, info.special, info.value_scale != 1.f, valid);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&buf_full[vb % C::kBuffers]);
            mbar_arrive(&raw_empty[st]);
          }
        }
      }
      done();
    }
    if (s_abort) {
      // a wait ran out: give the copies and products in flight the same time before their memory goes away
      if (tid == 0)
        for (uint32_t n = raws > C::kStages ? raws - C::kStages : 0; n < raws; ++n)
          mbar_wait_bounded(&raw_full[n % C::kStages], (n / C::kStages) & 1);
      if ((warp == 1 || (warp == 3 && C::kTiles == 2)) && elect_one()) {
        tc_commit(&s_drain[warp / 2]);
        mbar_wait_bounded(&s_drain[warp / 2], 0);
      }
    }
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::kColumns);
}

template <typename T, int D>
static cudaError_t launch(const Args& a, cudaStream_t st) {
  using C = PromptConfig<D>;
  static const cudaError_t opted =
      cudaFuncSetAttribute(prompt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (opted != cudaSuccess) return opted;
  return launch_dependent(prompt_kernel<T, D>, dim3(kSms), dim3(kPromptThreads), C::kSmem, st, a);
}

template <typename T>
static cudaError_t launch(int d, const Args& a, cudaStream_t st) {
  return d == 64 ? launch<T, 64>(a, st) : (d == 128 ? launch<T, 128>(a, st) : launch<T, 256>(a, st));
}

cudaError_t launch_prompt(int dtype, int head_dim, const Args& a, cudaStream_t st) {
  return dtype == KQ_F16 ? launch<__half>(head_dim, a, st) : launch<__nv_bfloat16>(head_dim, a, st);
}

}  // namespace attn

int read_prompt_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, attn::g_prompt_status, sizeof(v)) != cudaSuccess) return -1;
  if (clear && v) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(attn::g_prompt_status, &z, sizeof(z)) != cudaSuccess) return -1;
  }
  return (int)v;
}

}  // namespace kq
