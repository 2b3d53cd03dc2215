// Attention of a step's new tokens over the paged 4-bit cache.
//
// For a query row (a token and one of the query heads that share a key head)
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(c q . k_j - m),  c = scale log2(e),
// in one pass over the keys with a running reference m.  With one to a few new
// tokens a request this is bound by the bytes of the cache: 4.5 bits a value,
// two multiply-adds each per query row, so about 14 flops a byte at a group of
// four heads, which CUDA cores do not keep up with at 6.8 TB/s.  The kernel
// below feeds the warp-level tensor instruction (m16n8k16, fp16 in, fp32
// accumulators) from the codes as they lie in the cache:
//
//  - A 4-bit code masked in place in an fp16 half is the subnormal q 2^-24 (or
//    16 q 2^-24 one nibble further: the other operand, or the result, is
//    divided by 16), so a 32-bit word of eight codes becomes four operand
//    registers in a shift and four ANDs, with no conversion.  The tensor core
//    aligns a subnormal's products as if it were 2^-14, so its sums lose the
//    bits that a code leaves unused: for fp32 queries the codes are shifted to
//    the top of the mantissa (four shifts and four ANDs; rows of fp32 outputs
//    were up to 1.2e-5 off without).
//  - The zero point: -8 sum(q) is added to a group's score (32 products cancel
//    no more than their own size).  8 sum(p') grows with the context while the
//    sum that is left grows with its square root, so it is subtracted every 16
//    keys, by a product that both value products of a group start from (at the
//    very end it cost fp32 rows 1.3e-5 at 500 keys), or, for fp32 queries, from
//    the codes (an fp16 subtraction, exact on subnormals).
//  - Key scales multiply the score accumulators, one per group of 32
//    dimensions, in fp32; value scales multiply the probabilities before these
//    are rounded to fp16 (p' = p * scale).  Codes stay exact throughout.
//  - Eight query rows make one tile: rows 0..7 of the first product's A
//    operand hold the queries rounded to fp16 (scaled by a power of two per
//    row), rows 8..15, for fp32 queries, what that rounding left out, so that
//    the two accumulators of a score lie in one lane.  fp32 probabilities are
//    split the same way into two products.
//  - m moves only when a score passes it by 6 (p' then reaches 2^15 at most),
//    so that the accumulators are rarely rescaled.  The power of two that brings
//    p' there is a factor of its own: as part of m it would be lost beyond 2^24.
//
// Work is counted in tiles of keys per (request, key head, eight query rows),
// laid end to end and cut into equal runs, one per warp, whatever the requests'
// lengths.  A warp has its run streamed through its own ring of shared-memory
// stages (bulk copies of whole granules, 4608 bytes a tile), so warps never
// wait for one another.  A row cut between warps leaves partial sums in the
// workspace; a second launch joins them in a fixed order.
//
// Measured (a replayed graph, both launches, 4 us of them its own): 64 requests
// of 16384 tokens, 24 query and 4 key heads of 256, fp16: 261 us, 1.21 GB of
// cache; 32 ragged requests of up to 8000, 32 and 8 heads of 128, bf16: 50 us,
// 143 MB, the same in fp32: 53 us; 8 requests of 4 new tokens on 4100, fp32: 39
// us (each eight rows unpack the keys anew).  A further byte of cache comes at
// 5.1 (D = 256) and 4.8 TB/s (D = 128); finding the runs, first copies, uneven
// ends and joining are 20 to 25 us.  Neither bytes nor issue slots are used up:
// 59 and 52% of the slots are taken while warps run (per word of eight codes five
// instructions unpack, and there are the zero points, scales and softmax),
// tensor pipe 34 and 28%; warps wait for the fixed latency of the instructions
// before (1.6 cycles of 6.5 to 7 between two) and for the pipes that unpacking
// and products share (1.0 to 1.1).
//
// 16-bit rows are 2.9e-4 from exact at fp16 where rounding the output alone is
// 2.1e-4: p' is rounded to fp16, and score products keep 13 bits or more.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kq_attn.cuh"
#include "kq_device.cuh"
#include "kq_internal.h"
#include "kq_kv.cuh"

namespace kq {
namespace attn {

__device__ unsigned int g_attn_status = 0;
__device__ __forceinline__ void attn_flag(int status) { atomicOr(&g_attn_status, 1u << status); }

constexpr int kRows = 8;             // query rows of a tile
constexpr float kSlack = 6.f;        // log2 by which a score may pass the reference
constexpr int kHeadroom = 9;         // p' <= 2^(6 + 9)
constexpr int kCombineThreads = 256;
constexpr int kJoinRows = 16, kZeroCtas = 8;
// Row tiles, as the arguments bound them, up to which cut rows are found by a CTA a row tile, which can read its request
// before attend_kernel is done; beyond, by the runs.  8 key heads of 128, 32 requests of 8000 tokens, bf16: 256 row tiles,
// 50.6 us against 53.1 by the runs; 256 of 1000: 2048, 73.1 against 73.4; 512 of 500: 4096, 97.5 against 92.0; 32 of 1000 in
// fp32 under a max_new of 512, 65536 row tiles: 252 against 29.
constexpr int64_t kManyTiles = 2048;
template <int D>
constexpr int kJoinSlices = PromptShape<D>::kRows / kJoinRows;
// Tiles of a run where there are fewer than one for every warp: one request of 1300 tokens (8 key heads of 128) takes
// 16.4 us with one, 18.5 with two, 22.6 with eight; 32 requests of 1000 take 25 with any.
constexpr int kLeastRun = 1;

template <typename T, int D>
struct Config {
  static constexpr bool kSplit = sizeof(T) == 4;        // two fp16 parts
  // Consumer warps; with the copying warp four a scheduler and 128 registers for 16-bit queries, three and 168 or two and
  // 255 for fp32.  (Three a scheduler with 16-bit queries: 64 requests of 16384 tokens, 4 key heads of 256, took 273 us
  // instead of 266, and 32 ragged ones on 8 heads of 128 51.5 instead of 50.7; at 128 registers 136 bytes spill at D = 128,
  // 48 at 256.)  At D = 256 the queries of 16-bit rows lie in shared memory, read once a tile: sums and queries in
  // registers leave room for two, 283 us.
  static constexpr bool kQShared = D == 256 && !kSplit;
  static constexpr int kWarps = (!kSplit ? 16 : (D == 256 ? 8 : 12)) - 1;
  static constexpr int kStages = kQShared ? 2 : (kWarps > 11 ? 3 : (kWarps < 8 ? 6 : 4));  // what fits beside them
  static constexpr int kQueries = kQShared ? kWarps * (D / 32) * 512 : 0;  // bytes
  static constexpr int kTileGranules = 256 / D;
  static constexpr int kTile = kTileGranules * kGranule;  // keys
  static constexpr int kStageBytes = kTileGranules * Layout<D>::kBytes;
  static constexpr int kThreads = 32 * (kWarps + 1);      // and the warp that issues the copies
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kBarriers = kRing + kQueries;
  static constexpr int kSmem = kBarriers + kWarps * kStages * 20;  // two barriers and a word a stage
};
// D = 256: one granule of 4608 bytes; 128: two; 64: four.

constexpr int kMaxWarps = 15;
// Floats of a partial result: 8 rows x D sums, 8 references, 8 weights.
constexpr int64_t partial_floats(int d) { return kRows * (int64_t)d + 2 * kRows; }
template <int D>
constexpr int64_t kPartial = kRows * (int64_t)D + 2 * kRows;

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_from_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_from(float (&d)[4], const float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    static_assert(N == 2, "two or four words");
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}

// Pair j (nibbles j and j + 4 of a word, j = 0..3) of codes as two fp16
// subnormals q * kUnit * 2^-24, odd pairs times kOdd besides.
template <bool kSplit>
struct Codes;
template <>
struct Codes<false> {
  static constexpr int kUnitLog = 0;
  static constexpr float kOdd = 16.f;
  __device__ static uint32_t pair(uint32_t w, int j) { return (j < 2 ? w : w >> 8) & (j % 2 ? 0x00F000F0u : 0x000F000Fu); }
  static constexpr uint32_t kMinus8 = 0x80088008u, kMinus8Odd = 0x80808080u;  // the zero point of either kind of pair
};
template <>
struct Codes<true> {
  static constexpr int kUnitLog = 6;
  static constexpr float kOdd = 1.f;
  __device__ static uint32_t pair(uint32_t w, int j) {
    return (j == 0 ? w << 6 : (j == 1 ? w << 2 : (j == 2 ? w >> 2 : w >> 6))) & 0x03C003C0u;
  }
  // minus the zero point, exact
  __device__ static uint32_t centred(uint32_t w, int j) {
    const uint32_t codes = pair(w, j), eights = 0x02000200u;
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&codes), *reinterpret_cast<const __half2*>(&eights));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <typename T, int D>
struct Row {
  static constexpr int kQ = D / 32;  // groups
  static constexpr int kLo = Config<T, D>::kSplit ? kQ : 1;
  // (kQShared: one group's at a time, the others in shared memory)
  uint32_t hi[Config<T, D>::kQShared ? 1 : kQ][4];  // operand A rows 0..7: dimensions (0,4), (1,5), (2,6), (3,7) of 8 c .., odd pairs / kOdd
  uint32_t lo[kLo][4];               // rows 8..15
  float zero[kQ];                    // -8 sum(q) of each group
  float factor;                      // score in log2 units = factor * accumulated
  float m, l;                        // reference (log2), this lane's share of the weight; both it and o are sums of
                                     // p = 2^(score - m) up (up is not added to m, which beyond 2^24 would lose it)
  float up;                          // 2^kHeadroom over a power of two that no value scale so far passes
  float o[kQ][2][4];                 // sums: dimensions 4 r + {0, 2} (and one further, times kOdd), rows 2 c, 2 c + 1

  __device__ __forceinline__ void add(int q, int j, const float (&t)[4]) {
    float(&x)[4] = o[q][j];
    const float2 u = add2(make_float2(x[0], x[1]), make_float2(t[0], t[1]));
    const float2 v = add2(make_float2(x[2], x[3]), make_float2(t[2], t[3]));
    x[0] = u.x, x[1] = u.y, x[2] = v.x, x[3] = v.y;
  }
};

__device__ __forceinline__ int32_t row_tiles(const Request& q) { return (q.rows + kRows - 1) / kRows; }
__device__ __forceinline__ int64_t units_of(const Args& a, const Request& q) {
  return q.rows > a.few_rows ? 0 : (int64_t)row_tiles(q) * a.cache.kv_heads * q.tiles;
}

// Position in the list of work units: request, row within it (key head outer,
// query rows inner), tile.  Warp-uniform.
struct Cursor {
  int64_t unit, end, r;
  Request q;
  int32_t row, tile;           // tile: from the request's first
  int32_t need_lo, need_hi;    // tiles that the row looks at
  int32_t all_lo, all_hi;      // keys that every query row of the tile sees
  int32_t any_lo, any_hi;      // keys that one of them sees
};

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// 1 / x of a power of two.
__device__ __forceinline__ float inverse_pow2(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

template <typename T, int D, bool kMask>
__device__ __forceinline__ void attend_tile(Row<T, D>& w, const uint8_t* stage, int32_t key0, uint32_t bad,
                                            const Cursor& cur, const uint8_t* queries, const int2* sees) {
  using L = Layout<D>;
  using C = Config<T, D>;
  using Q = Codes<C::kSplit>;
  constexpr int G = L::kGroups, kBlocks = 2 * C::kTileGranules;
  const int lane = threadIdx.x & 31, c = lane & 3;
  // The largest of the tile's value scales: 256 bytes of them whatever D, two words a lane.
  float dmax;
  {
    constexpr int kLanes = 32 / C::kTileGranules;  // of a granule
    const uint2 v = *reinterpret_cast<const uint2*>(stage + lane / kLanes * L::kBytes + L::kValueScales + lane % kLanes * 8);
    __half2 h[2] = {__habs2(*reinterpret_cast<const __half2*>(&v.x)), __habs2(*reinterpret_cast<const __half2*>(&v.y))};
    if constexpr (kMask) {  // hidden keys' scales may be anything
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int in = lane % kLanes * 8 + 4 * i;  // byte in the granule's scales
        const int32_t key = key0 + lane / kLanes * kGranule + in % L::kScaleSlab / (2 * G);
        if (key < cur.any_lo || key >= cur.any_hi || (bad >> (lane / kLanes) & 1u)) h[i] = __float2half2_rn(0.f);
      }
    }
    const __half2 m = __hmax2(h[0], h[1]);
    dmax = __half2float(__hmax(__low2half(m), __high2half(m)));
  }
  float2 s[kBlocks];
  uint32_t seen = 0;  // bit 2 b + j: the row sees token 2 c + j of block b
  float top = -INFINITY;
  // scale * (q . code) of a group, for tokens 2 c and 2 c + 1 of a block, added to `sum`
  auto score = [&](const uint32_t(&hi)[4], int q, uint32_t codes, uint32_t scale0, uint32_t scale1, float2& sum) {
    float acc[4];
    uint32_t l0 = 0, l1 = 0, l2 = 0, l3 = 0;
    if constexpr (C::kSplit) l0 = w.lo[q][0], l1 = w.lo[q][1], l2 = w.lo[q][2], l3 = w.lo[q][3];
    mma_from_zero(acc, hi[0], l0, hi[1], l1, Q::pair(codes, 0), Q::pair(codes, 1));
    mma(acc, hi[2], l2, hi[3], l3, Q::pair(codes, 2), Q::pair(codes, 3));
    float2 dot = add2(make_float2(acc[0], acc[1]), make_float2(w.zero[q], w.zero[q]));
    if constexpr (C::kSplit) dot = add2(dot, make_float2(acc[2], acc[3]));
    const float2 d0 = unpack2(scale0), d1 = unpack2(scale1);
    sum = fma2(q % 2 ? make_float2(d0.y, d1.y) : make_float2(d0.x, d1.x), dot, sum);
  };
  auto block_words = [&](int b, int sl, uint32_t(&kw)[G], uint32_t(&ks)[G]) {  // ks: G scales of token 2 c, then of 2 c + 1
    const uint8_t* g0 = stage + (b / 2) * L::kBytes;
    load_words<G>(kw, g0 + L::kKeys + sl * L::kKeySlab + (b % 2) * L::kBlock + lane * (L::kBlock / 32));
    load_words<G>(ks, g0 + L::kKeyScales + sl * L::kScaleSlab + ((b % 2) * 8 + 2 * c) * G * 2);
  };
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) s[b] = make_float2(0.f, 0.f);
  if constexpr (C::kQShared) {
    static_assert(kBlocks == 2, "one granule a tile");
#pragma unroll
    for (int sl = 0; sl < L::kSlabs; ++sl) {
      uint32_t kw0[G], ks0[G], kw1[G], ks1[G];
      block_words(0, sl, kw0, ks0);
      block_words(1, sl, kw1, ks1);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        load_words<4>(w.hi[0], queries + ((sl * G + g) * 32 + lane) * 16);
        score(w.hi[0], sl * G + g, kw0[g], ks0[g / 2], ks0[G / 2 + g / 2], s[0]);
        score(w.hi[0], sl * G + g, kw1[g], ks1[g / 2], ks1[G / 2 + g / 2], s[1]);
      }
    }
  } else {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
      for (int sl = 0; sl < L::kSlabs; ++sl) {
        uint32_t kw[G], ks[G];
        block_words(b, sl, kw, ks);
#pragma unroll
        for (int g = 0; g < G; ++g) score(w.hi[sl * G + g], sl * G + g, kw[g], ks[g / 2], ks[G / 2 + g / 2], s[b]);
      }
    }
  }
  int2 row_sees;
  if constexpr (kMask) row_sees = sees[lane];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    s[b] = mul2(s[b], make_float2(w.factor, w.factor));
    if constexpr (kMask) {
      const int32_t key = key0 + 8 * b + 2 * c;
      const bool held = !(bad >> (b / 2) & 1u);
      const bool s0 = held && key >= row_sees.x && key < row_sees.y, s1 = held && key + 1 >= row_sees.x && key + 1 < row_sees.y;
      seen |= (uint32_t)s0 << (2 * b) | (uint32_t)s1 << (2 * b + 1);
      if (!s0) s[b].x = -INFINITY;
      if (!s1) s[b].y = -INFINITY;
    }
    top = fmaxf(top, fmaxf(s[b].x, s[b].y));
  }
  // whether a reference has to move
  const bool moves = top - w.m > kSlack, grows = dmax * w.up > pow2(kHeadroom);  // (exact where they are close)
  if (__any_sync(~0u, moves || grows)) {
    // every lane of a row agrees on whether it moves: a row's own scores alone decide its reference
    float row = top;
    row = fmaxf(row, __shfl_xor_sync(~0u, row, 1));
    row = fmaxf(row, __shfl_xor_sync(~0u, row, 2));
    float d = dmax;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) d = fmaxf(d, __shfl_xor_sync(~0u, d, o));
    const float before = w.m;
    float keep_up = 1.f;
    if (row - w.m > kSlack) w.m = row;
    if (d * w.up > pow2(kHeadroom)) {
      int e;
      frexpf(d, &e);  // d <= 2^e
      const float up = fminf(w.up, pow2(kHeadroom - min(e, 17)));
      keep_up = up * inverse_pow2(w.up);
      w.up = up;
    }
    const float keep = before == -INFINITY ? 0.f : exp2_approx(before - w.m) * keep_up;
    w.l *= keep;
    const float k0 = __shfl_sync(~0u, keep, 8 * c), k1 = __shfl_sync(~0u, keep, 8 * c + 4);
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
#pragma unroll
      for (int j = 0; j < 2; ++j) w.o[q][j][0] *= k0, w.o[q][j][1] *= k1, w.o[q][j][2] *= k0, w.o[q][j][3] *= k1;
    }
  }
  const float minus = w.m == -INFINITY ? 0.f : -w.m, up = w.up;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    s[b] = add2(s[b], make_float2(minus, minus));
    s[b] = mul2(make_float2(exp2_approx(s[b].x), exp2_approx(s[b].y)), make_float2(up, up));
    w.l += s[b].x + s[b].y;
  }
#pragma unroll
  for (int gr = 0; gr < C::kTileGranules; ++gr) {
    const uint8_t* g0 = stage + gr * L::kBytes;
#pragma unroll
    for (int sl = 0; sl < L::kSlabs; ++sl) {
      uint32_t v0[G], v1[G], s0[G], s1[G];
      load_words<G>(v0, g0 + L::kValues + sl * L::kKeySlab + lane * (L::kBlock / 32));
      load_words<G>(v1, g0 + L::kValues + sl * L::kKeySlab + L::kBlock + lane * (L::kBlock / 32));
      load_words<G>(s0, g0 + L::kValueScales + sl * L::kScaleSlab + (2 * c) * G * 2);
      load_words<G>(s1, g0 + L::kValueScales + sl * L::kScaleSlab + (8 + 2 * c) * G * 2);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int q = sl * G + g;
        const float2 a0 = unpack2(s0[g / 2]), a1 = unpack2(s0[G / 2 + g / 2]);
        const float2 b0 = unpack2(s1[g / 2]), b1 = unpack2(s1[G / 2 + g / 2]);
        float2 p0 = mul2(s[2 * gr], g % 2 ? make_float2(a0.y, a1.y) : make_float2(a0.x, a1.x));
        float2 p1 = mul2(s[2 * gr + 1], g % 2 ? make_float2(b0.y, b1.y) : make_float2(b0.x, b1.x));
        if constexpr (kMask) {  // a hidden key's scale may be anything
          if (!(seen >> (4 * gr) & 1u)) p0.x = 0.f;
          if (!(seen >> (4 * gr + 1) & 1u)) p0.y = 0.f;
          if (!(seen >> (4 * gr + 2) & 1u)) p1.x = 0.f;
          if (!(seen >> (4 * gr + 3) & 1u)) p1.y = 0.f;
        }
        const uint32_t h0 = pack2(p0.x, p0.y), h1 = pack2(p1.x, p1.y);
        // The tensor core truncates as it accumulates: 16 keys at a time, joined by rounded additions.
        if constexpr (C::kSplit) {
          const float2 r0 = unpack2(h0), r1 = unpack2(h1);
          const uint32_t e0 = pack2(p0.x - r0.x, p0.y - r0.y), e1 = pack2(p1.x - r1.x, p1.y - r1.y);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t u0 = Q::centred(v0[g], 2 * j), u1 = Q::centred(v0[g], 2 * j + 1);
            const uint32_t u2 = Q::centred(v1[g], 2 * j), u3 = Q::centred(v1[g], 2 * j + 1);
            float t[4];
            mma_from_zero(t, u0, u1, u2, u3, h0, h1);
            mma(t, u0, u1, u2, u3, e0, e1);
            w.add(q, j, t);
          }
        } else {
          float zero[4];  // -8 sum(p'), in the units of either row
          mma_from_zero(zero, Q::kMinus8, Q::kMinus8Odd, Q::kMinus8, Q::kMinus8Odd, h0, h1);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float t[4];
            mma_from(t, zero, Q::pair(v0[g], 2 * j), Q::pair(v0[g], 2 * j + 1), Q::pair(v1[g], 2 * j),
                     Q::pair(v1[g], 2 * j + 1), h0, h1);
            w.add(q, j, t);
          }
        }
      }
    }
  }
}

template <int kTile>
__device__ __forceinline__ void enter_row(const Args& a, Cursor& c) {
  const int32_t x = c.row % row_tiles(c.q) * kRows;
  const int32_t i0 = x / a.group, i1 = min(c.q.n - 1, (x + kRows - 1) / a.group);
  const int32_t hi = min(c.q.len, c.q.pos0 + i1 + 1);
  const int32_t lo = first_key(a, c.q.pos0 + i0);
  c.need_lo = lo / kTile - c.q.tile0;
  c.need_hi = hi > lo ? (hi - 1) / kTile + 1 - c.q.tile0 : 0;
}
template <int kTile>
__device__ __forceinline__ void next_row(const Args& a, Cursor& c) {
  c.tile = 0;
  if (++c.row == row_tiles(c.q) * a.cache.kv_heads) {
    c.row = 0;
    do c.q = request_of(a, ++c.r, kTile);
    while (units_of(a, c.q) == 0);  // a unit remains, so some request has it
  }
  enter_row<kTile>(a, c);
}
// Moves to the next tile that its row looks at; false at the end of the run.
template <int kTile>
__device__ __forceinline__ bool seek(const Args& a, Cursor& c) {
  while (c.unit < c.end) {
    if (c.tile == c.q.tiles) next_row<kTile>(a, c);
    if (c.tile >= c.need_lo && c.tile < c.need_hi) return true;
    const int32_t to = c.tile < c.need_lo ? min(c.need_lo, c.q.tiles) : c.q.tiles;
    const int32_t step = (int32_t)min((int64_t)(to - c.tile), c.end - c.unit);
    c.tile += step;
    c.unit += step;
  }
  return false;
}

template <typename T, int D>
__device__ __forceinline__ void begin_row(const Args& a, Cursor& cur, Row<T, D>& w, uint8_t* queries, int2* sees) {
  constexpr int kQ = D / 32;
  using C = Codes<Config<T, D>::kSplit>;
  constexpr float kZero = -8.f * (1 << C::kUnitLog) / 16777216.f;
  const int lane = threadIdx.x & 31, c = lane & 3;
  const int32_t x = cur.row % row_tiles(cur.q) * kRows + lane / 4, h = cur.row / row_tiles(cur.q);
  const int32_t i = x / a.group;
  const bool live = i < cur.q.n;
  const int32_t pos = cur.q.pos0 + i;
  // rows past the last one hold zeros and see everything: they never ask for the masked path
  const int32_t key_lo = live ? first_key(a, pos) : 0, key_hi = live ? max(0, min(pos + 1, cur.q.len)) : 0x7fffffff;
  sees[lane] = make_int2(key_lo, key_hi);  // a lane reads back what it wrote
  cur.all_lo = __reduce_max_sync(~0u, key_lo), cur.all_hi = __reduce_min_sync(~0u, key_hi);
  cur.any_lo = __reduce_min_sync(~0u, live ? key_lo : 0x7fffffff);
  cur.any_hi = __reduce_max_sync(~0u, live ? key_hi : 0);
  const T* src = static_cast<const T*>(a.q) + (int64_t)(cur.q.first + i) * a.q_token +
                 (int64_t)(h * a.group + x % a.group) * a.q_head + 8 * c;
  float x8[kQ][8], top = 0.f;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    if (live) {
      kv::load8(src + 32 * q, x8[q]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x8[q][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x8[q][j]));
  }
  top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
  top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
  // the row times 2^e lies below 2^15 (2^e itself stays a normal number)
  int e = 0;
  if (top > 0.f && top <= 3.402823466e38f) frexpf(top, &e);
  e = min(max(15 - e, -110), 110);
  const float up = ldexpf(1.f, e);
  w.factor = ldexpf(a.scale * 1.4426950408889634f, 24 - C::kUnitLog - e);
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    float zh = 0.f, zl = 0.f;
    uint32_t(&hi)[4] = w.hi[Config<T, D>::kQShared ? 0 : q];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float f = p % 2 ? 1.f / C::kOdd : 1.f, back = p % 2 ? C::kOdd : 1.f;
      const float u = x8[q][p] * up * f, v = x8[q][p + 4] * up * f;
      hi[p] = pack2(u, v);
      const float2 r = unpack2(hi[p]);
      zh += (r.x + r.y) * back;
      if constexpr (Config<T, D>::kSplit) {
        w.lo[q][p] = pack2(u - r.x, v - r.y);
        const float2 t = unpack2(w.lo[q][p]);
        zl += (t.x + t.y) * back;
      }
    }
    if constexpr (Config<T, D>::kQShared)  // a lane reads back what it wrote
      *reinterpret_cast<uint4*>(queries + (q * 32 + lane) * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    zh += zl;
    zh += __shfl_xor_sync(~0u, zh, 1);
    zh += __shfl_xor_sync(~0u, zh, 2);
    w.zero[q] = zh * kZero;
#pragma unroll
    for (int j = 0; j < 4; ++j) w.o[q][0][j] = w.o[q][1][j] = 0.f;
  }
  w.up = pow2(kHeadroom + 24);
  w.m = live ? -INFINITY : 0.f;
  w.l = 0.f;
}

// What a sum over codes is multiplied by.
template <typename T, int D>
constexpr float kOut = 16777216.f / (1 << Codes<Config<T, D>::kSplit>::kUnitLog);

// Ends a row (whole: the output itself) or this warp's part of it.
template <typename T, int D>
__device__ __forceinline__ void end_row(const Args& a, const Cursor& cur, Row<T, D>& w, float* partial) {
  const int lane = threadIdx.x & 31, r = lane / 4, c = lane & 3;
  w.l += __shfl_xor_sync(~0u, w.l, 1);
  w.l += __shfl_xor_sync(~0u, w.l, 2);
  const int32_t x0 = cur.row % row_tiles(cur.q) * kRows, h = cur.row / row_tiles(cur.q);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float l = __shfl_sync(~0u, w.l, 8 * c + 4 * j);
    const int32_t x = x0 + 2 * c + j, i = x / a.group;
    if (i >= cur.q.n) continue;
    const float f = partial ? inverse_pow2(w.up) : (l == 0.f ? 0.f : kOut<T, D> / l);
    T* dst = static_cast<T*>(a.out) + (int64_t)(cur.q.first + i) * a.out_token +
             (int64_t)(h * a.group + x % a.group) * a.out_head;
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
      const float f16 = f / Codes<Config<T, D>::kSplit>::kOdd;
      const float4 v = make_float4(w.o[q][0][j] * f, w.o[q][0][j + 2] * f16, w.o[q][1][j] * f, w.o[q][1][j + 2] * f16);
      if (partial) {
        *reinterpret_cast<float4*>(partial + (2 * c + j) * D + 32 * q + 4 * r) = v;
      } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(dst + 32 * q + 4 * r) = v;
      } else {
        union { uint2 u; T t[4]; } y;
        y.t[0] = kv::from_float<T>(v.x), y.t[1] = kv::from_float<T>(v.y);
        y.t[2] = kv::from_float<T>(v.z), y.t[3] = kv::from_float<T>(v.w);
        *reinterpret_cast<uint2*>(dst + 32 * q + 4 * r) = y.u;
      }
    }
  }
  if (partial && c == 0) {
    partial[kRows * D + r] = w.m;
    partial[kRows * D + kRows + r] = w.l * inverse_pow2(w.up);
  }
}

// A consumer warp per run, and one more warp whose lane i issues the copies of
// consumer i's tiles, some stages ahead of it.
template <typename T, int D>
__global__ void __launch_bounds__(Config<T, D>::kThreads, 1) attend_kernel(Args a) {
  using L = Layout<D>;
  using C = Config<T, D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_first[C::kThreads];  // units before each request of a chunk
  __shared__ int64_t s_warp[C::kWarps + 1];
  __shared__ Cursor s_cursor[C::kWarps];
  __shared__ int2 s_sees[C::kWarps][32];  // keys that a lane's row sees
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool producer = warp == C::kWarps;
  const int me = producer ? min(lane, C::kWarps - 1) : warp;  // the consumer that this thread works for
  uint8_t* ring = smem + me * C::kStages * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarriers) + me * C::kStages;
  uint64_t* empty = full + C::kWarps * C::kStages;
  volatile uint32_t* hidden = reinterpret_cast<uint32_t*>(smem + C::kBarriers + C::kWarps * C::kStages * 16) + me * C::kStages;
  if (!producer && lane < C::kStages) {
    mbar_init(&full[lane], 1);
    mbar_init(&empty[lane], 1);
    fence_barrier_init();
  }
  grid_dependency_wait();
  allow_dependent_launch();

  // The units before each request, kThreads requests at a time: once for the total, and (with more than one chunk)
  // again to find where this thread's run begins.
  const int64_t run = (int64_t)me * kSms + blockIdx.x;
  const int chunks = (int)((a.requests + C::kThreads - 1) / C::kThreads);
  int64_t total = 0;
  bool out_of_range = false;
  Cursor cur;
  cur.unit = cur.end = 0;
  for (int pass = 0; pass < (chunks > 1 ? 2 : 1); ++pass) {
    int64_t before = 0;
    for (int ch = 0; ch < chunks; ++ch) {
      const int64_t r = (int64_t)ch * C::kThreads + tid;
      const bool mine = r < a.requests;
      int64_t u = 0;
      if (mine) u = units_of(a, request_of(a, r, C::kTile, &out_of_range));
      int64_t inc = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += x;
      }
      __syncthreads();  // the previous chunk's sums have been read
      if (lane == 31) s_warp[warp] = inc;
      __syncthreads();
      int64_t at = before + inc - u, sum = before;
#pragma unroll
      for (int i = 0; i <= C::kWarps; ++i) {
        if (i < warp) at += s_warp[i];
        sum += s_warp[i];
      }
      s_first[tid] = at;
      if (blockIdx.x == 0 && pass == 0 && mine && !a.by_runs) a.base[r] = at;
      __syncthreads();
      if (pass == 0) total = sum;
      if (pass == 1 || chunks == 1) {
        const Runs runs(total, (int64_t)kSms * C::kWarps, kLeastRun);
        const int64_t u0 = runs.start(run), u1 = runs.start(run + 1);
        if (run < runs.count && u0 >= before && u0 < sum) {
          int l = 0, h = (int)min((int64_t)C::kThreads, a.requests - (int64_t)ch * C::kThreads);
          while (h - l > 1) {  // the last request that starts at or before u0
            const int m = (l + h) >> 1;
            if (s_first[m] <= u0) l = m; else h = m;
          }
          cur.unit = u0, cur.end = u1;
          cur.r = (int64_t)ch * C::kThreads + l;
          cur.q = request_of(a, cur.r, C::kTile);
          const int64_t in = u0 - s_first[l];
          cur.row = (int32_t)(in / cur.q.tiles);
          cur.tile = (int32_t)(in % cur.q.tiles);
        }
      }
      before = sum;
    }
  }
  if (blockIdx.x == 0) {
    if (tid == 0 && !a.by_runs) a.base[a.requests] = total;
    if (out_of_range) attn_flag(KQ_ERR_RANGE);
  }
  if (cur.unit < cur.end) enter_row<C::kTile>(a, cur);
  if (a.by_runs && !producer && lane == 0) {  // (while the first tiles are on their way)
    TileStart start{};
    start.from = start.to = (int32_t)run;
    if (cur.unit < cur.end) {
      const Runs runs(total, (int64_t)kSms * C::kWarps, kLeastRun);
      const int64_t lo = cur.unit - cur.tile;
      start.from = (int32_t)runs.of(lo), start.to = (int32_t)runs.of(lo + cur.q.tiles - 1);
      start.later = runs.start(start.from) < lo;
      start.first = cur.q.first, start.rows = cur.q.rows;
      start.x0 = cur.row % row_tiles(cur.q) * kRows, start.h = cur.row / row_tiles(cur.q);
    }
    a.starts[run] = start;
  }
  if (!producer && cur.unit == cur.end) return;

  if (producer) {
    const uint64_t policy = l2_policy_evict_first();
    const int per_page = a.cache.page_size / kGranule;
    const int64_t page_bytes = a.cache.kv_heads * a.cache.block_bytes;
    const bool in_one = per_page % C::kTileGranules == 0;  // a tile lies in one page
    // The row's tiles that are left, the page and granule within it of the next one, and what a row fixes; page `at`
    // of the request is `id`, the page after it in flight.
    int32_t left = 0, page = 0, sub = 0, pages = 0, at = -1, id = -1, next = -1;
    const int32_t* row = nullptr;
    const uint8_t* head = nullptr;
    int64_t row_of = -1;
    uint32_t made = 0;
    bool more = lane < C::kWarps;
    auto enter = [&]() {  // the next tile's row
      more = more && seek<C::kTile>(a, cur);
      if (!more) return;
      left = (int32_t)min((int64_t)(min(cur.need_hi, cur.q.tiles) - cur.tile), cur.end - cur.unit);
      if (cur.r != row_of) {
        row_of = cur.r, row = a.table + cur.r * a.table_stride, at = -1;
        pages = pages_of(cur.q.len, a.cache.page_size);  // the table's row holds them
      }
      const int32_t g0 = (cur.q.tile0 + cur.tile) * C::kTileGranules;
      page = g0 / per_page, sub = g0 - page * per_page;
      head = a.cache.data + cur.row / row_tiles(cur.q) * a.cache.block_bytes;
      // the tiles that follow are the row's
      cur.tile += left;
      cur.unit += left;
    };
    // The address of the granule at (page, sub), or NULL.
    auto source = [&]() -> const uint8_t* {
      if (page >= pages) return nullptr;
      if (page != at) {
        id = at >= 0 && page == at + 1 ? next : row[page];
        at = page;
        next = page + 1 < pages ? row[page + 1] : -1;
      }
      if (id >= 0 && id < a.cache.pages) return head + id * page_bytes + (int64_t)sub * L::kBytes;
      const int32_t key = (page * per_page + sub) * kGranule;
      if (key < cur.q.len && key > cur.q.lo - (in_one ? C::kTile : kGranule)) attn_flag(KQ_ERR_RANGE);
      return nullptr;  // (a page below a sliding window may be gone)
    };
    enter();
    // The lanes stay together: whichever find a free stage issue a tile, and only where none does the warp sleeps.  (With
    // a wait per lane the slowest consumer held up all the others' copies; and a tile's own arithmetic has to stay
    // short, or its stage comes back late: up to 15 lanes share the warp.)
    long long since = clock64();
    while (__any_sync(~0u, more)) {
      const int st = made % C::kStages;
      const bool free = more && (made < C::kStages || mbar_test_wait(&empty[st], (made / C::kStages - 1) & 1));
      if (!__any_sync(~0u, free)) {
        if (__any_sync(~0u, clock64() - since > kWaitLimitCycles)) break;  // a consumer gave up, and reports it
        __nanosleep(20);
        continue;
      }
      since = clock64();
      if (!free) continue;
      uint8_t* dst = ring + st * C::kStageBytes;
      if (in_one) {
        const uint8_t* src = source();
        hidden[st] = src ? 0u : (1u << C::kTileGranules) - 1;
        mbar_arrive_expect_tx(&full[st], src ? C::kStageBytes : 0);
        if (src) bulk_g2s(dst, src, C::kStageBytes, &full[st], policy);
        sub += C::kTileGranules;
        if (sub == per_page) sub = 0, ++page;
      } else {
        const uint8_t* src[C::kTileGranules];
        uint32_t have = 0;
#pragma unroll
        for (int i = 0; i < C::kTileGranules; ++i) {
          src[i] = source();
          have |= (uint32_t)(src[i] != nullptr) << i;
          if (++sub == per_page) sub = 0, ++page;
        }
        hidden[st] = ~have & ((1u << C::kTileGranules) - 1);
        mbar_arrive_expect_tx(&full[st], __popc(have) * L::kBytes);
#pragma unroll
        for (int i = 0; i < C::kTileGranules; ++i)
          if (src[i]) bulk_g2s(dst + i * L::kBytes, src[i], L::kBytes, &full[st], policy);
      }
      ++made;
      if (--left == 0) enter();
    }
    // the ring stays until the last copies have landed (they have, unless a consumer gave up)
    if (lane < C::kWarps)
      for (uint32_t i = made > C::kStages ? made - C::kStages : 0; i < made; ++i)
        mbar_wait_bounded(&full[i % C::kStages], (i / C::kStages) & 1);
    return;
  }

  // The cursor waits in shared memory while a row's tiles go by.
  Cursor& c = s_cursor[warp];
  uint8_t* queries = smem + C::kRing + warp * (C::kQueries / C::kWarps);
  Row<T, D> w;
  bool first = true;
  uint32_t used = 0;
  while (cur.unit < cur.end) {
    if (cur.tile == cur.q.tiles) next_row<C::kTile>(a, cur);
    begin_row<T, D>(a, cur, w, queries, s_sees[warp]);
    __syncwarp();
    if (lane == 0) c = cur;
    __syncwarp();
    const int32_t from = c.tile;
    const int32_t to = (int32_t)min((int64_t)c.q.tiles, from + (c.end - c.unit));
    for (int32_t t = max(from, c.need_lo); t < min(to, c.need_hi); ++t) {
      const int st = used % C::kStages;
      if (!mbar_wait_suspend(&full[st], (used / C::kStages) & 1)) {
        attn_flag(KQ_ERR_TIMEOUT);
        return;
      }
      const int32_t key0 = (c.q.tile0 + t) * C::kTile;
      const uint32_t bad = hidden[st];
      const uint8_t* stage = ring + st * C::kStageBytes;
      if (bad || key0 < c.all_lo || key0 > c.all_hi - C::kTile)
        attend_tile<T, D, true>(w, stage, key0, bad, c, queries, s_sees[warp]);
      else
        attend_tile<T, D, false>(w, stage, key0, 0, c, queries, s_sees[warp]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      ++used;
    }
    const bool whole = from == 0 && to == c.q.tiles;
    float* partial = whole ? nullptr : a.partials + (2 * run + (first ? 0 : 1)) * kPartial<D>;
    end_row<T, D>(a, c, w, partial);
    first = false;
    cur = c;
    cur.unit += to - from;
    cur.tile = to;
  }
}

// One part of a row joined to what there is of it (a row of NaN scores keeps its reference at -inf and its weight NaN).
template <int N>
struct Sum {
  float ref = -INFINITY, weight = 0.f, acc[N] = {};
  __device__ __forceinline__ void join(float m, float l, const float (&o)[N]) {
    const float now = fmaxf(ref, m);
    const float keep = ref == -INFINITY ? 0.f : exp2_approx(ref - now), f = m == -INFINITY ? 0.f : exp2_approx(m - now);
    weight = weight * keep + (m == -INFINITY ? l : l * f);
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = acc[e] * keep + o[e] * f;
    ref = now;
  }
};
// N consecutive values, N = 2, 4 or 8.
template <int N>
__device__ __forceinline__ void load_part(float (&o)[N], const float* p) {
  if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    o[0] = v.x, o[1] = v.y;
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + e);
      o[e] = v.x, o[e + 1] = v.y, o[e + 2] = v.z, o[e + 3] = v.w;
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_row(T* p, const float (&o)[N], float f) {
  union { uint32_t u[N * sizeof(T) / 4]; T t[N]; } y;
#pragma unroll
  for (int e = 0; e < N; ++e) y.t[e] = kv::from_float<T>(o[e] * f);
#pragma unroll
  for (int e = 0; e < (int)(N * sizeof(T) / 4); ++e) reinterpret_cast<uint32_t*>(p)[e] = y.u[e];
}

// Joins, in run order, the parts of rows that were cut between runs, and writes
// zeros where a row sees nothing.
//  - The first few_ctas CTAs: rows of row tiles of attend_kernel (eight rows of a
//    request and key head, cut at the same places).  The warps share out rows,
//    and then the parts of a row.
//    Without kByRuns, rows_per_cta rows of one row tile each, whether they were
//    cut or not, as many CTAs as requests of max_new tokens would have.
//    With it, eight boundaries between runs each, and the row tiles whose first
//    boundary is among them: a grid that follows from the number of runs,
//    whatever the caller's bounds are.
//  - The next: 16 rows of the row block that a boundary between two runs of the
//    prompt kernel falls in.
//  - The last kZeroCtas: what sees nothing of prompts (with kByRuns, of all requests).
constexpr int kBoundaries = 8;

// Rows first .. first + n - 1 of a row tile that runs `from` .. `to` hold, by the whole CTA; out(row): where a row goes.  Its
// sums lie in a run's first slot, in the second of run `from` where the run began with another row (`later`).
template <typename T, int D, typename Out>
__device__ __forceinline__ void join_rows(const Args& a, int first, int n, int32_t from, int32_t to, int32_t later, const Out& out,
                                          float (*s_sum)[D], float* s_ref, float* s_weight) {
  constexpr int kPer = D / 32, kWarps = kCombineThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // a power of two of rows, the remaining factor of the warps on the parts of each
  const int wide = n > 4 ? 8 : (n > 2 ? 4 : n), shares = kWarps / wide, in = warp % wide, share = warp / wide;
  Sum<kPer> s;
  if (in < n) {
#pragma unroll 4
    for (int32_t w = from + share; w <= to; w += shares) {
      const float* p = a.partials + (2 * (int64_t)w + (w == from ? later : 0)) * kPartial<D>;
      float o[kPer];
      load_part<kPer>(o, p + (first + in) * D + lane * kPer);
      s.join(p[kRows * D + first + in], p[kRows * D + kRows + first + in], o);
    }
  }
  if (lane == 0) s_ref[warp] = s.ref, s_weight[warp] = s.weight;
#pragma unroll
  for (int e = 0; e < kPer; ++e) s_sum[warp][lane * kPer + e] = s.acc[e];
  __syncthreads();
  if (share > 0 || in >= n) return;
  for (int v = 1; v < shares; ++v) {
    float o[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = s_sum[in + v * wide][lane * kPer + e];
    s.join(s_ref[in + v * wide], s_weight[in + v * wide], o);
  }
  store_row<T, kPer>(out(first + in) + lane * kPer, s.acc, s.weight == 0.f ? 0.f : kOut<T, D> / s.weight);
}

template <typename T, int D, bool kByRuns>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(Args a, int slices, int tile_rows, int rows_per_cta, int few_ctas,
                                                                  int prompt_ctas) {
  using C = Config<T, D>;
  using P = PromptShape<D>;
  constexpr int kPer = D / 32, kWarps = kCombineThreads / 32;
  __shared__ float s_sum[kWarps][D], s_ref[kWarps], s_weight[kWarps];
  __shared__ int64_t s_list[kCombineThreads];
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (What the call was given may be read before the launch in front is done, from L2: that one let this one start after
  // all before it were.)
  auto launches_before = []() {
    grid_dependency_wait();
    allow_dependent_launch();
  };
  auto row_out = [&](int32_t token0, int h, int32_t x) {
    return static_cast<T*>(a.out) + (int64_t)(token0 + x / a.group) * a.out_token +
           (int64_t)(h * a.group + x % a.group) * a.out_head;
  };
  if (!kByRuns && blockIdx.x < few_ctas) {
    const int per_tile = (tile_rows + rows_per_cta - 1) / rows_per_cta, part = blockIdx.x % per_tile;
    const int tile = blockIdx.x / per_tile;
    const int slice = tile % slices, h = tile / slices % a.cache.kv_heads;
    const int64_t r = tile / slices / a.cache.kv_heads;
    const Request q = request_of<true>(a, r, C::kTile);
    launches_before();
    const int first = part * rows_per_cta;
    const int32_t x0 = slice * kRows + first;
    if (q.rows > a.few_rows || x0 >= q.rows) return;
    const int n = min(rows_per_cta, q.rows - x0);
    if (q.tiles == 0) {
      for (int e = tid; e < n * D; e += kCombineThreads) row_out(q.first, h, x0 + e / D)[e % D] = kv::from_float<T>(0.f);
      return;
    }
    const Runs runs(a.base[a.requests], (int64_t)kSms * C::kWarps, kLeastRun);
    const int64_t lo = a.base[r] + ((int64_t)h * row_tiles(q) + slice) * q.tiles;
    const int32_t from = (int32_t)runs.of(lo), to = (int32_t)runs.of(lo + q.tiles - 1);
    if (from == to) return;
    join_rows<T, D>(a, first, n, from, to, runs.start(from) >= lo ? 0 : 1,
                    [&](int row) { return row_out(q.first, h, slice * kRows + row); }, s_sum, s_ref, s_weight);
    return;
  }
  launches_before();
  if (kByRuns && blockIdx.x < few_ctas) {
    // lane i of every warp looks at the i-th boundary
    const int32_t b0 = 1 + kBoundaries * blockIdx.x, b = b0 + lane % kBoundaries;
    TileStart start{};
    if (b < kSms * C::kWarps) start = a.starts[b];
    const uint32_t firsts = __ballot_sync(~0u, b == start.from + 1 && b <= start.to) & ((1u << kBoundaries) - 1);
    for (uint32_t left = firsts; left; left &= left - 1) {
      const int i = __ffs(left) - 1;
      const int32_t from = __shfl_sync(~0u, start.from, i), to = __shfl_sync(~0u, start.to, i);
      const int32_t later = __shfl_sync(~0u, start.later, i), token0 = __shfl_sync(~0u, start.first, i);
      const int32_t x0 = __shfl_sync(~0u, start.x0, i), rows = __shfl_sync(~0u, start.rows, i), h = __shfl_sync(~0u, start.h, i);
      join_rows<T, D>(a, 0, min(kRows, rows - x0), from, to, later, [&](int row) { return row_out(token0, h, x0 + row); }, s_sum,
                      s_ref, s_weight);
      __syncthreads();
    }
    return;
  }
  const int at = blockIdx.x - few_ctas;
  if (at < prompt_ctas) {
    const int64_t b = at / kJoinSlices<D> + 1;
    const Runs runs(*a.prompt_total, kSms, P::kLeastRun);
    if (b >= runs.count) return;
    const RunStart start = a.prompt_starts[b];
    // no tile of the row lies before this boundary, or an earlier boundary lies between its tiles too
    const int64_t lo = start.lo + P::kRowCost;
    if (start.at <= P::kRowCost || lo < runs.start(b - 1)) return;
    const Request q = request_of(a, start.r, P::kKeys);
    const int32_t first = at % kJoinSlices<D> * kJoinRows;
    const int32_t rows = min(P::kRows, q.rows - start.k * P::kRows);
    const int64_t w1 = runs.of(lo + start.tiles - 1);
#pragma unroll
    for (int i = 0; i < kJoinRows / kWarps; ++i) {
      const int32_t in = first + i * kWarps + warp;
      if (in >= rows) break;
      Sum<kPer> s;
#pragma unroll 2
      for (int64_t w = b - 1; w <= w1; ++w) {
        const float* p = a.prompt_partials + (2 * w + (runs.start(w) >= start.lo ? 0 : 1)) * P::kPartial;
        float o[kPer];
        load_part<kPer>(o, p + (int64_t)in * D + lane * kPer);
        s.join(p[P::kRows * D + in], p[P::kRows * D + P::kRows + in], o);
      }
      store_row<T, kPer>(row_out(q.first, start.h, start.k * P::kRows + in) + lane * kPer, s.acc,
                         s.weight == 0.f ? 0.f : 1.f / s.weight);
    }
    return;
  }
  // Every thread looks at a request; the CTA then writes the rows of those that were found.
  for (int64_t r0 = at - prompt_ctas; r0 < a.requests; r0 += (int64_t)kZeroCtas * kCombineThreads) {
    const int64_t mine = r0 + (int64_t)kZeroCtas * tid;
    if (tid == 0) s_count = 0;
    __syncthreads();
    if (mine < a.requests) {
      const Request q = request_of(a, mine, C::kTile);
      // (of a prompt only where it brings more tokens than it holds, or its length was cut)
      if (q.rows > a.few_rows ? q.pos0 < 0 || q.len != q.pos0 + q.n : kByRuns && q.n > 0 && q.tiles == 0)
        s_list[atomicAdd(&s_count, 1)] = mine;
    }
    __syncthreads();
    for (int i = 0; i < s_count; ++i) {
      const int64_t r = s_list[i];
      const Request q = request_of(a, r, P::kKeys);
      for (int32_t x0 = 0; x0 < q.rows; x0 += P::kRows) {
        if (q.rows > a.few_rows && row_block<D>(a, q, x0 / P::kRows).tiles) continue;
        const int32_t rows = min(P::kRows, q.rows - x0);
        for (int64_t e = tid; e < (int64_t)rows * a.cache.kv_heads * D; e += kCombineThreads)
          row_out(q.first, (int)(e / D / rows), x0 + (int32_t)(e / D % rows))[e % D] = kv::from_float<T>(0.f);
      }
    }
    __syncthreads();
  }
}

// Bounds from the call's arguments: query rows of a key head that one request brings to attend_kernel, and row tiles of all
// requests and key heads (2^40 stands for anything large).
static int64_t query_rows_of(const Args& a) { return std::min<int64_t>(a.few_rows, std::min(a.max_new, a.tokens) * a.group); }
static int64_t row_tiles_of(const Args& a) {
  const int64_t slices = (query_rows_of(a) + kRows - 1) / kRows * a.cache.kv_heads, most = (int64_t)1 << 40;
  return slices > most / a.requests ? most : slices * a.requests;
}

template <typename T, int D>
static cudaError_t launch(const Args& a, cudaStream_t st) {
  using C = Config<T, D>;
  static const cudaError_t opted =
      cudaFuncSetAttribute(attend_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (opted != cudaSuccess) return opted;
  if (cudaError_t e = launch_dependent(attend_kernel<T, D>, dim3(kSms), dim3(C::kThreads), C::kSmem, st, a)) return e;
  if (a.few_rows != 0x7fffffff) {
    if (cudaError_t e = launch_prompt(sizeof(T) == 4 ? -1 : (std::is_same_v<T, __half> ? KQ_F16 : KQ_BF16), D, a, st)) return e;
  }
  const bool prompts = a.few_rows != 0x7fffffff;
  // A row a CTA where that stays few: one request of 20000 tokens, whose rows lie in a hundred parts, took 28 us instead
  // of 52 with eight rows a CTA; with 256 row tiles a row a CTA cost 32 requests of 8000 tokens 4 us more.
  const int64_t tiles = row_tiles_of(a);
  const int slices = (int)(query_rows_of(a) + kRows - 1) / kRows, tile_rows = (int)std::min<int64_t>(query_rows_of(a), kRows);
  const int rows_per_cta = tiles <= 64 ? 1 : kRows;
  const int few_ctas = a.by_runs ? ((int)kSms * C::kWarps + kBoundaries - 2) / kBoundaries
                                 : (int)tiles * ((tile_rows + rows_per_cta - 1) / rows_per_cta);
  const int prompt_ctas = prompts ? kJoinSlices<D> * (kSms - 1) : 0;
  return launch_dependent(a.by_runs ? combine_kernel<T, D, true> : combine_kernel<T, D, false>,
                          dim3((unsigned)(few_ctas + prompt_ctas + (prompts || a.by_runs ? kZeroCtas : 0))), dim3(kCombineThreads), 0,
                          st, a, slices, tile_rows, rows_per_cta, few_ctas, prompt_ctas);
}

template <typename T>
static cudaError_t launch(int d, const Args& a, cudaStream_t st) {
  return d == 64 ? launch<T, 64>(a, st) : (d == 128 ? launch<T, 128>(a, st) : launch<T, 256>(a, st));
}

// Query rows of a request up to which attend_kernel takes it, with 16-bit queries; beyond, the prompt kernel.  8 requests
// of 4096 tokens, 32 query and 8 key heads of 128: 32 rows 54 us here against 59, 64 rows 85 against 60; 24 and 4 heads of
// 256: 24 rows 52 against 62, 48 rows 73 against 63; 14 and 2 heads of 64: 56 rows 31 against 35, 112 rows 39 against 36.
constexpr int32_t few_rows_of(int d) { return d == 64 ? 64 : 40; }

// The workspace: byte offsets of its parts, and its size.
struct Workspace {
  size_t base, starts, partials, prompt_total, prompt_starts, prompt_partials, bytes;
};
static Workspace workspace(const kq_kv_cache* c, int32_t q_heads, int64_t requests, int64_t tokens, int64_t max_new) {
  const int d = c->head_dim;
  const int64_t group = q_heads / c->kv_heads;
  const bool prompts = std::min(max_new, tokens) > few_rows_of(d) / group;
  const int64_t partial = d == 256 ? PromptShape<256>::kPartial : (d == 128 ? PromptShape<128>::kPartial : PromptShape<64>::kPartial);
  Workspace w{};
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += (size_t)round_up(bytes, 16);
    return here;
  };
  w.base = take((requests + 1) * 8);
  w.starts = take(kSms * kMaxWarps * (int64_t)sizeof(TileStart));
  w.partials = take(2 * kSms * kMaxWarps * partial_floats(d) * 4);
  w.prompt_total = take(prompts ? 8 : 0);
  w.prompt_starts = take(prompts ? kSms * (int64_t)sizeof(RunStart) : 0);
  w.prompt_partials = take(prompts ? 2 * kSms * partial * 4 : 0);
  w.bytes = at;
  return w;
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
  return attn::workspace(cache, q_heads, requests, tokens, max_new).bytes;
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
  a.table_stride = table_stride, a.requests = requests, a.tokens = tokens, a.max_new = max_new;
  a.window = (int32_t)(window > 0x7fffffff ? 0x7fffffff : window);
  a.q_heads = q_heads, a.group = q_heads / cache->kv_heads, a.scale = scale;
  const attn::Workspace w = attn::workspace(cache, q_heads, requests, tokens, max_new);
  uint8_t* ws = static_cast<uint8_t*>(d_ws);
  a.base = reinterpret_cast<int64_t*>(ws + w.base);
  a.starts = reinterpret_cast<attn::TileStart*>(ws + w.starts);
  a.partials = reinterpret_cast<float*>(ws + w.partials);
  a.prompt_total = reinterpret_cast<int64_t*>(ws + w.prompt_total);
  a.prompt_starts = reinterpret_cast<attn::RunStart*>(ws + w.prompt_starts);
  a.prompt_partials = reinterpret_cast<float*>(ws + w.prompt_partials);
  const bool prompts = dtype != KQ_F32 && std::min(max_new, tokens) > attn::few_rows_of(cache->head_dim) / a.group;
  a.few_rows = prompts ? attn::few_rows_of(cache->head_dim) : 0x7fffffff;
  a.by_runs = attn::row_tiles_of(a) > attn::kManyTiles;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  KQ_CUDA_TRY(dtype == KQ_F32 ? attn::launch<float>(cache->head_dim, a, st)
                              : (dtype == KQ_F16 ? attn::launch<__half>(cache->head_dim, a, st)
                                                 : attn::launch<__nv_bfloat16>(cache->head_dim, a, st)));
  return KQ_OK;
}

}  // extern "C"
