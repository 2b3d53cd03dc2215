// What the delta layers' kernels share: strided rows and the step's requests.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kq.h"

namespace kq {
namespace gdn {

// Rows of heads in bytes (data null: not there).
struct Rows {
  char* data;
  int64_t token_stride, head_stride;
  __device__ __forceinline__ char* at(int64_t token, int head) const {
    return data + token * token_stride + head * head_stride;
  }
};
inline Rows rows_of(const kq_heads* h, int size) {
  return h ? Rows{static_cast<char*>(h->data), h->token_stride * size, h->head_stride * size} : Rows{nullptr, 0, 0};
}

struct Requests {
  const int32_t* q_start;
  const int32_t* kv_len;  // or null
  const int32_t* slot;
  int64_t requests, tokens, slots;
};

// A request as it is computed: tokens first .. first + count - 1, none where it is skipped or left out.
struct Request {
  int32_t first, count, slot;
  bool fresh;
  int status;  // what the device status is told: 0 or KQ_ERR_RANGE
};
__device__ __forceinline__ Request read_request(const Requests& s, int64_t r, int64_t max_new) {
  Request q{};
  const int32_t lo = s.q_start[r], hi = s.q_start[r + 1], slot = s.slot[r];
  const int64_t n = (int64_t)hi - lo;
  if (lo < 0 || n < 0 || hi > s.tokens || n > max_new || slot >= s.slots) {
    q.status = KQ_ERR_RANGE;
    return q;
  }
  if (slot < 0 || n == 0) return q;
  q.first = lo, q.count = (int32_t)n, q.slot = slot;
  q.fresh = s.kv_len && s.kv_len[r] == q.count;
  return q;
}

struct RuleArgs {
  Rows q, k, v, out;
  const char* a;
  const char* b;
  int64_t a_stride, b_stride;  // bytes
  Requests s;
  float* state;
  const float* a_log;
  const float* dt_bias;
  int64_t max_new;
  int32_t k_heads, v_heads, unit, gates;
  float eps, scale;
  int32_t short_most;  // runs of up to so many tokens go token by token, longer ones in chunks
  int32_t beside;      // runs beside the walk launched before them: it waited for what they read, and they end after it
};

constexpr int kChunk = 64;     // tokens that a prompt is worked through in at a time
// Tokens that go one by one: a run's time is its tokens', a chunk's that of 64 and three launches (48 heads of bf16, one by one
// and in a chunk: one request of 33 tokens 22 and 24 us, of 48 29 and 24; four of 33 40 and 36; 16 of 33 128 and 77).
constexpr int kShortRun = 32;

int64_t prompt_workspace(int k_heads, int v_heads, int64_t requests, int64_t tokens, int dtype);
cudaError_t launch_prompt(const RuleArgs& a, int dtype, void* ws, cudaStream_t st);
int prompt_status(int clear);

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }
// z / (1 + e^-z) for results of T, 0 below -87.3.  e^-|z| in fp32 is made as 2^p, with what p = -|z| log2(e) lacks in fp32 brought
// in afterwards: 5 units of 2^-24, 10 in all, however large |z| is.  16-bit types, whose own rounding is 2^-12 of the value or more,
// leave that out: |z| 2^-23.7 + 2^-21, 2^-17 at |z| = 87.  (4096 tokens of 48 gated fp32 heads 45 us, without what p lacks 44, by
// expf and a division 49; 5900 tokens of 10240 fp32 channels 83, 82 and 91.)
template <typename T>
__device__ __forceinline__ float silu(float z) {
  float e, r;
  if constexpr (sizeof(T) == 4) {
    const float m = fminf(fabsf(z), 126.f), p = m * -1.44269502f;  // log2(e) is 1.44269502 + 1.925963e-8 to 48 bits
    const float rest = fmaf(m, -1.92596303e-8f, fmaf(m, -1.44269502f, -p));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(p));
    e = fmaf(e * rest, 0.69314718f, e);
    z = z < 0.f ? z * e : z;
  } else {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.44269504f));
  }
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return z * r;
}
// The logarithm of a token's decay from its gate.
__device__ __forceinline__ float log_decay(float a, float a_log, float dt_bias) {
  const float x = a + dt_bias;
  return -expf(a_log) * (fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))));
}

}  // namespace gdn

// check_heads of rows that are written: no two may share an element (kq_norm.cu).
int check_out_rows(const kq_heads* h, const char* name, int dtype, int64_t tokens, int heads, int dim);
// Whether two views of rows of `dim` elements are one; whether they share an element (kq_norm.cu).  The second is exact for views
// whose tokens are one stride apart, as those of one buffer are; of others, and of more than 4096 pairs of heads that do not adjoin,
// it says no.
bool same_view(const kq_heads* x, const kq_heads* y, int64_t tokens, int heads);
bool rows_overlap(const kq_heads* x, int x_heads, const kq_heads* y, int y_heads, int64_t tokens, int dim, int dtype);
int read_norm_status(int clear);
int read_gdn_status(int clear);
int read_sample_status(int clear);

}  // namespace kq
