"""One attention layer of a decode, on the quantized weights and the 4-bit cache.

    python examples/decode_layer.py [--requests 4] [--prompt 37] [--steps 5]

Runs a prompt and then single-token steps for a few requests through the calls
a decode makes, layer by layer (here one layer with the sizes of the Qwen3-4B
decode workload: hidden size 2560, 32 query and 8 key heads of 128):

    kq_slot_map       block tables, positions and slots from the requests' lengths
    kq_gemm_small_m   the q, k and v projections (Q8_0 weights, one stream for all rows)
    kq_kv_append      query/key norms and rotation; keys and values into the cache
    kq_attn_paged     attention over the block table
    kq_gemm_small_m   the output projection

and checks the last step's attention against FP64 over the same cache.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_weight_streaming_gb300 as kq  # noqa: E402
import synth  # noqa: E402
import workloads  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, D, PAGE = 2560, 32, 8, 128, 32


class Layer:
    """The layer's weights, rotation table and cache."""

    def __init__(self, requests, capacity, seed=0):
        mat = lambda n, k, i: workloads.build_matrix("q8_0", n, k, seed, synth.stream_id("test", synth.ROLE_W, 700 + i))  # noqa: E731
        self.wq, self.wk, self.wv = mat(Q_HEADS * D, HIDDEN, 0), mat(KV_HEADS * D, HIDDEN, 1), mat(KV_HEADS * D, HIDDEN, 2)
        self.wo = mat(HIDDEN, Q_HEADS * D, 3)
        rope = torch.from_numpy(kq.kq_rope_table_host(capacity, D, 1e6)).cuda()
        ones = torch.ones(D, device="cuda")
        self.norm = kq.QKNorm(Q_HEADS, KV_HEADS, D, D, ones, ones.clone(), rope)
        self.pages = requests * (-(-capacity // PAGE))
        self.cache = kq.KVCache(self.pages, PAGE, KV_HEADS, D)

    def project(self, W, x):
        """x [tokens, k] -> [tokens, n], at most 64 rows a call."""
        y = torch.empty(x.shape[0], W.n, device="cuda")
        ws = torch.empty(max(kq.kq_gemv_workspace_bytes(W, min(64, x.shape[0])), 16), dtype=torch.uint8, device="cuda")
        for i in range(0, x.shape[0], 64):
            m = min(64, x.shape[0] - i)
            kq.kq_gemm_small_m(W, x[i: i + m], m, y[i: i + m], ws)
        return y


class Requests:
    """Lengths, block tables and the free list, in device memory."""

    def __init__(self, layer, requests, capacity):
        self.cached = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.table = torch.zeros(requests, -(-capacity // PAGE), dtype=torch.int32, device="cuda")
        self.free = torch.randperm(layer.pages).to(torch.int32).cuda()

    def step(self, layer, x, new):
        """The layer's output for x [tokens, hidden], new[r] tokens of request r; returns (output, queries, attention,
        q_start, kv_len)."""
        r, t, most = len(new), x.shape[0], max(new)
        i = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        q_start, kv_len, positions, slots, used = i(r + 1), i(r), i(t), i(t), i(1)
        fresh = torch.tensor(new, dtype=torch.int32).cuda()
        kq.kq_slot_map(self.cached, fresh, PAGE, self.free, self.table, q_start, kv_len, positions, slots, used)
        q = layer.project(layer.wq, x).view(t, Q_HEADS, D)
        k = layer.project(layer.wk, x).view(t, KV_HEADS, D)
        v = layer.project(layer.wv, x).view(t, KV_HEADS, D)
        kq.kq_kv_append(layer.norm, layer.cache, q, k, v, positions, slots, q)  # queries in place
        out = torch.empty(t, Q_HEADS, D, device="cuda")
        n = kq.kq_attn_workspace_bytes(layer.cache, Q_HEADS, r, t, most)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        kq.kq_attn_paged(layer.cache, q, q_start, kv_len, self.table, out, D ** -0.5, most, ws=ws)
        y = layer.project(layer.wo, out.view(t, Q_HEADS * D))
        self.cached.copy_(kv_len)
        self.free = self.free[int(used.item()):].clone()
        return y, q, out, q_start, kv_len


def attention_fp64(layer, requests, q, q_start, kv_len):
    """The last step's attention from what the cache holds (read back with kq_kv_read), in FP64."""
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for r in range(kv_len.numel()):
        lo, hi, n = int(q_start[r]), int(q_start[r + 1]), int(kv_len[r])
        at = torch.arange(n, device="cuda")
        slots = (requests.table[r][at // PAGE] * PAGE + at % PAGE).to(torch.int32)
        k, v = torch.empty(n, KV_HEADS, D, device="cuda"), torch.empty(n, KV_HEADS, D, device="cuda")
        kq.kq_kv_read(layer.cache, slots, k, v)
        for h in range(Q_HEADS):
            s = (q[lo:hi, h].double() @ k[:, h * KV_HEADS // Q_HEADS].double().T) * D ** -0.5
            hidden = at[None, :] > torch.arange(n - (hi - lo), n, device="cuda")[:, None]
            p = torch.softmax(s.masked_fill(hidden, -float("inf")), -1)
            out[lo:hi, h] = p @ v[:, h * KV_HEADS // Q_HEADS].double()
    return out


def main(requests=4, prompt=37, steps=5, seed=0):
    """Returns the last step's relative error against FP64."""
    capacity = prompt + steps + requests
    layer = Layer(requests, capacity, seed)
    state = Requests(layer, requests, capacity)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for step in range(steps + 1):
        new = [prompt + i for i in range(requests)] if step == 0 else [1] * requests
        x = torch.randn(sum(new), HIDDEN, generator=gen, device="cuda")
        y, q, out, q_start, kv_len = state.step(layer, x, new)
    if kq.kq_device_status() != kq.KQ_OK:
        raise RuntimeError("device status not ok: " + kq.lib().kq_last_error().decode())
    want = attention_fp64(layer, state, q, q_start, kv_len)
    error = float((out.double() - want).norm() / want.norm())
    print(f"{requests} requests, {int(kv_len.sum())} tokens cached, output {tuple(y.shape)}: attention within {error:.2e} of FP64")
    return error


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--prompt", type=int, default=37)
    p.add_argument("--steps", type=int, default=5)
    a = p.parse_args()
    sys.exit(0 if main(a.requests, a.prompt, a.steps) < 1e-5 else 1)
