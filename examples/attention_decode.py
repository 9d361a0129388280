"""One attention block of a quantized model, token after token, on qmm.

    python examples/attention_decode.py [--tokens 64] [--cache q8_0] [--weights q4_0]
        [--prompt 100] [--dim 1024] [--heads 16] [--kv-heads 4]

Weights stay quantized, activations are f32.  A step is four launches (five
where the attention is split over the cache's length):

    q, k, v = W_qkv x           qmm_quantize_matvec_*   quantize x and multiply
    rotate, write the cache     qmm_rope_kv_write_*     q rotated, k rotated and quantized, v quantized
    attention over the cache    qmm_attn_decode_*
    y = W_o (attention)         qmm_quantize_matvec_*

The prompt's cache rows are written in one call, the steps run as one captured
graph, and every output is checked against the formulas in 64 bits, from the
rows that the cache really holds (read back with qmm_kv_read_*).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matmul_quantize_q8_amd as qmm  # noqa: E402


class AttentionBlock:
    """The block's weights, its cache, and the buffers of a step for one sequence."""

    def __init__(self, dim=1024, q_heads=16, kv_heads=4, weights="q4_0", cache="q8_0", page=32, max_len=512, seed=0):
        self.hq, self.h, self.d, self.max_len, self.page = q_heads, kv_heads, dim // q_heads, max_len, page
        self.weights, self.cache_fmt = weights, cache
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rows = (q_heads + 2 * kv_heads) * self.d
        self.w_qkv, self.dense_qkv = self._quantized(rows, dim, gen)
        self.w_out, self.dense_out = self._quantized(dim, dim, gen)
        freqs, mscale = qmm.qmm_rope_freqs(self.d, 10000.0)
        self.plan = qmm.RopePlan(freqs.cuda(), "half", mscale)
        n_pages = -(-max_len // page)
        self.cache = qmm.KVCache.empty(cache, n_pages, page, kv_heads, self.d)
        self.pages = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32).view(1, -1)
        self.workspace = qmm.attn_workspace(1, q_heads, kv_heads, self.d, max_len)
        # what a step reads and writes
        self.x = torch.zeros(dim, device="cuda")
        self.qkv = torch.zeros(1, q_heads + 2 * kv_heads, self.d, device="cuda")
        self.q = torch.zeros(1, q_heads, self.d, device="cuda")
        self.attended = torch.zeros(1, q_heads, self.d, device="cuda")
        self.y = torch.zeros(dim, device="cuda")
        self.position = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.slot = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.length = torch.zeros(1, dtype=torch.int32, device="cuda")

    def _quantized(self, n, k, gen):
        w = torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5
        wq = torch.empty(n * qmm.row_bytes(self.weights, k), dtype=torch.uint8, device="cuda")
        qmm.QUANTIZE_W[self.weights](w, wq, n, k)
        ids, dense = torch.arange(n, dtype=torch.int32, device="cuda"), torch.empty_like(w)
        qmm.GET_ROWS[self.weights](wq, ids, dense, n, n, k)
        return wq, dense

    def slots(self, positions):
        """Cache slots of positions of the sequence."""
        positions = positions.long()
        return self.pages[0, positions // self.page].long() * self.page + positions % self.page

    def prompt(self, x):
        """Write the cache rows of a prompt's activations [tokens][dim]; returns its rotated queries."""
        t, hq, h = x.shape[0], self.hq, self.h
        xq = torch.empty(t * qmm.row_bytes(qmm.ACT_FORMAT[self.weights], x.shape[1]), dtype=torch.uint8, device="cuda")
        qkv = torch.empty(t, hq + 2 * h, self.d, device="cuda")
        qmm.QUANTIZE_X[self.weights](x, xq, t, x.shape[1])
        qmm.MATMUL[self.weights](self.w_qkv, xq, qkv, t, qkv[0].numel(), x.shape[1])
        positions = torch.arange(t, dtype=torch.int32, device="cuda")
        q = qkv[:, :hq]
        qmm.ROPE_KV_WRITE[self.cache_fmt](q, q, qkv[:, hq:hq + h], qkv[:, hq + h:], self.cache, self.slots(positions),
                                          positions, self.plan)
        return q

    def at(self, x, position):
        """Set the step's inputs."""
        self.x.copy_(x)
        self.position.fill_(position)
        self.length.fill_(position + 1)
        self.slot.copy_(self.slots(self.position))

    def step(self):
        """One token: y from x, its rows written to the cache."""
        hq, h, dim = self.hq, self.h, self.x.numel()
        fused = qmm.QUANTIZE_MATVEC[self.weights]
        fused(self.w_qkv, self.x, None, self.qkv, self.qkv.numel(), dim)
        qmm.ROPE_KV_WRITE[self.cache_fmt](self.qkv[:, :hq], self.q, self.qkv[:, hq:hq + h], self.qkv[:, hq + h:],
                                          self.cache, self.slot, self.position, self.plan)
        qmm.ATTN_DECODE[self.cache_fmt](self.q, self.attended, self.cache, self.pages, self.length, self.max_len,
                                        self.workspace)
        fused(self.w_out, self.attended, None, self.y, dim, dim)

    def expected(self, position):
        """(attention, output) of the last step in 64 bits: from its rotated queries and the cache's rows,
        and from the attention's result and the decoded weights."""
        slots = self.slots(torch.arange(position + 1, device="cuda"))
        k = torch.empty(position + 1, self.h, self.d, device="cuda")
        v = torch.empty_like(k)
        qmm.KV_READ[self.cache_fmt](self.cache, slots, k, v)
        group = self.hq // self.h
        k, v = (x.double().repeat_interleave(group, 1).transpose(0, 1).contiguous() for x in (k, v))
        s = (k * self.q[0].double()[:, None]).sum(-1) * self.d ** -0.5
        a = (torch.softmax(s, -1)[..., None] * v).sum(1)
        return a, self.dense_out.double() @ self.attended.double().flatten()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=4)
    ap.add_argument("--cache", choices=qmm.KV_FORMATS, default="q8_0")
    ap.add_argument("--weights", choices=qmm.FUSED_FORMATS, default="q4_0")
    a = ap.parse_args()
    block = AttentionBlock(a.dim, a.heads, a.kv_heads, a.weights, a.cache, max_len=a.prompt + a.tokens)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dim = block.x.numel()
    block.prompt(torch.randn(a.prompt, dim, generator=gen, device="cuda"))
    xs = torch.randn(a.tokens, dim, generator=gen, device="cuda")

    block.at(xs[0], a.prompt)
    block.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step()
    worst_attn = worst_out = 0.0
    for i in range(a.tokens):
        block.at(xs[i], a.prompt + i)
        graph.replay()
        want, out = block.expected(a.prompt + i)
        worst_attn = max(worst_attn, float((block.attended[0] - want).abs().max() / want.abs().max()))
        worst_out = max(worst_out, float((block.y - out).norm() / out.norm()))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(200):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens after a prompt of {a.prompt}, {a.weights} weights, {a.cache} cache: "
          f"{begin.elapsed_time(end) * 5:.1f} us a step")
    print(f"attention: worst error {worst_attn:.2e} of the largest value; output projection (quantized activations): "
          f"{worst_out:.2e} in norm")
    # f32 rounding of the attention; 8-bit activations in the output product
    return 0 if worst_attn < 1e-5 and worst_out < 2e-2 else 1


if __name__ == "__main__":
    sys.exit(main())
