"""One transformer layer of a serving loop on the library: prompts, then decode steps, then parallel samples.

The layer is Gemma-3-4B shaped (hidden 2560, 8 query and 4 kv heads of 256, FFN 10240) with random block-quantized weights:
QKV projection of the RMS-normed input -> rotary positions -> KV cache append -> attention -> O projection -> FFN.  Prompts run
through lq_gemm and the batched attention, single tokens through the matvecs; the cache's pages come from lq_kv_reserve, and
lq_kv_fork lets two samples continue one prompt.  The decode step is captured into a CUDA graph.

    python examples/decode_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_weight_super_gb300 as lq  # noqa: E402
import synth  # noqa: E402

HIDDEN, N_Q, N_KV, D, FFN, PAGE, EPS = 2560, 8, 4, 256, 10240, 64, 1e-6
NQ, NKV = N_Q * D, N_KV * D


class Layer:
    """Weights, cache and workspaces of one layer, and its step."""

    def __init__(self, seed=0, n_pages=64, rows=4, max_pages=8, max_tokens=256):
        g = synth.rng(seed)
        up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.wq, self.wk, self.wv = up(synth.q4k(g, NQ, HIDDEN)), up(synth.q4k(g, NKV, HIDDEN)), up(synth.q6k(g, NKV, HIDDEN))
        self.wo, self.wd = up(synth.q4k(g, HIDDEN, NQ)), up(synth.q6k(g, HIDDEN, FFN))
        gate, upm = up(synth.q4k(g, FFN, HIDDEN)), up(synth.q4k(g, FFN, HIDDEN))
        self.wgu = torch.empty(2 * gate.numel(), dtype=torch.uint8, device="cuda")
        lq.lq_pack_gate_up(lq.LQ_Q4_K, gate, upm, FFN, HIDDEN, self.wgu)
        self.norm = torch.ones(HIDDEN, device="cuda")
        self.freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        k, v = (torch.zeros(n_pages * NKV * PAGE, dtype=torch.int8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros(n_pages, N_KV, device="cuda") for _ in range(2))
        self.cache = lq.LqKv8(k, v, ks, vs, n_pages, N_KV, PAGE, D)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.n_pages, self.rows, self.max_pages = n_pages, rows, max_pages
        self.table, self.ref, self.lens, self.info = i32(rows, max_pages) - 1, i32(n_pages), i32(rows), i32(2)
        f32 = lambda n: torch.empty(max_tokens, n, device="cuda")  # noqa: E731
        self.xn, self.q, self.k, self.v, self.att, self.o, self.h, self.y = (f32(n) for n in (HIDDEN, NQ, NKV, NKV, NQ, HIDDEN, FFN, HIDDEN))
        nb = max(lq.lq_kv8_attn_workspace_bytes(N_Q, N_KV, D, rows, max_tokens),
                 *(lq.lq_gemm_workspace_bytes(max_tokens, r, c) for r, c in ((NQ, HIDDEN), (HIDDEN, NQ), (2 * FFN, HIDDEN), (HIDDEN, FFN))))
        self.ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def reserve(self, start, cu, nseq):
        lq.lq_kv_reserve(self.table, self.max_pages, self.ref, self.n_pages, PAGE, start, cu, nseq, self.info)

    def step(self, x, ntok, start, cu, nseq, pos):
        """x [ntok][HIDDEN] of nseq sequences -> the layer's output rows (without the residual sums)."""
        nb, ws = self.ws.numel(), self.ws
        if ntok <= 8:
            lq.lq_qkv_mixed_rmsnorm(lq.LQ_Q4_K, self.wq, NQ, lq.LQ_Q4_K, self.wk, NKV, lq.LQ_Q6_K, self.wv, NKV, HIDDEN, x, self.norm, EPS, self.xn,
                                    self.q, self.k, self.v, ntok)
        else:
            lq.lq_rmsnorm(x, self.norm, EPS, self.xn, ntok, HIDDEN)
            for f, w, n, out in ((lq.LQ_Q4_K, self.wq, NQ, self.q), (lq.LQ_Q4_K, self.wk, NKV, self.k), (lq.LQ_Q6_K, self.wv, NKV, self.v)):
                lq.lq_gemm(f, w, n, HIDDEN, self.xn, out, ntok, ws, nb)
        lq.lq_rope(self.q, N_Q, NQ, self.q, NQ, self.k, N_KV, NKV, self.k, NKV, D, D, lq.LQ_ROPE_HALF, pos, 1, None, self.freq, ntok)
        lq.lq_kv8_append(self.cache, self.table, self.max_pages, start, cu, nseq, self.k, NKV, self.v, NKV, ntok)
        lq.lq_kv8_attn(self.cache, self.table, self.max_pages, start, cu, nseq, self.q, N_Q, NQ, ntok, D ** -0.5, 0.0, 0, None, None, self.att, NQ, ws, nb)
        lq.lq_gemm(lq.LQ_Q4_K, self.wo, HIDDEN, NQ, self.att, self.o, ntok, ws, nb)
        if ntok <= 8:
            lq.lq_ffn_gate_up_act_rmsnorm(lq.LQ_Q4_K, self.wgu, FFN, HIDDEN, self.o, self.norm, EPS, self.xn, self.h, ntok, lq.LQ_ACT_GEGLU_TANH)
        else:
            lq.lq_rmsnorm(self.o, self.norm, EPS, self.xn, ntok, HIDDEN)
            lq.lq_gemm_gate_up_act(lq.LQ_Q4_K, self.wgu, FFN, HIDDEN, self.xn, self.h, ntok, lq.LQ_ACT_GEGLU_TANH, ws, nb)
        lq.lq_gemm(lq.LQ_Q6_K, self.wd, HIDDEN, FFN, self.h, self.y, ntok, ws, nb)
        return self.y[:ntok]


def main(steps=4):
    layer = Layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    # two prompts of 100 and 37 tokens
    ns = [100, 37]
    x = torch.randn(sum(ns), HIDDEN, device="cuda", generator=g)
    cu, zero = i32(0, ns[0], sum(ns)), i32(0, 0)
    layer.reserve(zero, cu, 2)
    y = layer.step(x, sum(ns), zero, cu, 2, i32(*range(ns[0]), *range(ns[1])))
    layer.lens[:2] = i32(*ns)
    print("prompts:", tuple(y.shape), "rms %.3g" % y.square().mean().sqrt().item())
    # two more samples of the first prompt
    src, dst = (torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(2))
    lq.lq_kv_fork(layer.table, layer.rows, layer.max_pages, layer.ref, layer.n_pages, PAGE, layer.lens, i32(0, 0), i32(2, 3), 2, src, dst, layer.info)
    lq.lq_kv8_copy_pages([layer.cache], src, dst, 2)
    # decode steps of all four rows, as one graph: the lengths, positions and tokens are updated in place
    start, pos, x1 = layer.lens.clone(), layer.lens.clone()[None], torch.empty(4, HIDDEN, device="cuda")

    def decode():
        layer.reserve(start, None, 4)
        return layer.step(x1, 4, start, None, 4, pos)

    x1.normal_(generator=g)
    decode()                                       # (every kernel has run once before it is captured)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = decode()
    outs = []
    for i in range(steps):
        x1.normal_(generator=g)
        x1[3] = x1[2]                              # the samples 2 and 3 get the same tokens
        graph.replay()
        outs.append(out.clone())
        start += 1
        pos += 1
    layer.lens.copy_(start)
    print("decode steps:", steps, "lengths", layer.lens.tolist(), "pages in use", int((layer.ref > 0).sum()))
    # the samples end; the pool is closed up
    lq.lq_kv_release(layer.table, layer.rows, layer.max_pages, layer.ref, layer.n_pages, layer.lens, i32(2, 1), 2)
    mp = torch.empty(layer.n_pages, dtype=torch.int32, device="cuda")
    ms, md = (torch.empty(layer.n_pages // 2, dtype=torch.int32, device="cuda") for _ in range(2))
    lq.lq_kv_compact(layer.table, layer.rows, layer.max_pages, layer.ref, layer.n_pages, mp, ms, md, layer.info)
    lq.lq_kv8_copy_pages([layer.cache], ms, md, layer.n_pages // 2, layer.info)
    print("after release and compaction: pages in use", int((layer.ref > 0).sum()), "moved", layer.info[0].item())
    rc, bits = lq.lq_device_status()
    assert rc == 0 and bits == 0, (rc, bits)
    return y, outs, layer


if __name__ == "__main__":
    main()
