"""The operators between the QKV and the O projection, as a serving program calls them: rotary positions, the
8-bit paged KV cache (append, attention) and the cache's pages (fork, compact, copy).

own = False: run() computes them in elementary torch operations; own = True: through the library's entry points.
"""
import random

import torch

own = False
DEV = "cuda"

# ------------------------------------------------------------------------------------------------ cases
# Head layouts: 32 query / 8 kv heads of 128 (the Llama-3-8B shape of this repository's FFN workloads), 8 / 4 of 256 (the
# Gemma-3-4B layer, Q 2048 and K/V 1024 rows), and generic ones of 64.


def listed():
    return [
        # one token of one sequence: the smallest call, latency only
        dict(name="rope 1 token", op="rope", ntok=1, n_q=32, n_kv=8, d=128, rot=128, axes=1, pairing="half", far=131072),
        # an image's tokens with time, height and width positions, in the middle of a long context
        dict(name="rope 3 axes", op="rope", ntok=8192, n_q=8, n_kv=4, d=256, rot=256, axes=3, pairing="half", far=1000000),
        # one new token for each of 64 running sequences
        dict(name="append decode", op="append", nseq=64, n=1, start=1000, n_kv=8, d=128, page=64),
        # prompts of several sequences, one of them behind a cached prefix that ends inside a page
        dict(name="append prompts", op="append", nseq=5, n=4099, start=37, n_kv=4, d=256, page=64),
        # a single chat: latency of one token
        dict(name="attn decode 1", op="attn", nseq=1, n=1, len=4096, n_q=8, n_kv=4, d=256, page=64, window=0, cap=0.0, alibi=False, prefix=0),
        # a serving batch with ragged lengths, small pages
        dict(name="attn decode batch", op="attn", nseq=32, n=1, len=8192, n_q=32, n_kv=8, d=128, page=16, window=0, cap=0.0, alibi=False, prefix=0),
        # two very long documents
        dict(name="attn decode long", op="attn", nseq=2, n=1, len=131072, n_q=32, n_kv=8, d=128, page=128, window=0, cap=0.0, alibi=False, prefix=0),
        # a local layer: a window, kept first tokens, capped scores; a few tokens a step (a checked draft)
        dict(name="attn decode window", op="attn", nseq=48, n=3, len=6000, n_q=16, n_kv=16, d=64, page=32, window=1024, cap=50.0, alibi=False, prefix=16),
        # one long prompt
        dict(name="attn prompt", op="attn", nseq=1, n=4096, len=4096, n_q=32, n_kv=8, d=128, page=64, window=0, cap=0.0, alibi=False, prefix=0),
        # ragged chunks behind cached tokens: a distance bias, an image prefix seen in both directions
        dict(name="attn prompt bias", op="attn", nseq=6, n=777, len=2500, n_q=8, n_kv=4, d=256, page=64, window=0, cap=30.0, alibi=True, prefix=300),
        # parallel samples: children share the parents' full pages and get copies of their last ones
        dict(name="pages fork", op="fork", parents=8, children=64, len=5000, n_kv=8, d=128, page=64, layers=4, pool=8192),
        # a fragmented pool closed up
        dict(name="pages compact", op="compact", rows=96, len=4000, n_kv=8, d=128, page=64, layers=2, pool=8192, keep=0.4),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    n_q, n_kv, d = rng.choice([(32, 8, 128), (8, 4, 256), (16, 16, 64), (24, 2, 64), (40, 8, 128), (5, 5, 128), (12, 4, 256)])
    page = rng.choice([16, 32, 64, 128])
    op = rng.choice(["rope", "append", "append", "attn", "attn", "attn", "attn", "fork", "compact"])
    if op == "rope":
        rot = rng.choice([d, d // 2, d - 16])
        return dict(op=op, ntok=_log(rng, 1, 8192 * 256 // max(d * (n_q + n_kv) // 12, 256)), n_q=n_q, n_kv=n_kv, d=d, rot=rot, axes=rng.choice([1, 2, 3, 4]),
                    pairing=rng.choice(["half", "adjacent"]), far=_log(rng, 100, 1000000))
    if op == "append":
        nseq = _log(rng, 1, 128)
        return dict(op=op, nseq=nseq, n=_log(rng, 1, max(2, 16 * 1024 * 1024 // (nseq * n_kv * d))), start=rng.choice([0, _log(rng, 1, 3000)]), n_kv=n_kv, d=d, page=page)
    if op == "fork":
        parents = _log(rng, 1, 16)
        pool = (1 << 28) // (n_kv * d * page * 4)
        return dict(op=op, parents=parents, children=parents * _log(rng, 1, 8), len=_log(rng, 5, min(5000, pool * page // (2 * parents))), n_kv=n_kv, d=d, page=page,
                    layers=rng.choice([1, 2, 3]), pool=pool)
    if op == "compact":
        pool = (1 << 28) // (n_kv * d * page * 4)
        rows = _log(rng, 4, 96)
        return dict(op=op, rows=rows, len=max(1, int(pool * page * rng.uniform(0.2, 0.9)) // rows), n_kv=n_kv, d=d, page=page, layers=rng.choice([1, 2]), pool=pool,
                    keep=round(rng.uniform(0.1, 0.9), 3))
    c = dict(op=op, n_q=n_q, n_kv=n_kv, d=d, page=page, window=rng.choice([0, 0, _log(rng, 16, 4096)]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
             alibi=rng.choice([False, False, True]), prefix=rng.choice([0, 0, _log(rng, 1, 500)]))
    if rng.random() < 0.6:
        nseq = _log(rng, 1, 64)
        n = rng.choice([1, 1, 1, 2, 5])
        return dict(c, nseq=nseq, n=n, len=_log(rng, n, max(n + 1, min(65536, (1 << 27) // (nseq * n_kv * d)))))
    n = _log(rng, 9, 2500)
    nseq = max(1, min(8, _log(rng, 1, 8), (1 << 28) // (n * n * n_q)))
    return dict(c, nseq=nseq, n=n, len=min(n + rng.choice([0, _log(rng, 1, 2000)]), max(n, (1 << 29) // (n * n_q * nseq))))


def _ns(c):
    """New tokens of each sequence: the first has them all, the others fewer unless it is a decode step."""
    r = random.Random(c["nseq"] * 1009 + c["n"])
    return [c["n"] if i == 0 or c["n"] <= 8 else r.randint(max(1, c["n"] // 3), c["n"]) for i in range(c["nseq"])]


def _starts(c):
    """Cached tokens of each sequence before the step."""
    ns = _ns(c)
    r = random.Random(c["nseq"] * 2003 + c.get("len", c.get("start", 0)))
    if c["op"] == "append":
        return [c["start"] if i == 0 else r.randint(0, c["start"]) for i in range(c["nseq"])]
    most = c["len"] - c["n"]
    return [most if i == 0 else r.randint(most // 2, most) for i in range(c["nseq"])]


def _lens(c, rows):
    r = random.Random(rows * 31 + c["len"])
    return [c["len"] if i == 0 else r.randint(max(1, c["len"] // 2), c["len"]) for i in range(rows)]


# ------------------------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pool(g, n_pages, n_kv, page, d):
    """A pool of pages that holds values near N(0, 1): codes near 32 N(0, 1), a scale for each page and head."""
    k, v = (torch.empty(n_pages, n_kv, *s, dtype=torch.int8, device=DEV) for s in ((page, d), (d, page)))
    for t in (k, v):
        flat = t.view(-1)
        for i in range(0, flat.numel(), 1 << 27):
            part = flat[i:i + (1 << 27)]
            part.copy_((torch.randn(part.numel(), device=DEV, generator=g) * 32).round_().clamp_(-127, 127))
    ks, vs = (torch.exp(torch.randn(n_pages, n_kv, device=DEV, generator=g) * 0.3) / 32 for _ in range(2))
    return dict(k=k, v=v, ks=ks, vs=vs)


def _table(g, counts, n_pages, width):
    perm = torch.randperm(n_pages, device=DEV, generator=g).to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, perm[:at].long()


def _freq(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)


def _handle(p, n_pages, c):
    """The library's description of a pool, which a program keeps."""
    if not own:
        return None
    import block_quantized_weight_super_gb300 as lq
    return lq.LqKv8(p["k"], p["v"], p["ks"], p["vs"], n_pages, c["n_kv"], c["page"], c["d"])


def _workspace(c, ntok):
    """The library's scratch memory, one for all layers of a program."""
    if not own:
        return None
    import block_quantized_weight_super_gb300 as lq
    return torch.empty(lq.lq_kv8_attn_workspace_bytes(c["n_q"], c["n_kv"], c["d"], c["nseq"], ntok), dtype=torch.uint8, device=DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    randn = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    s = dict(c=c, op=c["op"])
    if c["op"] == "rope":
        # q and k as the QKV projection leaves them; positions of each axis; a pair's axis; a pair's frequency
        s |= dict(q=randn(c["ntok"], c["n_q"] * c["d"]), k=randn(c["ntok"], c["n_kv"] * c["d"]), freq=_freq(c["rot"]),
                  pos=torch.randint(0, c["far"], (c["axes"], c["ntok"]), device=DEV, generator=g).to(torch.int32),
                  axis=(torch.arange(c["rot"] // 2, device=DEV) * c["axes"] // (c["rot"] // 2)).to(torch.uint8))
        s |= dict(q_out=torch.empty_like(s["q"]), k_out=torch.empty_like(s["k"]))
        return s
    P = c["page"]
    if c["op"] in ("append", "attn"):
        ns, starts = _ns(c), _starts(c)
        counts = [-(-(a + n) // P) for a, n in zip(starts, ns)]
        n_pages = sum(counts) + 3
        cu = [0]
        for n in ns:
            cu.append(cu[-1] + n)
        p = _pool(g, n_pages, c["n_kv"], P, c["d"])
        table, _ = _table(g, counts, n_pages, max(counts))
        s |= p | dict(table=table, width=max(counts), start=_ints(starts), cu=_ints(cu), ntok=cu[-1], n_max=max(ns), l_max=max(a + n for a, n in zip(starts, ns)),
                      cache=_handle(p, n_pages, c))
        if c["op"] == "append":
            # rows of unequal size: some grow the scale of the page that they end up in, some do not
            for name in ("new_k", "new_v"):
                s[name] = randn(cu[-1], c["n_kv"] * c["d"]) * torch.exp(0.5 * randn(cu[-1], 1))
            return s
        s |= dict(q=2 * randn(cu[-1], c["n_q"] * c["d"]), out=torch.empty(cu[-1], c["n_q"] * c["d"], device=DEV), scale=c["d"] ** -0.5,
                  prefix=_ints([c["prefix"]] * c["nseq"]) if c["prefix"] else None,
                  slopes=2.0 ** (-8.0 * torch.arange(1, c["n_q"] + 1, device=DEV, dtype=torch.float32) / c["n_q"]) if c["alibi"] else None, ws=_workspace(c, cu[-1]))
        return s
    layers = [_pool(g, c["pool"], c["n_kv"], P, c["d"]) for _ in range(c["layers"])]
    s |= dict(layers=layers, caches=[_handle(p, c["pool"], c) for p in layers])
    if c["op"] == "fork":
        lens = _lens(c, c["parents"])
        counts = [-(-n // P) for n in lens]
        table, used = _table(g, counts + [0] * c["children"], c["pool"], max(counts))
        s |= dict(lens=_ints(lens + [0] * c["children"]), parent=_ints([i % c["parents"] for i in range(c["children"])]),
                  child=_ints([c["parents"] + i for i in range(c["children"])]), src=torch.empty(c["children"], dtype=torch.int32, device=DEV),
                  dst=torch.empty(c["children"], dtype=torch.int32, device=DEV))
    else:
        # rows that end give their pages back: what is left lies all over the pool
        lens = _lens(c, c["rows"])
        counts = [-(-n // P) for n in lens]
        r = random.Random(c["rows"])
        counts = [n if i == 0 or r.random() < c["keep"] else 0 for i, n in enumerate(counts)]
        while sum(counts) > c["pool"]:
            counts = [n - 1 if n > 1 else n for n in counts]
        table, used = _table(g, counts, c["pool"], max(counts))
        s |= dict(src=torch.empty(c["pool"] // 2, dtype=torch.int32, device=DEV), dst=torch.empty(c["pool"] // 2, dtype=torch.int32, device=DEV),
                  map=torch.empty(c["pool"], dtype=torch.int32, device=DEV), table0=table.clone())
    ref = torch.zeros(c["pool"], dtype=torch.int32, device=DEV)
    ref[used] = 1
    s |= dict(table=table, ref=ref, ref0=ref.clone(), info=torch.zeros(2, dtype=torch.int32, device=DEV))
    return s


# ------------------------------------------------------------------------------------------------ one pass


def run(state):
    return globals()["_" + state["op"]](state) if not own else globals()["_own_" + state["op"]](state)


def _rope(s):
    c = s["c"]
    n = c["rot"] // 2
    at = s["pos"].double()[s["axis"].long()] * s["freq"][:, None]  # angles in 64 bits: positions are far
    cos, sin = at.cos().float().T[:, None], at.sin().float().T[:, None]

    def turn(x):
        x = x.view(c["ntok"], -1, c["d"])
        y = x.clone()
        a, b = (slice(0, n), slice(n, 2 * n)) if c["pairing"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        return y.view(c["ntok"], -1)

    return turn(s["q"]), turn(s["k"])


def _own_rope(s):
    import block_quantized_weight_super_gb300 as lq
    c = s["c"]
    nq, nk = c["n_q"] * c["d"], c["n_kv"] * c["d"]
    lq.lq_rope(s["q"], c["n_q"], nq, s["q_out"], nq, s["k"], c["n_kv"], nk, s["k_out"], nk, c["d"], c["rot"],
               lq.LQ_ROPE_HALF if c["pairing"] == "half" else lq.LQ_ROPE_ADJACENT, s["pos"], c["axes"], s["axis"], s["freq"], c["ntok"])
    return s["q_out"], s["k_out"]


def _append(s):
    """Each touched page in turn of its sequence (those behind a sequence's last one do the last one again), all at once."""
    c, P = s["c"], s["c"]["page"]
    start, cu = s["start"].long(), s["cu"].long()
    n = cu[1:] - cu[:-1]
    first, last = start // P, (start + n - 1) // P
    j = torch.minimum(first[:, None] + torch.arange((s["n_max"] - 1) // P + 2, device=DEV), last[:, None])
    page = s["table"].long().gather(1, j)
    at = j[..., None] * P + torch.arange(P, device=DEV)  # positions [sequence, page, slot]
    new = ((at >= start[:, None, None]) & (at < (start + n)[:, None, None]))[..., None, None]
    old = (at < start[:, None, None])[..., None, None]
    row = (cu[:-1, None, None] + at - start[:, None, None]).clamp(0, s["ntok"] - 1)
    for codes, scales, x, turned in ((s["k"], s["ks"], s["new_k"], False), (s["v"], s["vs"], s["new_v"], True)):
        x = x.view(s["ntok"], c["n_kv"], c["d"])[row]  # [sequence, page, slot, head, dim]
        amax = torch.where(new, x.abs(), 0.0).amax((2, 4))
        was = torch.where(old.any(2)[..., 0], scales[page], 0.0)
        scale = torch.maximum(was, amax / 127.0)
        had = codes[page]
        had = had.permute(0, 1, 4, 2, 3) if turned else had.permute(0, 1, 3, 2, 4)
        again = torch.where(old, had.float() * was[:, :, None, :, None], x)
        by = scale[:, :, None, :, None]
        q = torch.where(by > 0, (again.double() / by.double()).round().clamp(-127, 127), 0.0).to(torch.int8)  # in 64 bits: values next to a border
        q = torch.where(new | (old & (by > was[:, :, None, :, None])), q, had)
        codes[page] = q.permute(0, 1, 3, 4, 2) if turned else q.permute(0, 1, 3, 2, 4)
        scales[page] = scale
    return s["k"], s["v"], s["ks"], s["vs"]  # the pool itself: whole codes, and the scales that make them values


def _own_append(s):
    import block_quantized_weight_super_gb300 as lq
    c = s["c"]
    ld = c["n_kv"] * c["d"]
    lq.lq_kv8_append(s["cache"], s["table"], s["width"], s["start"], s["cu"], c["nseq"], s["new_k"], ld, s["new_v"], ld, s["ntok"])
    return s["k"], s["v"], s["ks"], s["vs"]


def _attn(s):
    c, P = s["c"], s["c"]["page"]
    start, cu = s["start"].long(), s["cu"].long()
    n, nseq, n_max, l_max, kv, d = cu[1:] - cu[:-1], c["nseq"], s["n_max"], s["l_max"], c["n_kv"], c["d"]
    page = s["table"].long().clamp(min=0)
    k = (s["k"][page].float() * s["ks"][page][..., None, None]).permute(0, 2, 1, 3, 4).reshape(nseq, kv, -1, d)[:, :, :l_max]
    v = (s["v"][page].float() * s["vs"][page][..., None, None]).permute(0, 2, 1, 4, 3).reshape(nseq, kv, -1, d)[:, :, :l_max]
    i = torch.arange(n_max, device=DEV)
    row = (cu[:-1, None] + i).clamp(max=s["ntok"] - 1)
    g = c["n_q"] // kv
    q = s["q"].view(s["ntok"], kv, g, d)[row].permute(0, 2, 3, 1, 4).reshape(nseq, kv, g * n_max, d)
    t = (q @ k.transpose(-1, -2)).view(nseq, kv, g, n_max, l_max) * s["scale"]
    if c["cap"]:
        t = c["cap"] * torch.tanh(t / c["cap"])
    p, j = (start[:, None] + i)[..., None], torch.arange(l_max, device=DEV)
    if c["alibi"]:
        t = t - s["slopes"].view(kv, g)[None, :, :, None, None] * (p - j).abs().float()[:, None, None]
    sees = j <= p
    if c["window"]:
        sees = sees & (p - j < c["window"])
    if c["prefix"]:
        sees = sees | (j < s["prefix"].long()[:, None, None])
    sees = sees & (j < (start + n)[:, None, None])
    t = torch.where(sees[:, None, None], t, float("-inf"))
    t = torch.exp(t - t.amax(-1, keepdim=True))
    t = t / t.sum(-1, keepdim=True)
    o = (t.view(nseq, kv, g * n_max, l_max) @ v).view(nseq, kv, g, n_max, d).permute(0, 3, 1, 2, 4).reshape(nseq * n_max, kv * g * d)
    of = torch.repeat_interleave(torch.arange(nseq, device=DEV), n, output_size=s["ntok"])
    return o[of * n_max + torch.arange(s["ntok"], device=DEV) - cu[of]]


def _own_attn(s):
    import block_quantized_weight_super_gb300 as lq
    c = s["c"]
    ld = c["n_q"] * c["d"]
    lq.lq_kv8_attn(s["cache"], s["table"], s["width"], s["start"], s["cu"], c["nseq"], s["q"], c["n_q"], ld, s["ntok"], s["scale"], c["cap"], c["window"], s["prefix"],
                   s["slopes"], s["out"], ld, s["ws"], s["ws"].numel())
    return s["out"]


def _fork(s):
    """The children of the last pass end; new ones are forked from the parents."""
    c, P, table, ref, lens = s["c"], s["c"]["page"], s["table"], s["ref"], s["lens"]
    parent, child = s["parent"].long(), s["child"].long()
    held = table[child]
    ref.index_add_(0, held.clamp(min=0).long().view(-1), -(held >= 0).int().view(-1))
    n = lens[parent]
    full, tail = n // P, n % P > 0
    rank = tail.long().cumsum(0) - 1
    free = torch.sort((ref > 0).int(), stable=True).indices  # free pages first, the lowest first
    dst = torch.where(tail, free[rank.clamp(min=0)].int(), -1)
    rows, j = table[parent], torch.arange(table.shape[1], device=DEV, dtype=torch.int32)
    src = torch.where(tail, rows.gather(1, full.clamp(max=table.shape[1] - 1).long()[:, None])[:, 0], -1)
    shared = j < full[:, None]
    table[child] = torch.where(shared, rows, torch.where((j == full[:, None]) & tail[:, None], dst[:, None], -1))
    lens[child] = n
    ref.index_add_(0, rows.clamp(min=0).long().view(-1), shared.int().view(-1))
    ref.index_add_(0, dst.clamp(min=0).long(), tail.int())
    keep = table[parent[0], 0]  # a child without a tail: a page that stays, onto itself
    a, b = torch.where(tail, src, keep).long(), torch.where(tail, dst, keep).long()
    for p in s["layers"]:
        for name in ("k", "v", "ks", "vs"):
            p[name][b] = p[name][a]
    return [table, ref, lens, src, dst] + [p[name] for p in s["layers"] for name in ("k", "v", "ks", "vs")]


def _own_fork(s):
    import block_quantized_weight_super_gb300 as lq
    c, w = s["c"], s["table"].shape[1]
    rows = s["table"].shape[0]
    lq.lq_kv_release(s["table"], rows, w, s["ref"], c["pool"], s["lens"], s["child"], c["children"])
    lq.lq_kv_fork(s["table"], rows, w, s["ref"], c["pool"], c["page"], s["lens"], s["parent"], s["child"], c["children"], s["src"], s["dst"], s["info"])
    lq.lq_kv8_copy_pages(s["caches"], s["src"], s["dst"], c["children"], None)
    return [s["table"], s["ref"], s["lens"], s["src"], s["dst"]] + [p[name] for p in s["layers"] for name in ("k", "v", "ks", "vs")]


def _compact(s):
    """The same fragmented table each time: its pages move to the front of the pool."""
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    c, table, ref = s["c"], s["table"], s["ref"]
    used = ref > 0
    n, at = used.sum(), torch.arange(c["pool"], device=DEV)
    high, low = used & (at >= n), ~used & (at < n)
    to = torch.full((c["pool"] + 1,), -1, dtype=torch.int64, device=DEV)  # the page of each rank, a place for the others behind the last
    src, dst = (to.scatter(0, torch.where(m, m.long().cumsum(0) - 1, c["pool"]), at)[:-1] for m in (high, low))
    moved = torch.arange(c["pool"], device=DEV) < high.sum()
    src, dst = torch.where(moved, src, -1), torch.where(moved, dst, -1)
    place = torch.where(used, at, -1)
    place = torch.cat([place, place[:1]]).scatter(0, torch.where(moved, src, c["pool"]), dst)[:-1]
    table.copy_(torch.where(table >= 0, place[table.clamp(min=0).long()].int(), -1))
    count = torch.zeros_like(ref).scatter_add(0, place.clamp(min=0), torch.where(used, ref, 0))
    ref.copy_(count)
    src, dst = src[:c["pool"] // 2], dst[:c["pool"] // 2]  # at most half of the pool moves
    keep = n.clamp(max=c["pool"] - 1)  # ranks that move nothing: a page that does not move, onto itself
    a, b = torch.where(src >= 0, src, keep), torch.where(dst >= 0, dst, keep)
    for p in s["layers"]:
        for name in ("k", "v", "ks", "vs"):
            p[name][b] = p[name][a]
    return [table, ref, place.int(), src.int(), dst.int()] + [p[name] for p in s["layers"] for name in ("k", "v", "ks", "vs")]


def _own_compact(s):
    import block_quantized_weight_super_gb300 as lq
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    c, (rows, w) = s["c"], s["table"].shape
    lq.lq_kv_compact(s["table"], rows, w, s["ref"], c["pool"], s["map"], s["src"], s["dst"], s["info"])
    lq.lq_kv8_copy_pages(s["caches"], s["src"], s["dst"], c["pool"] // 2, s["info"])
    return [s["table"], s["ref"], s["map"], s["src"], s["dst"]] + [p[name] for p in s["layers"] for name in ("k", "v", "ks", "vs")]


# ------------------------------------------------------------------------------------------------ what a pass cannot do without


def _seen(c, start, n):
    """(query, key) pairs that a sequence's rows see, and the keys that any of them sees."""
    pairs, L = 0, start + n
    pre, w = min(c["prefix"], L), c["window"]
    for p in range(start, start + n):
        lo = max(0, p - w + 1) if w else 0
        pairs += p + 1 - lo + (min(pre, lo) + max(0, pre - (p + 1)))
    lo = max(0, start - w + 1) if w else 0
    return pairs, L - lo + min(pre, lo)


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["ntok"] * (c["n_q"] + c["n_kv"])
        return {"bytes": 8 * n * c["d"] + 4 * c["axes"] * c["ntok"], "flops": 3 * n * c["rot"]}
    P = c["page"]
    one = 2 * c["n_kv"] * (P * c["d"] + 4)  # a page of K and V with their scales
    if c["op"] == "append":
        ns, starts = _ns(c), _starts(c)
        touched = sum((a + n - 1) // P - a // P + 1 for a, n in zip(starts, ns))
        return {"bytes": sum(ns) * c["n_kv"] * c["d"] * 2 * 5 + touched * (16 * c["n_kv"] + 4), "flops": sum(ns) * c["n_kv"] * c["d"] * 2 * 3}
    if c["op"] == "attn":
        pairs = keys = pages = 0
        for a, n in zip(_starts(c), _ns(c)):
            x, y = _seen(c, a, n)
            pairs, keys, pages = pairs + x, keys + y, pages + -(-y // P)
        return {"bytes": keys * c["n_kv"] * c["d"] * 2 + pages * (8 * c["n_kv"] + 4) + sum(_ns(c)) * c["n_q"] * c["d"] * 8, "flops": 4 * pairs * c["n_q"] * c["d"]}
    if c["op"] == "fork":
        lens = _lens(c, c["parents"])
        tails = sum(lens[i % c["parents"]] % P > 0 for i in range(c["children"]))
        shared = sum(-(-lens[i % c["parents"]] // P) for i in range(c["children"]))
        return {"bytes": 2 * tails * c["layers"] * one + 12 * shared + 4 * tails, "flops": 0}
    r = random.Random(c["rows"])
    counts = [n if i == 0 or r.random() < c["keep"] else 0 for i, n in enumerate(-(-n // P) for n in _lens(c, c["rows"]))]
    used = min(sum(counts), c["pool"])
    moves = used * (c["pool"] - used) // c["pool"]  # used pages lie anywhere in the pool
    return {"bytes": 2 * moves * c["layers"] * one + 12 * c["pool"] + 8 * used, "flops": 0}


# ------------------------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), (s["pos"].double()[s["axis"].long()] * s["freq"][:, None]).T)[:, None]

        def turn(x):
            x = x.double().view(c["ntok"], -1, c["d"])
            r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
            if c["pairing"] == "half":
                r = torch.view_as_real(torch.complex(*r.chunk(2, -1)) * z).transpose(-1, -2).flatten(-2)
            else:
                r = torch.view_as_real(torch.view_as_complex(r.unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
            return torch.cat([r, rest], -1).view(c["ntok"], -1)

        return turn(s["q"]), turn(s["k"])
    if c["op"] == "append":
        P, cu, start, table = c["page"], s["cu"].tolist(), s["start"].tolist(), s["table"].tolist()
        scales = []
        for x, was in ((s["new_k"], s["ks"]), (s["new_v"], s["vs"])):
            x = x.double().view(s["ntok"], c["n_kv"], c["d"]).abs().amax(-1).cpu() / 127
            was = was.double().cpu()
            for i in range(c["nseq"]):
                at, end = start[i], start[i] + cu[i + 1] - cu[i]
                while at < end:
                    to = min(end, (at // P + 1) * P)
                    most, pg = x[cu[i] + at - start[i]:cu[i] + to - start[i]].amax(0), table[i][at // P]
                    was[pg] = torch.maximum(was[pg], most) if at % P else most
                    at = to
            scales.append(was)
        return [None, None] + scales
    if c["op"] != "attn":
        return None
    P, cu, start, g = c["page"], s["cu"].tolist(), s["start"].tolist(), c["n_q"] // c["n_kv"]
    out = torch.zeros(s["ntok"], c["n_q"], c["d"], dtype=torch.float64, device=DEV)
    for i in range(c["nseq"]):
        n, L = cu[i + 1] - cu[i], start[i] + cu[i + 1] - cu[i]
        pages = s["table"][i, :-(-L // P)].long()
        p, j = torch.arange(start[i], L, device=DEV)[:, None], torch.arange(L, device=DEV)[None]
        hidden = j > p
        if c["window"]:
            hidden |= p - j >= c["window"]
        if c["prefix"]:
            hidden &= j >= c["prefix"]
        for h in range(c["n_kv"]):
            k = (s["k"][pages, h].double() * s["ks"][pages, h].double()[:, None, None]).reshape(-1, c["d"])[:L]
            v = (s["v"][pages, h].double() * s["vs"][pages, h].double()[:, None, None]).transpose(1, 2).reshape(-1, c["d"])[:L]
            q = s["q"][cu[i]:cu[i + 1]].double().view(n, c["n_q"], c["d"])[:, h * g:(h + 1) * g].transpose(0, 1)
            t = torch.einsum("gnd,ld->gnl", q, k) * s["scale"]
            if c["cap"]:
                t = torch.tanh(t / c["cap"]) * c["cap"]
            if c["alibi"]:
                t -= s["slopes"].double()[h * g:(h + 1) * g, None, None] * (p - j).abs()
            t.masked_fill_(hidden, float("-inf"))
            out[cu[i]:cu[i + 1], h * g:(h + 1) * g] = torch.einsum("gnl,ld->gnd", torch.softmax(t, -1), v).transpose(0, 1)
    return out.view(s["ntok"], -1)
