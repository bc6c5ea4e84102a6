"""The attention's cases with many query rows again, in calls with enough sequences to fill the GPU: the same sequences over and
over, whose outputs have to be the same bits.  (A small call spreads its rows thinly over the GPU; a large one gives 128 at a time to
the tensor cores.)"""
import numpy as np
import pytest

import test_kv_cache as T
from test_kv_cache import lq  # noqa: F401  (the fixture)

torch = pytest.importorskip("torch")
ONE = T.run_attn


def many(lq, c, table, start, cu, q, n_q, scale, prefix=None, cache=None, **kw):
    if cu is None or cu[-1] < 16 * len(start):
        return ONE(lq, c, table, start, cu, q, n_q, scale, prefix=prefix, cache=cache, **kw)
    nseq, ntok, grp = len(start), int(cu[-1]), n_q // c.n_kv
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    m = max(1, 2 * sms // (c.n_kv * nseq * -(-ntok * grp // (128 * nseq))))
    cus = np.concatenate([np.asarray(cu[:-1]) + i * ntok for i in range(m)] + [[m * ntok]])
    got = ONE(lq, c, np.tile(table, (m, 1)), list(start) * m, cus, np.tile(q, (m, 1)), n_q, scale,
              prefix=None if prefix is None else list(prefix) * m, cache=cache, **kw).reshape(m, ntok, -1)
    assert all(np.array_equal(got[0], g, equal_nan=True) for g in got[1:])
    return got[0]


@pytest.fixture(autouse=True)
def repeated(monkeypatch):
    monkeypatch.setattr(T, "run_attn", many)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [c for c in T.ATTN if max(c[5]) > 16])
@pytest.mark.parametrize("mask", ["causal", "window", "prefix", "bias", "all"])
def test_attn(lq, case, mask):  # noqa: F811
    T.test_attn(lq, case, mask)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_unaligned_rows(lq, d):  # noqa: F811
    T.test_attn_unaligned_rows(lq, 90, d)


@pytest.mark.gpu
@pytest.mark.parametrize("name,n", [("test_attn_hidden_nan_stays_hidden", 100), ("test_attn_visible_nan_is_seen", 70), ("test_attn_extreme_scales", 80),
                                    ("test_attn_sharp_rows", 66), ("test_attn_bad_pages", 65), ("test_far_pages", 40)])
def test_again(lq, name, n):  # noqa: F811
    getattr(T, name)(lq, n)


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,n_kv,grp", [(128, 64, 8, 4), (64, 16, 8, 4), (256, 32, 8, 4)])
def test_long_prompt(lq, d, page, n_kv, grp):  # noqa: F811
    """one prompt long enough by itself, behind cached tokens, against fp64 on the device"""
    n, L = 400, 1900
    g = torch.Generator(device="cuda").manual_seed(d)
    pages, n_q = -(-L // page), n_kv * grp
    k = torch.randint(-127, 128, (pages, n_kv, page, d), dtype=torch.int8, device="cuda", generator=g)
    v = torch.randint(-127, 128, (pages, n_kv, d, page), dtype=torch.int8, device="cuda", generator=g)
    ks, vs = (torch.rand(pages, n_kv, device="cuda", generator=g) * 0.02 + 0.01 for _ in range(2))
    q = torch.randn(n, n_q * d, device="cuda", generator=g)
    out = torch.empty_like(q)
    table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)[None]
    ws = torch.empty(lq.lq_kv8_attn_workspace_bytes(n_q, n_kv, d, 1, n), dtype=torch.uint8, device="cuda")
    start, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([L - n], [0, n]))
    lq.lq_kv8_attn(lq.LqKv8(k, v, ks, vs, pages, n_kv, page, d), table, pages, start, cu, 1, q, n_q, n_q * d, n, d ** -0.5, 0.0, 0, None, None, out,
                   n_q * d, ws, ws.numel())
    t = table[0].long()
    K = (k[t].double() * ks[t].double()[..., None, None]).permute(1, 0, 2, 3).reshape(n_kv, -1, d)[:, :L]
    V = (v[t].double() * vs[t].double()[..., None, None]).permute(1, 0, 3, 2).reshape(n_kv, -1, d)[:, :L]
    s = torch.einsum("hgnd,hld->hgnl", q.double().view(n, n_kv, grp, d).permute(1, 2, 0, 3), K) * d ** -0.5
    s.masked_fill_(torch.arange(L, device="cuda")[None] > torch.arange(L - n, L, device="cuda")[:, None], float("-inf"))
    w = torch.softmax(s, -1)
    ref, mag = (torch.einsum("hgnl,hld->hgnd", w, x).permute(2, 0, 1, 3).reshape(n, -1) for x in (V, V.abs()))
    # as for the long caches: scores below 12 in size, weights in two pieces, L / 8 sums
    assert ((out.double() - ref).abs() <= mag * (2 * 60 * 2.0 ** -21 + 2.0 ** -20 + (L / 8 + 64) * T.R.U)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rise", [0.0, 0.02, 3.0, -3.0])
@pytest.mark.parametrize("pad", [0, 3])
def test_long_rows_whose_maximum_moves(lq, d, rise, pad):  # noqa: F811
    """scores that rise, or fall, by `rise` per key over 1500 keys: the running maximum stays, moves now and then or at every step, and
    the sums taken out of the accumulators on the way follow it; q and out rows on 16- and on 4-byte addresses"""
    rng = np.random.default_rng(d + pad)
    n, L, page = 90, 1500, 64
    pages = -(-L // page)
    c = T.R.Cache(pages, 1, page, d, rng)
    c.ks[:] = 1.0 / 32
    steps = np.rint(np.arange(pages * page) / (pages * page) * 254 - 127)          # dim 0 rises from -127 to 127
    c.k[..., 0] = steps.reshape(pages, 1, page).astype(np.int8)
    q = (rng.standard_normal((n, 2 * d)) * 0.05).astype(np.float32)
    q[:, 0] = q[:, d] = rise * pages * page / 254 * 32
    table = np.arange(pages, dtype=np.int32)[None]
    got = T.run_attn(lq, c, table, [L - n], [0, n], q, 2, 1.0, pad=pad)
    ref, bound = T.R.attn(c, table, [L - n], [0, n], q, 2, 1.0)
    T.check(got, ref, bound, f"rise {rise}")
