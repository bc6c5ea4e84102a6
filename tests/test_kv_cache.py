"""Rotary positions, the 8-bit paged KV cache, its attention and its pages: refusals on the host (no GPU), parity with the
64-bit statements of tests/kv_ref.py on the GPU."""
import ctypes as C

import numpy as np
import pytest

import kv_ref as R

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lq():
    import block_quantized_weight_super_gb300 as pkg
    from block_quantized_weight_super_gb300 import build
    build.build()
    pkg.lib()
    return pkg


FAKE = 0x10000      # aligned, never dereferenced: these calls return before any CUDA call


def fake_cache(lq, **kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, n_pages=8, n_kv=2, page=16, head_dim=64)
    a.update(kw)
    return lq.LqKv8(**a)


# ---------------------------------------------------------------- refusals (host)

def test_rope_refusals(lq):
    ok = dict(q=FAKE, n_q=4, ld_q=256, q_out=FAKE, ld_qo=256, k=FAKE, n_k=2, ld_k=128, k_out=FAKE, ld_ko=128, head_dim=64,
              rot_dim=64, pairing=1, pos=FAKE, n_axes=1, axis=None, freq=FAKE, ntok=3, stream=0)
    for change, status in [(dict(q=None), lq.LQ_EINVAL), (dict(q=FAKE + 2), lq.LQ_EALIGN), (dict(freq=FAKE + 4), lq.LQ_EALIGN),
                           (dict(ld_q=255), lq.LQ_ESHAPE), (dict(rot_dim=63), lq.LQ_ESHAPE), (dict(rot_dim=66), lq.LQ_ESHAPE),
                           (dict(rot_dim=0), lq.LQ_ESHAPE), (dict(pairing=3), lq.LQ_EINVAL), (dict(n_axes=0), lq.LQ_EINVAL),
                           (dict(ntok=-1), lq.LQ_ESHAPE), (dict(pos=None), lq.LQ_EINVAL), (dict(k_out=None), lq.LQ_EINVAL),
                           (dict(n_q=0), lq.LQ_ESHAPE), (dict(ld_qo=260), lq.LQ_EINVAL), (dict(head_dim=2048, rot_dim=2048), lq.LQ_ESHAPE)]:
        with pytest.raises(lq.LqError) as e:
            lq.lq_rope(**{**ok, **change})
        assert e.value.status == status, change
    assert lq.lq_rope(**{**ok, "ntok": 0}) == lq.LQ_OK
    assert lq.lq_rope(**{**ok, "ntok": 0, "n_k": 0, "k": None, "k_out": None}) == lq.LQ_OK


CACHE_REFUSALS = [(dict(page=24), 3), (dict(page=8), 3), (dict(page=512), 3), (dict(head_dim=96), 3), (dict(n_kv=0), 3),
                  (dict(n_pages=0), 3), (dict(k=None), 1), (dict(v=FAKE + 8), 2), (dict(k_scale=FAKE + 2), 2), (dict(v_scale=None), 1)]


def test_append_refusals(lq):
    ok = dict(table=FAKE, max_pages=4, start=FAKE, cu=FAKE, nseq=2, k=FAKE, ld_k=128, v=FAKE, ld_v=128, ntok=5, stream=0)
    for change, status in CACHE_REFUSALS:
        with pytest.raises(lq.LqError) as e:
            lq.lq_kv8_append(fake_cache(lq, **change), **ok)
        assert e.value.status == status, change
    for change, status in [(dict(table=None), 1), (dict(start=FAKE + 1), 2), (dict(cu=None), 1), (dict(cu=FAKE + 2), 2), (dict(nseq=-1), 3),
                           (dict(nseq=70000), 3), (dict(ntok=-1), 3), (dict(nseq=0), 1), (dict(ld_k=127), 3), (dict(v=None), 1), (dict(max_pages=0), 3)]:
        with pytest.raises(lq.LqError) as e:
            lq.lq_kv8_append(fake_cache(lq), **{**ok, **change})
        assert e.value.status == status, change
    assert lq.lq_kv8_append(fake_cache(lq), **{**ok, "ntok": 0}) == lq.LQ_OK
    assert lq.lib().lq_kv8_append(None, FAKE, 4, FAKE, FAKE, 2, FAKE, 128, FAKE, 128, 5, None) == lq.LQ_EINVAL


def test_attn_refusals(lq):
    ws = lq.lq_kv8_attn_workspace_bytes(4, 2, 64, 2, 5)
    assert ws > 0
    for bad in [(3, 2, 64, 2, 5), (4, 2, 96, 2, 5), (0, 2, 64, 2, 5), (4, 0, 64, 2, 5), (4, 2, 64, -1, 5), (4, 2, 64, 2, -5)]:
        assert lq.lq_kv8_attn_workspace_bytes(*bad) == 0
    ok = dict(table=FAKE, max_pages=4, start=FAKE, cu=FAKE, nseq=2, q=FAKE, n_q=4, ld_q=256, ntok=5, scale=0.1, softcap=0.0, window=0,
              prefix=None, slopes=None, out=FAKE, ld_out=256, workspace=FAKE, ws_bytes=ws, stream=0)
    for change, status in CACHE_REFUSALS:
        with pytest.raises(lq.LqError) as e:
            lq.lq_kv8_attn(fake_cache(lq, **change), **ok)
        assert e.value.status == status, change
    nan = float("nan")
    for change, status in [(dict(n_q=3), 3), (dict(n_q=0), 3), (dict(scale=nan), 1), (dict(softcap=-1.0), 1), (dict(softcap=nan), 1),
                           (dict(window=-1), 1), (dict(q=None), 1), (dict(out=FAKE + 2), 2), (dict(ld_out=255), 3), (dict(prefix=FAKE + 1), 2),
                           (dict(slopes=FAKE + 1), 2), (dict(workspace=None), 4), (dict(ws_bytes=ws - 1), 4), (dict(workspace=FAKE + 128), 2),
                           (dict(cu=None), 1), (dict(table=FAKE + 2), 2)]:
        with pytest.raises(lq.LqError) as e:
            lq.lq_kv8_attn(fake_cache(lq), **{**ok, **change})
        assert e.value.status == status, change
    assert lq.lq_kv8_attn(fake_cache(lq), **{**ok, "ntok": 0}) == lq.LQ_OK


def test_page_refusals(lq):
    def refused(f, ok, changes):
        for change, status in changes:
            with pytest.raises(lq.LqError) as e:
                f(**{**ok, **change})
            assert e.value.status == status, (f.__name__, change)

    ok = dict(table=FAKE, max_pages=4, ref=FAKE, n_pages=8, page=16, start=FAKE, cu=None, nseq=2, info=FAKE, stream=0)
    refused(lq.lq_kv_reserve, ok, [(dict(table=None), 1), (dict(ref=FAKE + 2), 2), (dict(page=20), 3), (dict(nseq=9000), 3), (dict(info=None), 1),
                                   (dict(n_pages=0), 3), (dict(max_pages=0), 3), (dict(start=None), 1)])
    assert lq.lq_kv_reserve(**{**ok, "nseq": 0}) == lq.LQ_OK
    ok = dict(table=FAKE, n_rows=4, max_pages=4, ref=FAKE, n_pages=8, page=16, lens=FAKE, parent=FAKE, child=FAKE, n=2, src=FAKE, dst=FAKE, info=FAKE,
              stream=0)
    refused(lq.lq_kv_fork, ok, [(dict(lens=None), 1), (dict(parent=None), 1), (dict(child=FAKE + 1), 2), (dict(n=5000), 3), (dict(n=-1), 3),
                                (dict(src=None), 1), (dict(page=1), 3), (dict(n_rows=0), 3)])
    assert lq.lq_kv_fork(**{**ok, "n": 0}) == lq.LQ_OK
    ok = dict(table=FAKE, n_rows=4, max_pages=4, ref=FAKE, n_pages=8, lens=None, rows=FAKE, n=2, stream=0)
    refused(lq.lq_kv_release, ok, [(dict(rows=None), 1), (dict(n=-1), 3), (dict(n_rows=0), 3), (dict(lens=FAKE + 2), 2)])
    assert lq.lq_kv_release(**{**ok, "n": 0}) == lq.LQ_OK
    ok = dict(table=FAKE, n_rows=4, max_pages=4, ref=FAKE, n_pages=8, map=FAKE, src=FAKE, dst=FAKE, info=FAKE, stream=0)
    refused(lq.lq_kv_compact, ok, [(dict(map=None), 1), (dict(src=None), 1), (dict(dst=FAKE + 2), 2), (dict(n_rows=-1), 3), (dict(info=FAKE + 2), 2)])
    a, b = fake_cache(lq), fake_cache(lq, page=32)
    ok = dict(layers=[a, a], src=FAKE, dst=FAKE, n=2, count=None, stream=0)
    refused(lq.lq_kv8_copy_pages, ok, [(dict(src=None), 1), (dict(layers=[a, b]), 3), (dict(n=-1), 3), (dict(count=FAKE + 2), 2)])
    assert lq.lq_kv8_copy_pages(**{**ok, "n": 0}) == lq.LQ_OK
    assert lq.lib().lq_kv8_copy_pages(None, 1, FAKE, FAKE, 1, None, None) == lq.LQ_EINVAL


def test_struct_layout(lq):
    """the binding's struct has the header's layout (4 pointers, an int64, three int32, padded to 8)"""
    assert C.sizeof(lq.LqKv8) == 56
    assert [getattr(lq.LqKv8, n).offset for n in ("k", "v", "k_scale", "v_scale", "n_pages", "n_kv", "page", "head_dim")] == \
        [0, 8, 16, 24, 32, 40, 44, 48]


# ---------------------------------------------------------------- the statements themselves (host)

def test_append_statement_by_hand():
    """one page filled token by token: the scale follows the largest value, earlier codes are rounded again"""
    c = R.Cache(1, 1, 16, 64)
    table = np.array([[0]], np.int32)
    x = np.zeros((3, 64), np.float32)
    x[0, 0], x[1, 1], x[2, 2] = 1.27, 2.54, 0.635
    for i in range(3):
        c.append(table, [i], [0, 1], x[i:i + 1], -x[i:i + 1])
    assert c.ks[0, 0] == np.float32(2.54) * (np.float32(1) / np.float32(127))
    assert c.k[0, 0, 0, 0] == 64 and c.k[0, 0, 1, 1] == 127 and c.k[0, 0, 2, 2] == 32     # 63.5 and 31.75: to even, up
    assert c.v[0, 0, 0, 0] == -64 and c.v[0, 0, 1, 1] == -127


def test_attn_statement_by_hand():
    """one visible key gives its value; equal keys give the mean; a window of one gives the own value"""
    rng = np.random.default_rng(0)
    c = R.Cache(2, 1, 16, 64, rng)
    table = np.array([[1, 0]], np.int32)
    q = rng.standard_normal((1, 64)).astype(np.float32)
    V = np.concatenate([c.v[1, 0].T * np.float64(c.vs[1, 0]), c.v[0, 0].T * np.float64(c.vs[0, 0])])
    np.testing.assert_allclose(R.attn(c, table, [0], [0, 1], q, 1, 0.125)[0][0], V[0])
    np.testing.assert_allclose(R.attn(c, table, [19], [0, 1], q, 1, 0.0)[0][0], V[:20].mean(0))
    np.testing.assert_allclose(R.attn(c, table, [19], [0, 1], q, 1, 0.3, window=1)[0][0], V[19])
    np.testing.assert_allclose(R.attn(c, table, [19], [0, 1], q, 1, 0.0, window=1, prefix=[2])[0][0], V[[0, 1, 19]].mean(0))
    assert (R.attn(c, table, [-1], [0, 1], q, 1, 0.3)[0] == 0).all()


# ---------------------------------------------------------------- GPU

def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def up_cache(lq, c):
    t = [dev(x) for x in (c.k, c.v, c.ks, c.vs)]
    return lq.LqKv8(*t, c.n_pages, c.n_kv, c.page, c.d), t


def status(lq):
    return lq.lq_device_status()[1]


def run_attn(lq, c, table, start, cu, q, n_q, scale, softcap=0.0, window=0, prefix=None, slopes=None, pad=0, cache=None):
    ntok, nseq, w = q.shape[0], len(start), n_q * c.d
    cc = cache or up_cache(lq, c)[0]
    qd = torch.full((ntok, w + pad), 7.0, device="cuda")
    qd[:, :w] = dev(q)
    out = torch.full((ntok, w + pad), float("nan"), device="cuda")
    nb = lq.lq_kv8_attn_workspace_bytes(n_q, c.n_kv, c.d, nseq, ntok)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")           # scratch holds NaN patterns
    lq.lq_kv8_attn(cc, dev(table.astype(np.int32)), table.shape[1], dev(np.asarray(start, np.int32)),
                   None if cu is None else dev(np.asarray(cu, np.int32)), nseq, qd, n_q, w + pad, ntok, scale, softcap, window,
                   None if prefix is None else dev(np.asarray(prefix, np.int32)), None if slopes is None else dev(slopes.astype(np.float32)),
                   out, w + pad, ws, nb)
    torch.cuda.synchronize()
    assert torch.isnan(out[:, w:]).all()
    return out[:, :w].cpu().numpy()


def table_of(rng, counts, n_pages, width=None):
    t = np.full((len(counts), width or max(max(counts), 1)), -1, np.int32)
    perm, at = rng.permutation(n_pages), 0
    for i, n in enumerate(counts):
        t[i, :n] = perm[at:at + n]
        at += n
    return t


def check(got, ref, bound, what=""):
    got = got.astype(np.float64)
    assert np.isfinite(got).all(), what
    bad = np.abs(got - ref) > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {(np.abs(got - ref) / bound).max():.3g} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("ntok,n_q,n_k,d,rot,adjacent,axes,far", [
    (1, 32, 8, 128, 128, False, 1, 131072), (1, 3, 0, 64, 64, True, 1, 10), (5, 8, 4, 256, 256, False, 3, 1 << 20),
    (7, 5, 5, 64, 48, False, 2, 1 << 30), (300, 4, 2, 128, 64, True, 4, 5000), (2, 1, 1, 6, 6, False, 1, 100), (3, 2, 1, 20, 10, False, 2, 100),
    (0, 4, 2, 64, 64, False, 1, 10)])
def test_rope(lq, ntok, n_q, n_k, d, rot, adjacent, axes, far):
    rng = np.random.default_rng(ntok + d)
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    axis = rng.integers(0, axes, rot // 2).astype(np.uint8)
    pos = rng.integers(-far, far, (axes, ntok)).astype(np.int32)
    for pad, place in ((0, False), (4, False), (3, False), (0, True)):
        x = [rng.standard_normal((ntok, n * d)).astype(np.float32) for n in (n_q, n_k)]
        xi = [torch.full((ntok, n * d + pad), 3.0, device="cuda") for n in (n_q, n_k)]
        for a, b in zip(xi, x):
            a[:, :b.shape[1]] = dev(b)
        xo = xi if place else [torch.full_like(a, 5.0) for a in xi]
        lq.lq_rope(xi[0], n_q, n_q * d + pad, xo[0], n_q * d + pad, xi[1] if n_k else None, n_k, n_k * d + pad, xo[1] if n_k else None,
                   n_k * d + pad, d, rot, lq.LQ_ROPE_ADJACENT if adjacent else lq.LQ_ROPE_HALF, dev(pos), axes,
                   dev(axis) if axes > 1 else None, dev(freq), ntok)
        for n, a, b in zip((n_q, n_k), xo, x):
            if n and ntok:
                ref, bound = R.rope(b, n, d, rot, adjacent, pos, axis if axes > 1 else 0 * axis, freq)
                check(a[:, :n * d].cpu().numpy(), ref, bound + 1e-30, f"pad {pad}")
                assert (a[:, n * d:] == (3.0 if place else 5.0)).all()
    assert status(lq) == 0


@pytest.mark.gpu
def test_rope_bad_axis(lq):
    """an axis out of range leaves its pairs as they are and is reported"""
    x = torch.randn(2, 64, device="cuda")
    y = torch.empty_like(x)
    axis = torch.zeros(32, dtype=torch.uint8, device="cuda")
    axis[3] = 9
    lq.lq_rope(x, 1, 64, y, 64, None, 0, 0, None, 0, 64, 64, lq.LQ_ROPE_HALF, torch.ones(2, 2, dtype=torch.int32, device="cuda"), 2, axis,
               torch.ones(32, dtype=torch.float64, device="cuda"), 2)
    assert (y[:, 3] == x[:, 3]).all() and (y[:, 35] == x[:, 35]).all() and (y[:, 4] != x[:, 4]).all()
    assert status(lq) == lq.LQ_STATUS_BADARG and status(lq) == 0


def append_both(lq, c, table, start, cu, k, v, pad=0):
    cc, t = up_cache(lq, c)
    ntok, w = k.shape
    kd, vd = (torch.full((ntok, w + pad), float("nan"), device="cuda") for _ in range(2))
    kd[:, :w], vd[:, :w] = dev(k), dev(v)
    lq.lq_kv8_append(cc, dev(table), table.shape[1], dev(np.asarray(start, np.int32)), None if cu is None else dev(np.asarray(cu, np.int32)),
                     len(start), kd, w + pad, vd, w + pad, ntok)
    c.append(table, start, np.arange(len(start) + 1) if cu is None else cu, k, v)
    torch.cuda.synchronize()
    for name, got, ref in zip(("k", "v", "k_scale", "v_scale"), t, (c.k, c.v, c.ks, c.vs)):
        np.testing.assert_array_equal(got.cpu().numpy(), ref, err_msg=name)
    return cc


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,n_kv", [(64, 16, 3), (128, 32, 2), (256, 64, 1), (128, 128, 2), (64, 256, 1), (256, 16, 4)])
@pytest.mark.parametrize("pad", [0, 4, 1])
def test_append(lq, d, page, n_kv, pad):
    """ragged: empty, one token, a page's end, several pages, padding, a large and a small continuation"""
    rng = np.random.default_rng(d + page + pad)
    start = [0, 5, page - 1, 3, -2, page, -7, 2 * page + 1]
    ns = [1, 0, 1, 2 * page + 3, 4, page, 3, 5]
    cu = R.cu_of(ns)
    counts = [max(0, -(-(a + n) // page)) for a, n in zip(start, ns)]
    c = R.Cache(sum(counts) + 2, n_kv, page, d, rng)
    c.ks *= 30 if pad == 4 else 1            # earlier scales above the new ones in one variant
    table = table_of(rng, counts, sum(counts) + 2)
    k, v = (rng.standard_normal((cu[-1], n_kv * d)).astype(np.float32) * np.float32(rng.uniform(0.1, 4)) for _ in range(2))
    append_both(lq, c, table, start, cu, k, v, pad)
    assert status(lq) == 0


@pytest.mark.gpu
def test_append_borders(lq):
    """values on the borders between codes, tiny and huge scales, zeros, NaN and infinities"""
    rng = np.random.default_rng(5)
    d, page = 64, 16
    c = R.Cache(8, 1, page, d)
    table = np.arange(8, dtype=np.int32)[:, None]
    k = np.zeros((8, d), np.float32)
    for i, a in enumerate([127.0, 3.7, 1e-38, 1e-44, 3e38, 0.0]):
        s = np.float32(a) / np.float32(127)
        # every half-integer multiple of the scale, one step below it and one above
        h = (rng.integers(-127, 127, d) + 0.5) * np.float64(s)
        h = h.astype(np.float32)
        h[::3], h[1::3] = np.nextafter(h[::3], np.float32(9)), np.nextafter(h[1::3], np.float32(-9))
        k[i] = np.clip(h, -a, a)
        k[i, 7] = a
    k[6], k[7] = rng.standard_normal(d), rng.standard_normal(d)
    k[6, 3], k[7, 60] = np.nan, -np.inf
    append_both(lq, c, table, [0] * 8, None, k, k[::-1].copy())
    assert np.isnan(c.ks[6, 0]) and np.isnan(c.ks[7, 0]) and np.isnan(c.vs[0, 0])
    append_both(lq, c, table, [1] * 8, None, k[::-1].copy() * np.float32(1.7), k)          # the next slot: earlier codes again
    append_both(lq, c, table, [0] * 8, None, k[:1].repeat(8, 0), k[:1].repeat(8, 0))       # fresh pages forget the NaN
    assert np.isfinite(c.ks).all()


@pytest.mark.gpu
def test_append_bad_pages(lq):
    """a missing page, one outside the pool and a position past the table: those tokens are left out and reported"""
    rng = np.random.default_rng(6)
    c = R.Cache(4, 2, 16, 64, rng)
    table = np.array([[0, -1], [99, 1], [2, 3]], np.int32)
    ns = [20, 20, 40]
    cu = R.cu_of(ns)
    k, v = (rng.standard_normal((80, 128)).astype(np.float32) for _ in range(2))
    append_both(lq, c, table, [0, 0, 0], cu, k, v)
    assert status(lq) == lq.LQ_STATUS_BADARG and status(lq) == 0


@pytest.mark.gpu
def test_append_token_by_token(lq):
    """a page filled by single steps, as decoding does"""
    rng = np.random.default_rng(7)
    c = R.Cache(6, 2, 16, 128)
    table = np.array([[4, 1, 0], [2, 5, 3]], np.int32)
    for i in range(40):
        k, v = (rng.standard_normal((2, 256)).astype(np.float32) * np.float32(1 + 0.1 * i) for _ in range(2))
        append_both(lq, c, table, [i, i], None, k, v)


ATTN = [
    # d, page, n_q, n_kv, starts, new tokens
    (128, 16, 8, 2, [0], [1]), (128, 64, 4, 4, [63], [1]), (64, 32, 16, 2, [64, 0, 500], [1, 1, 1]), (256, 64, 8, 4, [700], [1]),
    (128, 128, 5, 1, [127, 128, 129, 1000], [1, 1, 1, 1]), (64, 256, 12, 1, [255, 256, 300], [1, 1, 1]), (256, 16, 2, 2, [15, 16, 17, 40], [1] * 4),
    (128, 16, 8, 8, [100, -1, 31, -5], [1, 1, 1, 1]), (64, 16, 24, 2, [77, 200], [3, 2]), (128, 32, 40, 8, [90, 0], [2, 5]),
    (128, 64, 8, 2, [0], [130]), (64, 16, 4, 4, [33, 0, 70], [100, 1, 65]), (256, 32, 4, 2, [10], [77]), (128, 16, 2, 1, [-3, 5, 0], [40, 0, 300]),
    (64, 128, 6, 2, [200, 0], [129, 257]), (256, 64, 8, 4, [5, 128], [64, 200]), (128, 64, 32, 2, [1500], [17]), (64, 64, 9, 1, [0], [260]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ATTN)
@pytest.mark.parametrize("mask", ["causal", "window", "prefix", "bias", "all"])
def test_attn(lq, case, mask):
    d, page, n_q, n_kv, start, ns = case
    rng = np.random.default_rng(abs(hash((d, page, n_q, tuple(start)))) % 1000)
    cu = R.cu_of(ns)
    counts = [max(0, -(-(a + n) // page)) for a, n in zip(start, ns)]
    c = R.Cache(sum(counts) + 1, n_kv, page, d, rng)
    table = table_of(rng, counts, c.n_pages)
    q = (rng.standard_normal((cu[-1], n_q * d)) * 3).astype(np.float32)
    q *= np.exp(rng.standard_normal((cu[-1], 1)) * 2).astype(np.float32)    # rows of unequal size
    opt = dict(causal={}, window=dict(window=37), prefix=dict(prefix=[50] * len(start)), bias=dict(slopes=2.0 ** -np.arange(1, n_q + 1)),
               all=dict(window=20, prefix=[3] * len(start), slopes=2.0 ** -np.arange(1, n_q + 1), softcap=20.0))[mask]
    one = all(n == 1 for n in ns)
    got = run_attn(lq, c, table, start, None if one else cu, q, n_q, d ** -0.5, pad=4 if mask == "window" else 0, **opt)
    ref, bound = R.attn(c, table, start, cu, q, n_q, d ** -0.5, **opt)
    check(got, ref, bound, f"{case} {mask}")
    assert status(lq) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attn_unaligned_rows(lq, n, d):
    """q and out rows on 4-byte addresses"""
    rng = np.random.default_rng(d + n)
    c = R.Cache(9, 2, 16, d, rng)
    table = table_of(rng, [8], 9)
    q = rng.standard_normal((n, 4 * d)).astype(np.float32)
    got = run_attn(lq, c, table, [30], [0, n], q, 4, d ** -0.5, pad=1)
    ref, bound = R.attn(c, table, [30], [0, n], q, 4, d ** -0.5)
    check(got, ref, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 100])
def test_attn_hidden_nan_stays_hidden(lq, n):
    """NaN scales on pages that no visible key lies on: behind a window, behind the end, in the rest of the pool"""
    rng = np.random.default_rng(8)
    for d in (64, 128, 256):
        c = R.Cache(60, 2, 16, d, rng)
        table = table_of(rng, [50], 60, width=52)
        table[0, 50:] = table[0, 0]
        start = 600
        seen = set()
        for p in range(start, start + n):
            seen |= set(range((p - 31) // 16, p // 16 + 1)) | {0}
        hide = [p for p in range(60) if p not in set(table[0, sorted(seen)])]
        c.ks[hide], c.vs[hide] = np.nan, np.nan
        q = rng.standard_normal((n, 4 * d)).astype(np.float32)
        got = run_attn(lq, c, table, [start], [0, n], q, 4, d ** -0.5, window=32, prefix=[16])
        ref, bound = R.attn(c, table, [start], [0, n], q, 4, d ** -0.5, window=32, prefix=[16])
        check(got, ref, bound, f"d {d}")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 70])
def test_attn_visible_nan_is_seen(lq, n):
    """a visible page with a NaN scale, and a NaN query, give NaN and not a number; other rows are not touched"""
    rng = np.random.default_rng(9)
    c = R.Cache(30, 2, 16, 128, rng)
    table = table_of(rng, [20, 10], 30)
    q = rng.standard_normal((2 * n, 512)).astype(np.float32)
    cu = [0, n, 2 * n]
    clean = run_attn(lq, c, table, [200, 80], cu, q, 4, 0.1)
    c.vs[table[0, 3], 0] = np.nan
    got = run_attn(lq, c, table, [200, 80], cu, q, 4, 0.1)
    assert np.isnan(got[:n, :256]).all()
    assert np.array_equal(got[:n, 256:], clean[:n, 256:]) and np.array_equal(got[n:], clean[n:])
    c.vs[table[0, 3], 0] = 0.1
    q[0, 5] = np.nan
    got = run_attn(lq, c, table, [200, 80], cu, q, 4, 0.1)
    assert np.isnan(got[0, :128]).all() and np.array_equal(got[n:], clean[n:])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 80])
def test_attn_extreme_scales(lq, n):
    """value scales that differ by 2^60 between pages, key scales of 0 and queries of 0"""
    rng = np.random.default_rng(10)
    for d in (64, 128, 256):
        c = R.Cache(20, 1, 16, d, rng)
        table = table_of(rng, [18], 20)
        c.vs[table[0, :6]] *= np.float32(2.0 ** -60)
        c.vs[table[0, 6:9]] = 0
        c.ks[table[0, 2:4]] = 0
        q = rng.standard_normal((n, 2 * d)).astype(np.float32)
        q[:, :d] = 0
        for start in (40, 180):          # tiny values alone; beside large ones
            got = run_attn(lq, c, table, [start], [0, n], q, 2, d ** -0.5)
            ref, bound = R.attn(c, table, [start], [0, n], q, 2, d ** -0.5)
            check(got, ref, bound, f"d {d} start {start}")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 66])
def test_attn_sharp_rows(lq, n):
    """scores that rise along the keys by thousands: the running maximum moves at every step"""
    rng = np.random.default_rng(11)
    for d in (64, 128, 256):
        c = R.Cache(12, 1, 32, d, rng)
        table = np.arange(12, dtype=np.int32)[None]
        for up in (1, -1):
            ramp = np.rint(np.linspace(-127, 127, 384))[::up].reshape(12, 1, 32)
            c.k[..., 0] = ramp.astype(np.int8)
            c.ks[:] = 1.0
            q = np.zeros((n, 2 * d), np.float32)
            q[:, 0], q[:, d] = 20.0, -20.0
            got = run_attn(lq, c, table, [300], [0, n], q, 2, 1.0)
            ref, bound = R.attn(c, table, [300], [0, n], q, 2, 1.0)
            check(got, ref, bound, f"d {d} up {up}")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 65])
def test_attn_bad_pages(lq, n):
    """keys without a page are left out and reported; a row without any key left is zero"""
    rng = np.random.default_rng(12)
    c = R.Cache(6, 1, 16, 64, rng)
    table = np.array([[0, -1, 2, 77, 4], [-1, -1, -1, -1, -1]], np.int32)
    q = rng.standard_normal((2 * n, 128)).astype(np.float32)
    start = [79 - n + 1 + 40, 40]          # the first one passes the table's end
    cu = [0, n, 2 * n]
    got = run_attn(lq, c, table, start, cu, q, 2, 0.125)
    ref, bound = R.attn(c, table, start, cu, q, 2, 0.125)
    check(got, ref, bound)
    assert (got[n:] == 0).all()
    assert status(lq) == lq.LQ_STATUS_BADARG and status(lq) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 40])
def test_far_pages(lq, n):
    """page offsets past 2^32 bytes"""
    d, page, n_kv = 128, 64, 8
    n_pages = (1 << 32) // (page * n_kv * d) + 40
    rng = np.random.default_rng(13)
    k, v = (torch.zeros(n_pages, n_kv * page * d, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n_pages, n_kv, device="cuda") for _ in range(2))
    far = lq.LqKv8(k, v, ks, vs, n_pages, n_kv, page, d)
    L = 5 * page
    table = np.array([[n_pages - 1 - 3 * i for i in range(6)]], np.int32)
    near = np.arange(6, dtype=np.int32)[None]
    x, y = (torch.randn(L, n_kv * d, device="cuda") for _ in range(2))
    small = R.Cache(6, n_kv, page, d)
    cs, _ = up_cache(lq, small)
    q = rng.standard_normal((n, 2 * n_kv * d)).astype(np.float32)
    outs = []
    for cc, t in ((far, table), (cs, near)):
        lq.lq_kv8_append(cc, dev(t), 6, dev(np.array([0], np.int32)), dev(np.array([0, L], np.int32)), 1, x, n_kv * d, y, n_kv * d, L)
        outs.append(run_attn(lq, small, t, [L - n], [0, n], q, 2 * n_kv, 0.1, cache=cc))
    assert np.array_equal(*outs) and np.isfinite(outs[0]).all() and np.abs(outs[0]).max() > 0
    # copies there and back
    a, b = table[0, :5].copy(), (table[0, :5] - 1).copy()
    lq.lq_kv8_copy_pages([far], dev(a), dev(b), 5)
    assert torch.equal(k[a.tolist()], k[b.tolist()]) and torch.equal(vs[a.tolist()], vs[b.tolist()])


@pytest.mark.gpu
@pytest.mark.parametrize("n,L,d,page", [(1, 20000, 128, 16), (2, 9000, 256, 64), (1, 40000, 64, 256), (300, 3000, 128, 64), (150, 2600, 256, 32), (200, 3000, 64, 16)])
def test_attn_long(lq, n, L, d, page):
    """long caches, split over many workers, against fp64 on the device"""
    g = torch.Generator(device="cuda").manual_seed(L)
    n_kv, n_q = 2, 6
    pages = -(-L // page)
    k = torch.randint(-127, 128, (pages, n_kv, page, d), dtype=torch.int8, device="cuda", generator=g)
    v = torch.randint(-127, 128, (pages, n_kv, d, page), dtype=torch.int8, device="cuda", generator=g)
    ks, vs = (torch.rand(pages, n_kv, device="cuda", generator=g) * 0.02 + 0.01 for _ in range(2))
    q = torch.randn(n, n_q * d, device="cuda", generator=g)
    out = torch.empty_like(q)
    table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)[None]
    nb = lq.lq_kv8_attn_workspace_bytes(n_q, n_kv, d, 1, n)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lq.lq_kv8_attn(lq.LqKv8(k, v, ks, vs, pages, n_kv, page, d), table, pages, torch.tensor([L - n], dtype=torch.int32, device="cuda"), cu, 1, q, n_q,
                   n_q * d, n, d ** -0.5, 0.0, 0, None, None, out, n_q * d, ws, nb)
    t = table[0].long()
    K = (k[t].double() * ks[t].double()[..., None, None]).permute(1, 0, 2, 3).reshape(n_kv, -1, d)[:, :L]
    V = (v[t].double() * vs[t].double()[..., None, None]).permute(1, 0, 3, 2).reshape(n_kv, -1, d)[:, :L]
    Q = q.double().view(n, n_kv, 3, d).permute(1, 2, 0, 3)
    s = torch.einsum("hgnd,hld->hgnl", Q, K) * d ** -0.5
    j = torch.arange(L, device="cuda")
    s.masked_fill_(j[None] > torch.arange(L - n, L, device="cuda")[:, None], float("-inf"))
    w = torch.softmax(s, -1)
    ref = torch.einsum("hgnl,hld->hgnd", w, V).permute(2, 0, 1, 3).reshape(n, -1)
    mag = torch.einsum("hgnl,hld->hgnd", w, V.abs()).permute(2, 0, 1, 3).reshape(n, -1)
    # scores below 12 in size (2^-21 of the pieces on a sum of absolute terms below 60), weights in two pieces, L / 8 sums
    bound = mag * (2 * 60 * 2.0 ** -21 + 2.0 ** -20 + (L / 8 + 64) * R.U)
    assert ((out.double() - ref).abs() <= bound).all()
    first = out.clone()
    lq.lq_kv8_attn(lq.LqKv8(k, v, ks, vs, pages, n_kv, page, d), table, pages, torch.tensor([L - n], dtype=torch.int32, device="cuda"), cu, 1, q, n_q,
                   n_q * d, n, d ** -0.5, 0.0, 0, None, None, out, n_q * d, ws, nb)
    assert torch.equal(first, out)          # the same inputs, the same bits


@pytest.mark.gpu
def test_pages(lq):
    """a random life of a pool: reserve, fork, release, compact, against the statement; and every refusal on the device"""
    rng = np.random.default_rng(14)
    rows, width, n_pages, page = 12, 9, 60, 16
    m = R.Pages(rows, width, n_pages, page)
    table, ref, lens = dev(m.table), dev(m.ref), dev(m.lens)
    info = torch.full((2,), 9, dtype=torch.int32, device="cuda")

    def same(what, got=None):
        np.testing.assert_array_equal(table.cpu().numpy(), m.table, err_msg=what)
        np.testing.assert_array_equal(ref.cpu().numpy(), m.ref, err_msg=what)
        np.testing.assert_array_equal(lens.cpu().numpy(), m.lens, err_msg=what)
        if got is not None:
            assert tuple(info.tolist()) == tuple(got), (what, info.tolist(), got)

    for step in range(60):
        kind = rng.integers(0, 4)
        if kind == 0 or step < 4:
            ns = rng.integers(0, 40, rows) * (rng.random(rows) < 0.4)
            cu = R.cu_of(ns)
            start = m.lens.copy()
            got = m.reserve(start, cu)
            lq.lq_kv_reserve(table, width, ref, n_pages, page, dev(start), dev(cu), rows, info)
            same(f"{step} reserve", got)
            if got == (0, 0):
                m.lens += ns.astype(np.int32)
                lens.copy_(dev(m.lens))
        elif kind == 1:
            empty, full = np.flatnonzero(m.lens == 0), np.flatnonzero(m.lens > 0)
            if len(empty) and len(full):
                child = rng.permutation(empty)[:rng.integers(1, len(empty) + 1)].astype(np.int32)
                parent = rng.choice(full, len(child)).astype(np.int32)
                s, d, got = m.fork(parent, child)
                src, dst = (torch.full((len(child),), 7, dtype=torch.int32, device="cuda") for _ in range(2))
                lq.lq_kv_fork(table, rows, width, ref, n_pages, page, lens, dev(parent), dev(child), len(child), src, dst, info)
                same(f"{step} fork", got)
                np.testing.assert_array_equal(src.cpu().numpy(), s)
                np.testing.assert_array_equal(dst.cpu().numpy(), d)
        elif kind == 2:
            r = rng.integers(0, rows, 3).astype(np.int32)       # a row twice, empty rows
            m.release(r)
            lq.lq_kv_release(table, rows, width, ref, n_pages, lens, dev(r), 3)
            same(f"{step} release")
        else:
            mp, s, d, k = m.compact()
            gm = torch.full((n_pages,), 7, dtype=torch.int32, device="cuda")
            src, dst = (torch.full((n_pages // 2,), 7, dtype=torch.int32, device="cuda") for _ in range(2))
            lq.lq_kv_compact(table, rows, width, ref, n_pages, gm, src, dst, info)
            same(f"{step} compact", (k, 0))
            for a, b in ((gm, mp), (src, s), (dst, d)):
                np.testing.assert_array_equal(a.cpu().numpy(), b)
    assert status(lq) == 0
    # out of range on the device: nothing changes
    one = lambda *v: dev(np.array(v, np.int32))  # noqa: E731
    lq.lq_kv_reserve(table, width, ref, n_pages, page, one(width * page), None, 1, info)
    same("past the table", (0, 1))
    src = dst = torch.empty(1, dtype=torch.int32, device="cuda")
    for p, c in ((-1, 0), (0, rows), (rows + 5, 1)):
        lq.lq_kv_fork(table, rows, width, ref, n_pages, page, lens, one(p), one(c), 1, src, dst.clone(), info)
        same("fork of no row", (0, 1))
    lq.lq_kv_release(table, rows, width, ref, n_pages, lens, one(-3, rows), 2)
    same("release of no row")
    assert status(lq) == lq.LQ_STATUS_BADARG


@pytest.mark.gpu
@pytest.mark.parametrize("n_pages", [1, 2, 4095, 4097, 50000])
def test_pages_large(lq, n_pages):
    """pools of one tile more and less, many sequences, long requests"""
    rng = np.random.default_rng(n_pages)
    nseq, width = 300, 200
    m = R.Pages(nseq, width, n_pages, 16)
    m.ref[:] = rng.random(n_pages) < 0.5
    if n_pages > 1:
        m.ref[rng.integers(0, n_pages)] = 3
    ns = rng.integers(0, 30 * n_pages // nseq + 2, nseq).clip(0, width * 16)
    ns[5] = min(width * 16, 2 * n_pages)
    cu, start = R.cu_of(ns), np.zeros(nseq, np.int32)
    table, ref, info = dev(m.table), dev(m.ref), torch.zeros(2, dtype=torch.int32, device="cuda")
    got = m.reserve(start, cu)
    lq.lq_kv_reserve(table, width, ref, n_pages, 16, dev(start), dev(cu), nseq, info)
    assert tuple(info.tolist()) == got
    np.testing.assert_array_equal(table.cpu().numpy(), m.table)
    np.testing.assert_array_equal(ref.cpu().numpy(), m.ref)
    mp, s, d, k = m.compact()
    gm = torch.empty(n_pages, dtype=torch.int32, device="cuda")
    src, dst = (torch.empty(max(n_pages // 2, 1), dtype=torch.int32, device="cuda") for _ in range(2))
    lq.lq_kv_compact(table, nseq, width, ref, n_pages, gm, src, dst, info)
    np.testing.assert_array_equal(gm.cpu().numpy(), mp)
    np.testing.assert_array_equal(src.cpu().numpy()[:n_pages // 2], s)
    np.testing.assert_array_equal(dst.cpu().numpy()[:n_pages // 2], d)
    np.testing.assert_array_equal(table.cpu().numpy(), m.table)
    np.testing.assert_array_equal(ref.cpu().numpy(), m.ref)


@pytest.mark.gpu
@pytest.mark.parametrize("layers", [1, 3, 70])
def test_copy_pages(lq, layers):
    rng = np.random.default_rng(15)
    cs = [R.Cache(8, 3, 16, 64, rng) for _ in range(layers)]
    ups = [up_cache(lq, c) for c in cs]
    src, dst = np.array([0, -1, 2, 3, 1], np.int32), np.array([4, 5, -1, 6, 7], np.int32)
    lq.lq_kv8_copy_pages([u[0] for u in ups], dev(src), dev(dst), 5, dev(np.array([4], np.int32)))
    for c, (_, t) in zip(cs, ups):
        for x in (c.k, c.v, c.ks, c.vs):
            x[4], x[6] = x[0], x[3]
        for got, want in zip(t, (c.k, c.v, c.ks, c.vs)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
    lq.lq_kv8_copy_pages([ups[0][0]], dev(np.array([0], np.int32)), dev(np.array([8], np.int32)), 1)
    assert status(lq) == lq.LQ_STATUS_BADARG


@pytest.mark.gpu
def test_streams_and_graphs(lq):
    """calls on a stream of its own, and a step captured into a graph and replayed with other inputs in place"""
    rng = np.random.default_rng(16)
    d, page, n_kv, n_q = 128, 16, 2, 8
    c = R.Cache(16, n_kv, page, d, rng)
    table = table_of(rng, [4, 5, 3], 16, width=6)
    start = np.array([30, 70, -1], np.int32)
    cc, _ = up_cache(lq, c)
    td, sd = dev(table), dev(start)
    q, k, v = (torch.zeros(3, n * d, device="cuda") for n in (n_q, n_kv, n_kv))
    out = torch.empty(3, n_q * d, device="cuda")
    nb = lq.lq_kv8_attn_workspace_bytes(n_q, n_kv, d, 3, 3)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def step(stream=None):
        lq.lq_kv8_append(cc, td, 6, sd, None, 3, k, n_kv * d, v, n_kv * d, 3, stream)
        lq.lq_kv8_attn(cc, td, 6, sd, None, 3, q, n_q, n_q * d, 3, 0.1, 0.0, 0, None, None, out, n_q * d, ws, nb, stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    c.append(table, start, np.arange(4), np.zeros((3, n_kv * d), np.float32), np.zeros((3, n_kv * d), np.float32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        start = start + 1
        new = [rng.standard_normal((3, n * d)).astype(np.float32) for n in (n_q, n_kv, n_kv)]
        for a, b in zip((q, k, v), new):
            a.copy_(dev(b))
        sd.copy_(dev(start))
        graph.replay()
        torch.cuda.synchronize()
        c.append(table, start, np.arange(4), new[1], new[2])
        ref, bound = R.attn(c, table, start, np.arange(4), new[0], n_q, 0.1)
        check(out.cpu().numpy(), ref, bound, f"replay {i}")
    assert status(lq) == 0


@pytest.mark.gpu
def test_example_layer(lq):
    """the example's prompts, decode graph, forks and compaction: finite outputs, equal samples equal, and the prompts' attention
    over the appended cache against the 64-bit statement"""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode_layer as ex
    y, outs, layer = ex.main(steps=3)
    assert torch.isfinite(y).all()
    for o in outs:
        assert torch.isfinite(o).all()
        assert torch.equal(o[2], o[3])
    # one more decode step of row 0 (row 3 shares its prompt's pages): attention against the statement over the layer's own cache
    P, rows = ex.PAGE, [0, 3]
    start = layer.lens[rows].clone()
    table = layer.table[rows].contiguous()
    c = R.Cache(layer.n_pages, ex.N_KV, P, ex.D)
    k, v, ks, vs = layer.cache.tensors
    c.k, c.v = k.view(c.k.shape).cpu().numpy(), v.view(c.v.shape).cpu().numpy()
    c.ks, c.vs = ks.cpu().numpy(), vs.cpu().numpy()
    q = np.random.default_rng(3).standard_normal((2, ex.NQ)).astype(np.float32)
    got = run_attn(lq, c, table.cpu().numpy(), (start - 1).tolist(), None, q, ex.N_Q, 0.0625, cache=layer.cache)
    ref, bound = R.attn(c, table.cpu().numpy(), (start - 1).tolist(), np.arange(3), q, ex.N_Q, 0.0625)
    check(got, ref, bound)
    assert int((layer.ref > 0).sum()) == int((layer.table >= 0).sum()) - int((layer.ref - 1).clamp(min=0).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rope_frequency_not_finite(lq, bad):
    """a pair whose frequency is not finite is copied and reported; the others are rotated"""
    import torch
    x = torch.randn(3, 64, device="cuda")
    freq = torch.ones(32, dtype=torch.float64, device="cuda")
    freq[5] = bad
    pos = torch.tensor([[1, 2, 3]], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    lq.lq_device_status()
    lq.lq_rope(x, 1, 64, out, 64, None, 0, 0, None, 0, 64, 64, lq.LQ_ROPE_HALF, pos, 1, None, freq, 3)
    rc, bits = lq.lq_device_status()
    assert bits == 2
    assert torch.equal(out[:, [5, 37]], x[:, [5, 37]])
    c, s = torch.cos(pos[0].double()), torch.sin(pos[0].double())
    want = x[:, 6].double() * c - x[:, 38].double() * s
    assert (out[:, 6].double() - want).abs().max() < 4e-6
