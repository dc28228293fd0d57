"""The product of 8-bit integers with token and channel scales on the GPU
against its oracle.

The integer sum is exact.  Each float32 step rounds by at most half a step
(2^-24 relative): the sum's conversion, two scale products, the bias and the
residual added; then one rounding to the output's dtype (2^-24 or 2^-8).
"""
import numpy as np
import pytest
import torch

import spatially_sparse_incremental_b200 as sige
from helpers import bits
from oracle import qcache as oq
from test_gpu_qcache import tile_list

pytestmark = pytest.mark.gpu
DEV = "cuda"


def operands(rng, n, h, w, c, co, extreme=False):
    lo, hi = (-128, 128) if extreme else (-127, 128)
    a = rng.integers(lo, hi, (n, h, w, c)).astype(np.int8)
    wt = rng.integers(lo, hi, (co, 1, 1, c)).astype(np.int8)
    if extreme:
        a[..., :] = -128
        wt[:] = -128
    sa = (rng.random((n, h, w, 1)) * 0.02).astype(np.float32)
    sa[rng.random((n, h, w, 1)) < 0.05] = 0
    sw = (rng.random((co, 1, 1, 1)) * 0.01).astype(np.float32)
    return a, sa, wt, sw


def cache(codes, scales):
    return sige.QCache(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), "s8")


def check(got, a, sa, wt, sw, bias, res, dtype, tok=None):
    """got [T, Co] against the oracle at tokens `tok` of the flat operands."""
    c, co = a.shape[-1], wt.shape[0]
    A, S = a.reshape(-1, c), sa.reshape(-1)
    R = None if res is None else oq.f64(res).reshape(-1, co)
    if tok is not None:
        A, S, R = A[tok], S[tok], None if R is None else R[tok]
    ref = oq.qlinear(A, S, wt.reshape(co, c), sw.reshape(-1), None if bias is None else bias, R)
    prod = np.abs(oq.qlinear(A, S, wt.reshape(co, c), sw.reshape(-1)))
    tot = prod + (0 if bias is None else np.abs(bias)) + (0 if R is None else np.abs(R))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    allow = 3.01 * 2.0 ** -24 * prod + 2 * 2.0 ** -24 * tot + half * np.abs(ref) * 1.0001 + 1e-44
    d = np.abs(oq.f64(got).reshape(ref.shape) - ref)
    assert (d <= allow).all(), f"max |d| / allowance = {(d / allow).max():.3g}"


def run_case(seed, n, h, w, c, co, dtype, bias=True, residual=False, extreme=False):
    rng = np.random.default_rng(seed)
    a, sa, wt, sw = operands(rng, n, h, w, c, co, extreme)
    b = rng.normal(size=co).astype(np.float32) if bias else None
    r = torch.from_numpy(rng.normal(size=(n, h, w, co))).to(dtype) if residual else None
    y = sige.sige_qlinear(cache(a, sa), cache(wt, sw), None if b is None else torch.from_numpy(b).to(DEV),
                          residual=None if r is None else r.to(DEV), dtype=dtype)
    torch.cuda.synchronize()
    check(y, a, sa, wt, sw, b, r, dtype)
    return y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,h,w,c,co", [
    (1, 16, 16, 320, 320), (1, 1, 1, 1280, 1280), (1, 1, 3, 64, 8), (2, 13, 11, 640, 640), (1, 8, 8, 16, 16),
    (1, 13, 11, 74, 51), (1, 1, 1, 1, 1), (1, 5, 3, 33, 129), (3, 17, 9, 144, 328), (1, 32, 32, 1280, 72), (1, 4, 4, 5120, 320),
    (1, 1, 2, 48, 1000), (1, 20, 20, 128, 257), (1, 1, 40, 2048, 96), (4, 16, 16, 96, 1300), (1, 3, 43, 272, 7),
])
def test_every_token(n, h, w, c, co, dtype):
    run_case(c + co, n, h, w, c, co, dtype)
    run_case(c + co + 1, n, h, w, c, co, dtype, bias=False, residual=True)


def test_more_tokens_than_the_launch_has_blocks():
    run_case(3, 2, 128, 96, 64, 640, torch.bfloat16, residual=True)
    run_case(4, 1, 150, 150, 320, 48, torch.float32)


@pytest.mark.parametrize("c", [131071, 131056])
def test_largest_sums(c):
    """Codes of -128 throughout at the most channels: sums of 2^14 c."""
    run_case(7, 1, 1, 2, c, 3, torch.float32, extreme=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,h,w,c,co,b,frac", [
    (1, 16, 16, 1280, 1280, 1, 0.08), (1, 64, 64, 320, 320, 4, 0.1), (2, 13, 11, 640, 200, 4, 0.3), (1, 9, 7, 48, 24, 2, 0.5),
    (2, 24, 24, 320, 960, 8, 0.4), (1, 30, 30, 74, 51, 4, 0.3), (1, 40, 40, 5120, 640, 2, 0.02), (1, 64, 64, 64, 64, 64, 1.0),
    (3, 16, 16, 128, 40, 1, 0.01), (2, 32, 32, 256, 512, 4, 1.0),
])
def test_listed_tiles(n, h, w, c, co, b, frac, dtype):
    rng = np.random.default_rng(c + b)
    a, sa, wt, sw = operands(rng, n, h, w, c, co)
    idx, where = tile_list(rng, h, w, b, frac)
    bias = rng.normal(size=co).astype(np.float32)
    res = torch.from_numpy(rng.normal(size=(n, h, w, co))).to(dtype)
    y0 = torch.from_numpy(rng.normal(size=(n, h, w, co))).to(dtype)
    y = y0.to(DEV)
    sige.sige_qlinear(cache(a, sa), cache(wt, sw), torch.from_numpy(bias).to(DEV), y, residual=res.to(DEV), **where)
    torch.cuda.synchronize()
    t1 = oq.tokens(idx, b, h, w)
    tok = (np.arange(n)[:, None] * (h * w) + t1[None]).reshape(-1)
    rest = np.setdiff1d(np.arange(n * h * w), tok)
    got = y.cpu().view(-1, co)
    assert torch.equal(bits(got[rest]), bits(y0.view(-1, co)[rest]))
    check(got[tok], a, sa, wt, sw, bias, res, dtype, tok)


def test_lists_that_are_short_long_or_out_of_the_map():
    rng = np.random.default_rng(1)
    for c in (64, 36):   # both kernels
        n, h, w, co = 2, 10, 10, 48
        a, sa, wt, sw = operands(rng, n, h, w, c, co)
        A, W = cache(a, sa), cache(wt, sw)
        full = sige.sige_qlinear(A, W)
        tiles = torch.tensor([[4, 4], [4, 4], [8, 8], [-4, 0], [0, -1], [12, 0], [0, 400], [0, 0]], dtype=torch.int32, device=DEV)
        for count, cap, listed in ((0, 8, []), (-3, 8, []), (99, 3, [(4, 4), (8, 8)]), (8, 8, [(4, 4), (8, 8), (0, 0)])):
            y = torch.full((n, h, w, co), 3.0, dtype=torch.bfloat16, device=DEV)
            sige.sige_qlinear(A, W, None, y, idx=tiles, capacity=cap, block=4,
                              count=torch.tensor([count], dtype=torch.int32, device=DEV))
            hit = torch.zeros((h, w), dtype=torch.bool, device=DEV)
            for i, j in listed:
                hit[i:i + 4, j:j + 4] = True
            assert torch.equal(y[:, hit], full[:, hit]) and (y[:, ~hit] == 3).all()


def test_poisoned_and_empty_tokens():
    """A token with a NaN scale gives NaN in its own row only; one with scale 0
    the bias."""
    rng = np.random.default_rng(2)
    for c in (64, 36):
        a, sa, wt, sw = operands(rng, 1, 4, 50, c, 40)
        sa[0, 1, 7], sa[0, 2, 3] = np.nan, 0
        a[0, 1, 7] = 0
        b = rng.normal(size=40).astype(np.float32)
        y = sige.sige_qlinear(cache(a, sa), cache(wt, sw), torch.from_numpy(b).to(DEV), dtype=torch.float32).cpu()
        bad = torch.isnan(y)
        assert bad[0, 1, 7].all() and bad.sum() == 40
        assert torch.equal(y[0, 2, 3], torch.from_numpy(b))


def test_unaligned_operands():
    """Codes, outputs, residual and bias that start off 16 bytes."""
    rng = np.random.default_rng(9)
    n, h, w, c, co = 1, 9, 9, 64, 72
    a, sa, wt, sw = operands(rng, n, h, w, c, co)
    b = torch.from_numpy(rng.normal(size=co).astype(np.float32)).to(DEV)
    r = torch.from_numpy(rng.normal(size=(n, h, w, co))).to(torch.bfloat16).to(DEV)
    ref = sige.sige_qlinear(cache(a, sa), cache(wt, sw), b, residual=r)

    def off(t, k):
        buf = torch.empty(t.numel() + k, dtype=t.dtype, device=DEV)
        buf[k:].copy_(t.reshape(-1))
        return buf[k:].view(t.shape)

    A, W = cache(a, sa), cache(wt, sw)
    for ka, kw, kb, kr, ky in ((1, 0, 0, 0, 0), (0, 4, 0, 0, 0), (0, 0, 1, 0, 0), (0, 0, 0, 1, 0), (0, 0, 0, 0, 1), (0, 0, 3, 4, 2),
                               (0, 0, 0, 8, 8)):
        y = off(torch.zeros_like(ref), ky)
        sige.sige_qlinear(sige.QCache(off(A.codes, ka), off(A.scales, ka), "s8"),
                          sige.QCache(off(W.codes, kw), off(W.scales, kw), "s8"), off(b, kb), y, residual=off(r, kr))
        assert torch.equal(y, ref), (ka, kw, kb, kr, ky)


def test_streams_graphs_and_repeats():
    """Two streams at once, a captured graph replayed on new values, and the
    same call again: the same bits each time."""
    rng = np.random.default_rng(13)
    n, h, w, c, co = 1, 32, 32, 640, 1280
    a, sa, wt, sw = operands(rng, n, h, w, c, co)
    A, W = cache(a, sa), cache(wt, sw)
    idx, where = tile_list(rng, h, w, 4, 0.1)
    ref = sige.sige_qlinear(A, W)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    outs = [sige.sige_qlinear(A, W, stream=s) for _ in range(4) for s in (s1, s2)]
    y0 = torch.zeros_like(ref)
    y1 = torch.zeros_like(ref)
    torch.cuda.synchronize()
    tiles = [sige.sige_qlinear(A, W, None, y, stream=s, **where) for s, y in ((s1, y0), (s2, y1))]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs) and torch.equal(tiles[0], tiles[1])
    ws = sige.zeros_workspace(256, DEV)
    out = torch.zeros_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sige.sige_qlinear(A, W, None, out, workspace=ws, **where)
    A.codes.copy_(torch.from_numpy(rng.integers(-127, 128, (n, h, w, c)).astype(np.int8)))
    graph.replay()
    eager = sige.sige_qlinear(A, W, None, torch.zeros_like(ref), **where)
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    assert sige.sige_get_error(ws) == sige.OK


def test_binding_refusals_on_the_gpu():
    rng = np.random.default_rng(0)
    a, sa, wt, sw = operands(rng, 1, 4, 4, 64, 16)
    A, W = cache(a, sa), cache(wt, sw)
    with pytest.raises(ValueError, match="residual"):
        sige.sige_qlinear(A, W, residual=torch.zeros((1, 4, 4, 16), device=DEV))
    with pytest.raises(ValueError, match="different devices|CUDA"):
        sige.sige_qlinear(A, sige.QCache(W.codes.cpu(), W.scales.cpu(), "s8"))
    with pytest.raises(ValueError, match="fit"):
        sige.sige_qlinear(A, W, None, torch.zeros((1, 4, 4, 17), device=DEV))
    grouped = sige.QCache(A.codes, torch.ones((1, 4, 4, 2), device=DEV), "s8")
    with pytest.raises(sige.SigeError, match="unsupported"):
        sige.sige_qlinear(grouped, W)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("co", [1, 8, 15, 22, 40, 100, 333, 1000])
@pytest.mark.parametrize("n,h,w,c", [(1, 9, 15, 64), (2, 31, 33, 336), (1, 1, 3, 5120)])
def test_output_widths(n, h, w, c, co, dtype):
    """Channels that are no whole sectors, at every access width, whole maps and
    lists, with K split and without."""
    run_case(c + co, n, h, w, c, co, dtype, residual=True)
    rng = np.random.default_rng(c + co)
    a, sa, wt, sw = operands(rng, n, h, w, c, co)
    A, W = cache(a, sa), cache(wt, sw)
    full = sige.sige_qlinear(A, W, dtype=dtype)
    _, where = tile_list(rng, h, w, 4, 0.5)
    y = torch.full_like(full, 3.0)
    sige.sige_qlinear(A, W, None, y, **where)
    idx = where["idx"][:int(where["count"])].tolist()
    hit = torch.zeros((h, w), dtype=torch.bool, device=DEV)
    for i, j in idx:
        hit[i:i + 4, j:j + 4] = True
    assert torch.equal(y[:, hit], full[:, hit]) and (y[:, ~hit] == 3).all()


@pytest.mark.parametrize("n,h,w,c,co", [(1, 3, 5, 5121, 40), (1, 20, 20, 1025, 130), (2, 33, 31, 127, 300), (1, 12, 11, 129, 64),
                                        (1, 64, 64, 100, 1000), (1, 2, 2, 8190, 9)])
def test_channels_staged_by_threads(n, h, w, c, co):
    """Channels that are not a multiple of 16: last chunks of one byte, of all but
    one, more chunks than stages, more units than CTAs."""
    run_case(c, n, h, w, c, co, torch.bfloat16, residual=True)


@pytest.mark.parametrize("c", [64, 257, 1282])
@pytest.mark.parametrize("ao,wo", [(1, 2), (3, 0), (4, 7), (0, 13)])
def test_codes_at_any_byte(c, ao, wo):
    rng = np.random.default_rng(c + ao)
    n, h, w, co = 1, 5, 7, 70
    a, sa, wt, sw = operands(rng, n, h, w, c, co)
    def at(x, off):
        buf = torch.full((x.size + off + 16,), 77, dtype=torch.int8, device=DEV)
        v = buf[off:off + x.size].view(x.shape)
        v.copy_(torch.from_numpy(x))
        return v
    A = sige.QCache(at(a, ao), torch.from_numpy(sa).to(DEV), "s8")
    W = sige.QCache(at(wt, wo), torch.from_numpy(sw).to(DEV), "s8")
    y = sige.sige_qlinear(A, W, dtype=torch.float32)
    torch.cuda.synchronize()
    check(y, a, sa, wt, sw, None, None, torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,h,w,c,co", [(1, 16, 16, 320, 320), (1, 1, 3, 1280, 64), (1, 9, 15, 64, 51), (1, 13, 11, 74, 40)])
def test_scales_at_the_ends_of_the_range(n, h, w, c, co, dtype):
    """Token scales up to 2^119 and channel scales down to 2^-126, the other way
    round, and ordinary tokens beside them: finite wherever the value is."""
    rng = np.random.default_rng(c)
    a, sa, wt, sw = operands(rng, n, h, w, c, co)
    ends = np.ldexp(1.0 + rng.random(sa.shape), rng.choice([-126, -40, 0, 60, 97, 110, 118], sa.shape)).astype(np.float32)
    for lo, hi in ((-126, -110), (-100, -60), (-30, 0)):
        tok = np.where(rng.random(sa.shape) < 0.7, np.minimum(ends, np.float32(2.0 ** (124 - 24 - hi) if hi > -24 else 3e38)), sa)
        ch = np.ldexp(1.0 + rng.random(sw.shape), rng.integers(lo, hi, sw.shape)).astype(np.float32)
        for x, y in ((tok.astype(np.float32), ch),
                     (np.ldexp(1.0 + rng.random(sa.shape), rng.integers(lo, hi, sa.shape)).astype(np.float32),
                      np.resize(tok, sw.shape).astype(np.float32))):
            res = torch.from_numpy(rng.normal(size=(n, h, w, co))).to(dtype)
            got = sige.sige_qlinear(cache(a, x), cache(wt, y), residual=res.to(DEV), dtype=dtype)
            torch.cuda.synchronize()
            ref = oq.qlinear(a.reshape(-1, c), x.reshape(-1), wt.reshape(co, c), y.reshape(-1))
            assert np.abs(ref).max() < 2.0 ** 127 and torch.isfinite(got).all()
            check(got, a, x, wt, y, None, res, dtype)
