"""Attention over quantised key / value caches on the GPU against its oracle,
and the whole layer in codes.

Bound of an output element, with p the exact weights and V the values the codes
stand for: the tensor-core kernel rounds each weight times its value's scale to
bf16 (2^-8 relative), the scores are float32 sums of dh products (dh + 4
roundings of 2^-24 of the terms' magnitudes, which the exponential turns into a
relative error of the weights, in numerator and denominator), the exponential is
good to 2^-22, the sums over the keys to keys * 2^-24, and the result is rounded
to bf16 (2^-8 relative).
"""
import numpy as np
import pytest
import torch

import spatially_sparse_incremental_b200 as sige
from helpers import bits
from oracle import qcache as oq
from test_gpu_qcache import random_cache, tile_list

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bound(q, k, ref, ref_abs, heads, keys):
    T, D = q.shape
    dh, dvh = D // heads, ref.shape[1] // heads
    out = np.empty_like(ref)
    for h in range(heads):
        a, b = slice(h * dh, (h + 1) * dh), slice(h * dvh, (h + 1) * dvh)
        terms = (np.abs(q[:, a]) @ np.abs(k[:, a]).T).max(-1, keepdims=True) / np.sqrt(dh)
        e = terms * (dh + 4) * 2.0 ** -24
        out[:, b] = ref_abs[:, b] * (2.0 ** -8 + 2 * (e + 2.0 ** -22) + 2 * keys * 2.0 ** -24)
    return out * 1.001 + np.abs(ref) * 2.0 ** -8 + 1e-30


def compare(o, q, k, v, heads, tok, counts=None):
    """o [N, T, Dv] at the tokens of q [N, HW, D] float64."""
    for i in range(q.shape[0]):
        c = None if counts is None else counts[i]
        ref, ref_abs = oq.attention(q[i][tok], k[i], v[i], heads, c)
        L = k.shape[1] if c is None else max(0, min(c, k.shape[1]))
        got = o[i].double().numpy()
        if L == 0:
            assert not got.any()
            continue
        allow = bound(q[i][tok], k[i][:L], ref, ref_abs, heads, L)
        d = np.abs(got - ref)
        assert (d <= allow).all(), f"item {i}: max |d| / bound = {(d / allow).max():.3g}"


def case(seed, n, h, w, heads, dh, dvh, keys, kf, vf, b=None, frac=0.3, counts=None, token_scale=False, qscale=1.0):
    rng = np.random.default_rng(seed)
    D, Dv = heads * dh, heads * dvh
    q = torch.from_numpy(rng.normal(0, qscale, size=(n, h, w, D))).to(torch.bfloat16)
    K, kq, ksc = random_cache(rng, n, keys, 1, D, D if token_scale else dh, kf)
    V, vq, vsc = random_cache(rng, n, keys, 1, Dv, Dv if token_scale else dvh, vf)
    idx, where = (None, {}) if b is None else tile_list(rng, h, w, b, frac)
    o0 = torch.from_numpy(rng.normal(size=(n, h, w, Dv))).to(torch.bfloat16)
    o = o0.to(DEV)
    kc = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV)
    ws = sige.zeros_workspace(256, DEV)
    sige.sige_attention_qcache(q.to(DEV), K, V, heads, o, key_counts=kc, workspace=ws, **where)
    torch.cuda.synchronize()
    assert sige.sige_get_error(ws) == sige.OK
    tok = oq.tokens(idx, b or 1, h, w)
    rest = np.setdiff1d(np.arange(h * w), tok)
    got = o.cpu().view(n, h * w, Dv)
    assert torch.equal(bits(got[:, rest]), bits(o0.view(n, h * w, Dv)[:, rest]))
    compare(got[:, tok], oq.f64(q).reshape(n, h * w, D), oq.values(kq, ksc)[:, :, 0], oq.values(vq, vsc)[:, :, 0], heads, tok,
            counts)
    return o


@pytest.mark.parametrize("kf,vf", [("s8", "s8"), ("e4m3", "e4m3"), ("s4", "s4"), ("s8", "e4m3"), ("s4", "s8")])
@pytest.mark.parametrize("n,h,w,heads,dh,dvh,keys,b", [
    (1, 16, 16, 8, 40, 40, 256, 4), (1, 16, 16, 1, 64, 64, 256, 2), (2, 12, 12, 2, 80, 80, 77, 4), (1, 13, 11, 2, 64, 32, 143, 4),
    (1, 9, 7, 4, 8, 8, 63, 1), (1, 8, 8, 2, 128, 128, 300, 8), (1, 8, 8, 1, 160, 160, 130, 4), (1, 5, 5, 3, 30, 10, 50, 4),
    (1, 7, 7, 1, 256, 256, 40, 4), (2, 16, 16, 2, 32, 32, 1, 4),
])
def test_formats_and_heads(n, h, w, heads, dh, dvh, keys, b, kf, vf):
    case(dh + keys, n, h, w, heads, dh, dvh, keys, kf, vf, b)


@pytest.mark.parametrize("fmt", ["s8", "e4m3", "s4"])
@pytest.mark.parametrize("n,h,w,heads,dh,keys,b,frac", [
    (1, 64, 64, 8, 40, 4096, 4, 0.02), (1, 64, 64, 8, 40, 4096, 4, 0.15), (2, 32, 32, 2, 64, 1024, 8, 0.05), (1, 48, 40, 8, 8, 1920, 2, 0.03),
    (1, 20, 20, 2, 80, 2000, 2, 0.1), (1, 16, 16, 2, 160, 1025, 1, 0.1),
])
def test_long_keys(n, h, w, heads, dh, keys, b, frac, fmt):
    case(h + dh, n, h, w, heads, dh, dh, keys, fmt, fmt, b, frac)


@pytest.mark.parametrize("dh", [40, 80, 30])
def test_every_token_without_a_list(dh):
    case(1, 2, 24, 24, 4, dh, dh, 576, "s8", "s8")
    case(2, 1, 1, 1, 4, dh, dh, 200, "e4m3", "e4m3")
    case(3, 1, 13, 11, 1, dh, dh, 129, "s4", "s8")


def test_several_blocks_for_each_cta():
    case(5, 2, 48, 48, 8, 40, 40, 300, "s8", "s8")


@pytest.mark.parametrize("dh", [40, 80, 30])
def test_key_counts(dh):
    """A padded batch: no keys, one, a part, all, more than there are, fewer than none."""
    case(7, 6, 10, 10, 2, dh, dh, 150, "s8", "e4m3", 4, counts=[0, 1, 77, 150, 1000, -5])
    case(8, 4, 12, 12, 2, dh, dh, 1030, "s8", "s8", 2, frac=0.05, counts=[0, 1030, 513, 128])


@pytest.mark.parametrize("dh", [64, 30])
def test_padding_may_hold_anything(dh):
    """Keys and values past the count with NaN scales change nothing."""
    rng = np.random.default_rng(4)
    q = torch.from_numpy(rng.normal(size=(1, 8, 8, 2 * dh))).to(torch.bfloat16).to(DEV)
    K, _, _ = random_cache(rng, 1, 200, 1, 2 * dh, dh, "s8")
    V, _, _ = random_cache(rng, 1, 200, 1, 2 * dh, dh, "e4m3")
    kc = torch.tensor([141], dtype=torch.int32, device=DEV)
    ref = sige.sige_attention_qcache(q, K, V, 2, key_counts=kc)
    K.scales[:, 141:] = float("nan")
    V.scales[:, 141:] = float("inf")
    V.codes.view(torch.uint8)[:, 141:] = 0x7F      # the format's NaN
    assert torch.equal(sige.sige_attention_qcache(q, K, V, 2, key_counts=kc), ref)
    assert torch.isfinite(ref).all()


@pytest.mark.parametrize("dh", [64, 80, 30])
def test_a_poisoned_key_poisons_the_row(dh):
    rng = np.random.default_rng(6)
    q = torch.from_numpy(rng.normal(size=(2, 4, 4, dh))).to(torch.bfloat16).to(DEV)
    K, _, _ = random_cache(rng, 2, 300, 1, dh, dh, "s8")
    V, _, _ = random_cache(rng, 2, 300, 1, dh, dh, "s8")
    K.scales[1, 200] = float("nan")
    o = sige.sige_attention_qcache(q, K, V, 1)
    assert torch.isnan(o[1]).all() and torch.isfinite(o[0]).all()


@pytest.mark.parametrize("dh", [64, 128, 30])
def test_growing_and_large_scores(dh):
    """Scores that rise along the keys by far more than 2^8 and a large common
    offset move the running maximum chunk after chunk."""
    case(9, 1, 8, 8, 1, dh, dh, 1500, "s8", "s8", 4, qscale=30.0)
    rng = np.random.default_rng(10)
    u = rng.normal(size=dh)
    u /= np.linalg.norm(u)
    q = torch.from_numpy(4 * u + 0.3 * rng.normal(size=(1, 4, 4, dh))).to(torch.bfloat16)
    kv = (np.linspace(-50, 110, 1200)[:, None] * u + 0.3 * rng.normal(size=(1200, dh))).astype(np.float32)[None, :, None]
    kq, ks = oq.quantise(kv, dh, "s8")
    K = sige.QCache(torch.from_numpy(oq.stored(kq, "s8")).view(torch.int8).to(DEV), torch.from_numpy(ks).to(DEV), "s8")
    V, vq, vs = random_cache(rng, 1, 1200, 1, dh, dh, "s8")
    o = sige.sige_attention_qcache(q.to(DEV), K, V, 1)
    compare(o.cpu().view(1, 16, dh), oq.f64(q).reshape(1, 16, dh), oq.values(kq, ks)[:, :, 0], oq.values(vq, vs)[:, :, 0], 1,
            np.arange(16))


def test_one_scale_per_token():
    case(11, 1, 16, 16, 4, 40, 40, 256, "s8", "s8", 4, token_scale=True)
    case(12, 1, 8, 8, 2, 30, 30, 64, "s8", "s8", 4, token_scale=True)


@pytest.mark.parametrize("dh", [40, 30])
def test_lists_that_are_short_long_or_out_of_the_map(dh):
    rng = np.random.default_rng(14)
    n, h, w = 2, 10, 10
    q = torch.from_numpy(rng.normal(size=(n, h, w, dh))).to(torch.bfloat16).to(DEV)
    K, _, _ = random_cache(rng, n, 100, 1, dh, dh, "s8")
    V, _, _ = random_cache(rng, n, 100, 1, dh, dh, "s8")
    full = sige.sige_attention_qcache(q, K, V, 1).float()
    tiles = torch.tensor([[4, 4], [4, 4], [8, 8], [-4, 0], [0, -1], [12, 0], [0, 400], [0, 0]], dtype=torch.int32, device=DEV)
    for count, cap, listed in ((0, 8, []), (-3, 8, []), (99, 3, [(4, 4), (8, 8)]), (8, 8, [(4, 4), (8, 8), (0, 0)])):
        o = torch.full((n, h, w, dh), 3.0, dtype=torch.bfloat16, device=DEV)
        sige.sige_attention_qcache(q, K, V, 1, o, idx=tiles, capacity=cap, block=4,
                                   count=torch.tensor([count], dtype=torch.int32, device=DEV))
        hit = torch.zeros((h, w), dtype=torch.bool, device=DEV)
        for i, j in listed:
            hit[i:i + 4, j:j + 4] = True
        # the split of the keys may differ between the two calls: two roundings of the weights
        assert torch.allclose(o[:, hit].float(), full[:, hit], rtol=2.0 ** -6, atol=2.0 ** -7 * float(full.abs().max()))
        assert (o[:, ~hit] == 3).all()


@pytest.mark.parametrize("dh", [40, 100])
def test_unaligned_operands(dh):
    rng = np.random.default_rng(15)
    q = torch.from_numpy(rng.normal(size=(1, 6, 6, dh))).to(torch.bfloat16)
    K, kq, ks = random_cache(rng, 1, 90, 1, dh, dh, "s8")
    V, vq, vs = random_cache(rng, 1, 90, 1, dh, dh, "e4m3")

    def off(t, k):
        buf = torch.empty(t.numel() + k, dtype=t.dtype, device=DEV)
        buf[k:].copy_(t.reshape(-1))
        return buf[k:].view(t.shape)

    for a, b, c, d in ((1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (4, 8, 4, 4)):
        o = off(torch.zeros((1, 6, 6, dh), dtype=torch.bfloat16, device=DEV), d)
        sige.sige_attention_qcache(off(q.to(DEV), a), sige.QCache(off(K.codes, b), off(K.scales, b), "s8"),
                                   sige.QCache(off(V.codes, c), off(V.scales, c), "e4m3"), 1, o)
        compare(o.cpu().view(1, 36, dh), oq.f64(q).reshape(1, 36, dh), oq.values(kq, ks)[:, :, 0],
                oq.values(vq, vs)[:, :, 0], 1, np.arange(36))


def test_streams_and_graphs():
    rng = np.random.default_rng(16)
    q = torch.from_numpy(rng.normal(size=(1, 32, 32, 320))).to(torch.bfloat16).to(DEV)
    K, _, _ = random_cache(rng, 1, 1024, 1, 320, 40, "s8")
    V, _, _ = random_cache(rng, 1, 1024, 1, 320, 40, "e4m3")
    _, where = tile_list(rng, 32, 32, 4, 0.1)
    ref = sige.sige_attention_qcache(q, K, V, 8)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [sige.sige_attention_qcache(q, K, V, 8, stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    out, ws = torch.zeros_like(ref), sige.zeros_workspace(256, DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sige.sige_attention_qcache(q, K, V, 8, out, workspace=ws, **where)
    q.copy_(torch.from_numpy(rng.normal(size=(1, 32, 32, 320))).to(torch.bfloat16))
    graph.replay()
    eager = sige.sige_attention_qcache(q, K, V, 8, torch.zeros_like(ref), **where)
    torch.cuda.synchronize()
    assert torch.equal(out, eager)


# ------------------------------------------------------------------ the layer

@pytest.mark.parametrize("cross,kf,heads,C", [(False, "s8", 8, 320), (False, "e4m3", 2, 128), (True, "s4", 4, 64), (False, "s8", 3, 90)])
def test_layer_runs_its_steps(cross, kf, heads, C):
    """sige_attention_sparse_q equals its steps called one by one, bit for bit;
    each step is held to its oracle, given the step before."""
    rng = np.random.default_rng(C)
    n, h, w, b, keys = 2, 16, 16, 4, 77
    dh = C // heads
    idx, where = tile_list(rng, h, w, b, 0.2)
    x = torch.from_numpy(rng.normal(size=(n, h, w, C))).to(torch.bfloat16).to(DEV)
    weights = [sige.sige_qcache_write(torch.from_numpy(rng.normal(0, C ** -0.5, size=(C, 1, 1, C)).astype(np.float32)).to(DEV),
                                      sige.qcache_empty(C, 1, 1, C)) for _ in range(4)]
    wq, wk, wv, wo = weights
    bo = torch.from_numpy(rng.normal(size=C).astype(np.float32)).to(DEV)
    shape = (n, keys, 1, C) if cross else (n, h, w, C)
    K0, _, _ = random_cache(rng, *shape, dh, kf)
    V0, _, _ = random_cache(rng, *shape, dh, kf)
    clone = lambda c: sige.QCache(c.codes.clone(), c.scales.clone(), c.format)
    y0 = torch.from_numpy(rng.normal(size=(n, h, w, C))).to(torch.bfloat16).to(DEV)
    kc = torch.tensor([keys, 13], dtype=torch.int32, device=DEV) if cross else None
    K, V, y = clone(K0), clone(V0), y0.clone()
    sige.sige_attention_sparse_q(x, where["idx"], where["count"], where["capacity"], b, wq, wo, bo, heads, K, V, y,
                                 wk=None if cross else wk, wv=None if cross else wv, residual=x, key_counts=kc)
    # the steps
    K1, V1, y1 = clone(K0), clone(V0), y0.clone()
    xq = sige.sige_qcache_write(x, sige.qcache_empty(n, h, w, C), **where)
    q = sige.sige_qlinear(xq, wq, **where)
    if not cross:
        for wt, c in ((wk, K1), (wv, V1)):
            sige.sige_qcache_write(sige.sige_qlinear(xq, wt, **where), c, **where)
    o = sige.sige_attention_qcache(q, K1, V1, heads, key_counts=kc, **where)
    oqc = sige.sige_qcache_write(o, sige.qcache_empty(n, h, w, C), **where)
    sige.sige_qlinear(oqc, wo, bo, y1, residual=x, **where)
    torch.cuda.synchronize()
    assert torch.equal(y, y1)
    assert torch.equal(K.codes.view(torch.uint8), K1.codes.view(torch.uint8)) and torch.equal(V.scales, V1.scales)
    tok = oq.tokens(idx, b, h, w)
    rest = np.setdiff1d(np.arange(h * w), tok)
    flat = lambda t: t.cpu().view(n, h * w, -1)
    assert torch.equal(flat(y)[:, rest], flat(y0)[:, rest])
    assert torch.equal(flat(K.codes.view(torch.uint8))[:, rest] if not cross else flat(x)[:, rest],
                       flat(K0.codes.view(torch.uint8))[:, rest] if not cross else flat(x)[:, rest])
    # every step against the oracle, from the tensors the step before left
    def vals(c):
        return oq.f64(sige.sige_qcache_read(c, dtype=torch.float32)).reshape(n, -1, C)
    xs, ss = oq.quantise(oq.f64(x).reshape(n, h * w, C)[:, tok], C, "s8")
    assert np.array_equal(xq.codes.cpu().numpy().reshape(n, h * w, C)[:, tok], xs)
    assert np.array_equal(xq.scales.cpu().numpy().reshape(n, h * w, 1)[:, tok], ss)
    W = lambda c: oq.f64(c.codes).reshape(C, C) * oq.f64(c.scales).reshape(C, 1)
    qref = (xs * ss.astype(np.float64)) @ W(wq).T
    assert (np.abs(oq.f64(q).reshape(n, h * w, C)[:, tok] - qref) <= np.abs(qref) * (2.0 ** -8 + 2.0 ** -21)).all()
    compare(flat(o)[:, tok], oq.f64(q).reshape(n, h * w, C), vals(K1), vals(V1), heads, tok,
            None if kc is None else kc.tolist())
    os_, osc = oq.quantise(oq.f64(o).reshape(n, h * w, C)[:, tok], C, "s8")
    yref = (os_ * osc.astype(np.float64)) @ W(wo).T + oq.f64(bo) + oq.f64(x).reshape(n, h * w, C)[:, tok]
    mag = np.abs((os_ * osc.astype(np.float64)) @ W(wo).T) + np.abs(oq.f64(bo)) + np.abs(oq.f64(x).reshape(n, h * w, C)[:, tok])
    assert (np.abs(oq.f64(y).reshape(n, h * w, C)[:, tok] - yref) <= np.abs(yref) * 2.0 ** -8 * 1.0001 + mag * 2.0 ** -21).all()


@pytest.mark.parametrize("kf,vf", [("s8", "e4m3"), ("e4m3", "s8"), ("s4", "s4")])
@pytest.mark.parametrize("dh,dvh", [(192, 192), (184, 136), (136, 40), (24, 192), (100, 100), (12, 20), (190, 2), (66, 130), (254, 200)])
def test_head_widths(dh, dvh, kf, vf):
    """Every width class, aligned or not, with one block of queries for a unit and
    with the keys split."""
    case(dh, 2, 9, 10, 2, dh, dvh, 143, kf, vf, 4)
    case(dvh, 1, 6, 6, 1, dh, dvh, 1111, kf, vf, 2)


@pytest.mark.parametrize("dh,dvh", [(1, 1), (3, 5), (37, 37), (129, 63), (191, 33)])
def test_odd_head_widths(dh, dvh):
    case(dh, 2, 9, 10, 3, dh, dvh, 143, "s8", "e4m3", 4)
    case(dvh, 1, 6, 6, 1, dh, dvh, 1111, "e4m3", "s8", 2)
    # 4-bit codes of odd heads begin at odd halves of a byte
    case(dh + 1, 1, 7, 9, 4, dh, dvh, 150, "s4", "s4", 4, token_scale=True)


@pytest.mark.parametrize("dh", [100, 136, 192])
def test_two_blocks_a_unit_of_wide_heads(dh):
    case(dh, 2, 48, 47, 8, dh, dh, 200, "s8", "s8", counts=[200, 65])


@pytest.mark.parametrize("kf,vf", [("s8", "s8"), ("e4m3", "s4")])
@pytest.mark.parametrize("dh", [16, 40, 100, 128, 160])
@pytest.mark.parametrize("keys,counts", [(1, None), (2, [2, 1]), (32, [32, 17]), (150, [31, 32]), (4096, [3, 32])])
def test_short_items_keep_their_weights(dh, keys, counts, kf, vf):
    """Up to 32 keys: weights in two bf16 terms, 2^-17 (twice half a step, once for
    the first term's remainder) in the place of one term's 2^-8; the rest as bound()."""
    rng = np.random.default_rng(dh + keys)
    n, h, w, heads = 2, 9, 8, 2
    q = torch.from_numpy(rng.normal(size=(n, h, w, heads * dh))).to(torch.bfloat16)
    K, kq, ks = random_cache(rng, n, keys, 1, heads * dh, dh, kf)
    V, vq, vs = random_cache(rng, n, keys, 1, heads * dh, dh, vf)
    kc = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV)
    o = sige.sige_attention_qcache(q.to(DEV), K, V, heads, key_counts=kc)
    o = o.double().cpu().numpy().reshape(n, h * w, -1)
    k = (kq.reshape(*ks.shape, -1).astype(np.float64) * ks[..., None]).reshape(n, keys, -1)
    v = (vq.reshape(*vs.shape, -1).astype(np.float64) * vs[..., None]).reshape(n, keys, -1)
    qd = q.double().numpy().reshape(n, h * w, -1)
    for i in range(n):
        L = keys if counts is None else counts[i]
        ref, ref_abs = oq.attention(qd[i], k[i], v[i], heads, L)
        allow = bound(qd[i], k[i][:L], ref, ref_abs, heads, L) - ref_abs * (2.0 ** -8 - 2.0 ** -17)
        assert (np.abs(o[i] - ref) <= allow).all()


def test_two_graphs_share_a_workspace():
    """The layer captured twice with one workspace and replayed on two streams at
    once: each replay gives the eager call's bits."""
    rng = np.random.default_rng(44)
    n, h, w, C, heads, b = 1, 32, 32, 320, 8, 4
    weights = [sige.sige_qcache_write(torch.from_numpy(rng.normal(0, C ** -0.5, size=(C, 1, 1, C)).astype(np.float32)).to(DEV),
                                      sige.qcache_empty(C, 1, 1, C)) for _ in range(4)]
    wq, wk, wv, wo = weights
    ws = sige.zeros_workspace(256, DEV)
    runs = []
    for frac in (0.1, 0.5):
        _, where = tile_list(rng, h, w, b, frac)
        x = torch.from_numpy(rng.normal(size=(n, h, w, C))).to(torch.bfloat16).to(DEV)
        kv = [random_cache(rng, n, h, w, C, C // heads, "s8")[0] for _ in range(2)]
        y = torch.zeros_like(x)
        call = lambda x=x, where=where, kv=kv, y=y: sige.sige_attention_sparse_q(
            x, where["idx"], where["count"], where["capacity"], b, wq, wo, None, heads, *kv, y, wk=wk, wv=wv, workspace=ws)
        call()
        torch.cuda.synchronize()
        want = y.clone()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, stream, y, want, call))   # (the call keeps the graph's inputs alive)
    for _ in range(20):
        for graph, stream, y, _, _ in runs:
            with torch.cuda.stream(stream):
                y.zero_()
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for _, _, y, want, _ in runs)
    assert not ws.any()


@pytest.mark.parametrize("fmt", ["s8", "e4m3"])
@pytest.mark.parametrize("dh", [40, 80, 160, 30, 200])
def test_large_values(dh, fmt):
    """Finite values give finite results, however large: at even weights (a sum of
    as many weights as there are keys), where the scores rise along the keys (an
    exponent base of the first ones lies 2^35 below the maximum), where only some
    keys' values are large, and for the few keys of a short item."""
    rng = np.random.default_rng(dh)
    u = rng.normal(size=dh)
    u /= np.linalg.norm(u)
    # (ends of the scores, in base 2: 0 and `rise`, whatever the width)
    for keys, rise, top, mixed in ((1200, 0, 2.0 ** 123, False), (1200, 35, 2.0 ** 100, False), (1200, 35, 2.0 ** 90, True),
                                   (1200, -35, 2.0 ** 100, True), (20, 3, 2.0 ** 125, False)):
        q = torch.from_numpy(u + 0.01 * rng.normal(size=(1, 4, 5, dh))).to(torch.bfloat16)
        kv = (np.linspace(0, rise * np.log(2) * np.sqrt(dh), keys)[:, None] * u + 0.01 * rng.normal(size=(keys, dh)))
        kq, ks = oq.quantise(kv.astype(np.float32)[None, :, None], dh, fmt)
        vv = top * (1 + rng.random(size=(keys, dh)))
        if mixed:
            vv[rng.random(keys) < 0.7] *= 2.0 ** -90
        vq, vs = oq.quantise(vv.astype(np.float32)[None, :, None], dh, fmt)
        store = {"s8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt]
        K = sige.QCache(torch.from_numpy(oq.stored(kq, fmt)).view(store).to(DEV), torch.from_numpy(ks).to(DEV), fmt)
        V = sige.QCache(torch.from_numpy(oq.stored(vq, fmt)).view(store).to(DEV), torch.from_numpy(vs).to(DEV), fmt)
        o = sige.sige_attention_qcache(q.to(DEV), K, V, 1)
        assert torch.isfinite(o).all(), (keys, rise, top, mixed)
        compare(o.cpu().view(1, 20, dh), oq.f64(q).reshape(1, 20, dh), oq.values(kq, ks)[:, :, 0], oq.values(vq, vs)[:, :, 0], 1,
                np.arange(20))


@pytest.mark.parametrize("n,h,w,heads,dh,keys,counts", [
    (32, 8, 8, 8, 40, 260, None), (25, 8, 16, 8, 40, 129, None), (20, 8, 8, 8, 80, 200, None), (19, 5, 5, 8, 30, 150, None),
    (12, 24, 16, 8, 40, 300, None), (9, 24, 16, 8, 40, 300, None), (10, 19, 17, 8, 100, 70, None), (150, 3, 3, 1, 160, 90, None),
    (40, 4, 4, 4, 40, 200, "ragged"), (23, 24, 13, 4, 80, 140, "ragged"),
])
def test_more_units_than_ctas(n, h, w, heads, dh, keys, counts):
    """One, two or three blocks of queries an item and more of them than the launch
    has CTAs: alone or two to a unit."""
    counts = None if counts is None else [(37 * i) % (keys + 1) for i in range(n)]
    case(n + dh, n, h, w, heads, dh, dh, keys, "s8", "e4m3", counts=counts)


def test_a_refused_layer_changes_nothing():
    """Whatever step would refuse: the caches and the output keep their bytes."""
    rng = np.random.default_rng(3)
    n, h, w, C, heads, b = 1, 8, 8, 64, 2, 4
    q8 = lambda co, ci: sige.sige_qcache_write(torch.from_numpy(rng.normal(size=(co, 1, 1, ci)).astype(np.float32)).to(DEV),
                                               sige.qcache_empty(co, 1, 1, ci))
    _, where = tile_list(rng, h, w, b, 0.5)
    x = torch.from_numpy(rng.normal(size=(n, h, w, C))).to(torch.bfloat16).to(DEV)
    K, V = (random_cache(rng, n, h, w, C, C // heads, "s8")[0] for _ in range(2))
    y = torch.from_numpy(rng.normal(size=(n, h, w, C))).to(torch.bfloat16).to(DEV)
    good = dict(x=x, **where, wq=q8(C, C), wo=q8(C, C), bo=None, heads=heads, k_map=K, v_map=V, y=y, wk=q8(C, C), wv=q8(C, C))
    state = lambda: [t.clone() for t in (K.codes, K.scales, V.codes, V.scales, y)]
    before = state()
    grouped = sige.QCache(good["wo"].codes, torch.ones((C, 1, 1, 2), device=DEV), "s8")
    for bad in (dict(wv=q8(C, 32)), dict(wv=q8(32, C)), dict(wo=q8(C, 32)), dict(wo=grouped), dict(wo=q8(48, C)), dict(heads=3), dict(heads=0),
                dict(heads=4096), dict(y=y[:, :4]), dict(y=y.float().double()), dict(residual=x.float()), dict(residual=y), dict(bo=torch.ones(3, device=DEV)),
                dict(key_counts=torch.ones(2, dtype=torch.int32, device=DEV)), dict(v_map=K), dict(v_map=random_cache(rng, n, 4, w, C, 32, "s8")[0]),
                dict(v_map=random_cache(rng, n, h, w, C, 16, "s8")[0]), dict(k_map=random_cache(rng, n, h, w, C, 8, "e4m3")[0]),
                dict(workspace=torch.zeros(64, dtype=torch.uint8, device=DEV)), dict(wq=q8(32, C)), dict(block=65), dict(bo=torch.ones(C)),
                dict(count=None), dict(capacity=10 ** 6), dict(capacity=-1)):
        with pytest.raises((ValueError, sige.SigeError)):
            sige.sige_attention_sparse_q(**{**good, **bad})
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(before, state())), bad
    sige.sige_attention_sparse_q(**good)
    torch.cuda.synchronize()
    assert not any(torch.equal(a, c) for a, c in zip(before, state()))


@pytest.mark.parametrize("cross,kf,vf", [(False, "s8", "e4m3"), (False, "s4", "s8"), (True, "s8", "s4"), (True, "e4m3", "e4m3")])
def test_layer_and_its_caches(cross, kf, vf):
    """The context's caches keep every byte; those of a self-attention get, at the
    listed tokens, what quantising the projections there gives, codes and scales,
    and keep the rest."""
    rng = np.random.default_rng(21)
    n, h, w, C, heads, b = 2, 10, 9, 64, 4, 4
    idx, where = tile_list(rng, h, w, b, 0.3)
    x = torch.from_numpy(rng.normal(size=(n, h, w, C))).to(torch.bfloat16).to(DEV)
    wq, wk, wv, wo = (sige.sige_qcache_write(torch.from_numpy(rng.normal(0, C ** -0.5, size=(C, 1, 1, C)).astype(np.float32)).to(DEV),
                                             sige.qcache_empty(C, 1, 1, C)) for _ in range(4))
    shape = (n, 31, 1, C) if cross else (n, h, w, C)
    K, V = (random_cache(rng, *shape, C // heads, f)[0] for f in (kf, vf))
    raw = lambda c: (c.codes.view(torch.uint8).cpu().clone(), c.scales.cpu().clone())
    K0, V0 = raw(K), raw(V)
    y = torch.zeros((n, h, w, C), dtype=torch.bfloat16, device=DEV)
    sige.sige_attention_sparse_q(x, where["idx"], where["count"], where["capacity"], b, wq, wo, None, heads, K, V, y,
                                 wk=None if cross else wk, wv=None if cross else wv)
    torch.cuda.synchronize()
    if cross:
        assert all(torch.equal(a, c) for a, c in zip((*K0, *V0), (*raw(K), *raw(V))))
        return
    tok = oq.tokens(idx, b, h, w)
    rest = np.setdiff1d(np.arange(h * w), tok)
    xq = sige.sige_qcache_write(x, sige.qcache_empty(n, h, w, C))
    for cache, before, wt, fmt in ((K, K0, wk, kf), (V, V0, wv, vf)):
        p = oq.f64(sige.sige_qlinear(xq, wt)).reshape(n, h * w, C)[:, tok]
        q, s = oq.quantise(p, C // heads, fmt)
        codes, scales = (t.view(n, h * w, -1).numpy() for t in raw(cache))
        want = oq.stored(q, fmt)
        got = codes[:, tok]
        if fmt == "e4m3":   # -0 and 0 are the same value
            got, want = np.where(got == 128, 0, got), np.where(want == 128, 0, want)
        assert np.array_equal(got, want) and np.array_equal(scales[:, tok], s)
        assert np.array_equal(codes[:, rest], before[0].view(n, h * w, -1).numpy()[:, rest])
        assert np.array_equal(scales[:, rest], before[1].view(n, h * w, -1).numpy()[:, rest])


@pytest.mark.parametrize("n,h,w,heads,dh,keys,counts", [(2, 48, 48, 8, 40, 700, None), (3, 32, 32, 8, 80, 77, [77, 0, 41]), (32, 8, 8, 8, 40, 300, None),
                                                        (1, 13, 12, 8, 160, 900, None)])
def test_whole_maps_repeat_their_bits(n, h, w, heads, dh, keys, counts):
    """Units of two blocks, of one, and split ones: the same bits again, on two
    streams at once and with other work in between."""
    rng = np.random.default_rng(n)
    q = torch.from_numpy(rng.normal(size=(n, h, w, heads * dh))).to(torch.bfloat16).to(DEV)
    K, V = (random_cache(rng, n, keys, 1, heads * dh, dh, f)[0] for f in ("s8", "e4m3"))
    kc = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV)
    ref = sige.sige_attention_qcache(q, K, V, heads, key_counts=kc)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(10):
        for s in streams:
            outs.append(sige.sige_attention_qcache(q, K, V, heads, key_counts=kc, stream=s))
            with torch.cuda.stream(s):
                torch.empty(1 << 22, device=DEV).normal_()
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
