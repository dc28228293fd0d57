"""The quantised cache, the product and the attention over the cache at the ends
of their ranges: the longest maps and offsets past 32 bits."""
import numpy as np
import pytest
import torch

import spatially_sparse_incremental_b200 as sige
from oracle import qcache as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"
MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def one_list(*tiles):
    return dict(idx=torch.tensor(tiles, dtype=torch.int32, device=DEV), capacity=len(tiles),
                count=torch.tensor([len(tiles)], dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("tall", [True, False])
@pytest.mark.parametrize("block", [4, 64])
def test_a_clipped_tile_at_the_end_of_the_longest_map(tall, block):
    """2^31 - 1 pixels in a row or a column: the last tile's rows (columns) past the
    map have numbers past 32 bits, and are left out like those of any tile."""
    at = MOST - 2
    shape = (1, MOST, 1, 1) if tall else (1, 1, MOST, 1)
    where = dict(one_list((at, 0) if tall else (0, at)), block=block)
    part = lambda t: t.view(-1)[at - 2:]
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    part(x).copy_(torch.tensor([1.0, 2.0, 3.0, -4.0]))
    cache = sige.qcache_empty(*shape)
    part(cache.codes).fill_(9)
    part(cache.scales).fill_(0.5)
    sige.sige_qcache_write(x, cache, **where)
    assert part(cache.codes).tolist() == [9, 9, 127, -127]
    assert part(cache.scales).tolist() == [0.5, 0.5, np.float32(3) / np.float32(127), np.float32(4) / np.float32(127)]
    y = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    part(y).fill_(7)
    sige.sige_qcache_read(cache, y, **where)
    assert part(y).tolist() == [7, 7, 3, -4]
    part(y).fill_(7)
    w = sige.QCache(torch.full((1, 1, 1, 1), 2, dtype=torch.int8, device=DEV), torch.ones((1, 1, 1, 1), device=DEV), "s8")
    sige.sige_qlinear(cache, w, None, y, **where)
    assert part(y).tolist() == [7, 7, 6, -8]
    del cache
    part(y).fill_(7)
    kv = sige.QCache(torch.full((1, 3, 1, 1), 100, dtype=torch.int8, device=DEV), torch.full((1, 3, 1, 1), 0.25, device=DEV), "s8")
    sige.sige_attention_qcache(x, kv, kv, 1, y, **where)
    assert part(y).tolist() == [7, 7, 25, 25]


@pytest.mark.parametrize("fmt", ["s8", "e4m3"])
def test_offsets_past_32_bits(fmt):
    """Codes of 4.3 GB and maps of 8.6 GB: the last pixels of the last item are
    written, read, multiplied and attended to as any others."""
    n, h, w, c = 3, 1024, 1100, 1296
    rng = np.random.default_rng(2)
    assert n * h * w * c > 2 ** 32
    x = torch.empty((n, h, w, c), dtype=torch.bfloat16, device=DEV)
    v = torch.from_numpy(rng.normal(size=(4, 4, c))).to(torch.bfloat16)
    x[2, h - 4:, w - 4:] = v.to(DEV)
    cache = sige.qcache_empty(n, h, w, c, fmt, group=648 if fmt == "e4m3" else None)
    where = dict(one_list((h - 4, w - 4)), block=4)
    sige.sige_qcache_write(x, cache, **where)
    q, s = oq.quantise(v.float().numpy(), cache.group, fmt)
    got = cache.codes[2, h - 4:, w - 4:].cpu().view(torch.uint8).numpy()
    want = oq.stored(q, fmt)
    if fmt == "e4m3":   # -0 and 0 are the same value
        got, want = np.where(got == 128, 0, got), np.where(want == 128, 0, want)
    assert np.array_equal(got, want) and np.array_equal(cache.scales[2, h - 4:, w - 4:].cpu().numpy(), s)
    x[2, h - 4:, w - 4:] = 0
    sige.sige_qcache_read(cache, x, **where)
    val = oq.values(q, s)
    back = x[2, h - 4:, w - 4:].double().cpu().numpy()
    assert (np.abs(back - val) <= np.abs(val) * (2.0 ** -8 + 2.0 ** -24)).all()
    if fmt == "s8":
        wt = sige.sige_qcache_write(torch.from_numpy(rng.normal(size=(8, 1, 1, c)).astype(np.float32)).to(DEV), sige.qcache_empty(8, 1, 1, c))
        y = sige.sige_qlinear(cache, wt, dtype=torch.float32, **where)[2, h - 4:, w - 4:].double().cpu().numpy()
        ref = oq.qlinear(q.reshape(16, c), s.reshape(16), oq.f64(wt.codes).reshape(8, c), oq.f64(wt.scales).reshape(8))
        assert (np.abs(y.reshape(16, 8) - ref) <= np.abs(ref) * 3.01 * 2.0 ** -24).all()
    # a query over the last 16 keys alone: the others' scores are kept far below by a zero key
    cache.codes.view(torch.uint8).zero_()
    cache.scales.fill_(1.0)
    sige.sige_qcache_write(x, cache, **where)
    qq = torch.zeros((n, 1, 1, c), dtype=torch.bfloat16, device=DEV)
    i = int(np.abs(val.reshape(16, c)[:, 0]).argmax())
    qq[2, 0, 0, :72] = 400 * torch.sign(x[2, h - 4 + i // 4, w - 4 + i % 4, :72])
    o = sige.sige_attention_qcache(qq, cache, cache, 18)[2, 0, 0, :72].double().cpu().numpy()
    q2, s2 = oq.quantise(back, cache.group, fmt)
    k = oq.values(q2, s2).reshape(16, c)[:, :72]
    ref, ref_abs = oq.attention(qq[2, 0, 0, :72].double().cpu().numpy()[None], k, k, 1)
    # (the weight rounded, the result rounded; 2^-10 for scores of 2^12 in float32, dh + 4
    # roundings of 2^-24 each; the zero keys' 1.1M weights are below e^-1000)
    assert (np.abs(o - ref[0]) <= np.abs(ref[0]) * 2.0 ** -8 + ref_abs[0] * (2.0 ** -8 + 2.0 ** -5)).all()


def test_a_list_without_places_is_no_pixel():
    """A tile list of shape [0, 2] (its tensor has no address) is an empty list, not
    every pixel."""
    rng = np.random.default_rng(8)
    draw = lambda *shape: torch.from_numpy(rng.normal(size=shape)).to(torch.bfloat16).to(DEV)
    n, h, w, c = 1, 8, 8, 32
    none = dict(idx=torch.empty((0, 2), dtype=torch.int32, device=DEV), count=torch.zeros(1, dtype=torch.int32, device=DEV), capacity=0,
                block=4)
    tail = dict(none, idx=torch.zeros((4, 2), dtype=torch.int32, device=DEV)[4:])
    wt = sige.sige_qcache_write(draw(c, 1, 1, c), sige.qcache_empty(c, 1, 1, c))
    K, V = (sige.sige_qcache_write(draw(n, h, w, c), sige.qcache_empty(n, h, w, c, group=16)) for _ in range(2))
    A = sige.sige_qcache_write(draw(n, h, w, c), sige.qcache_empty(n, h, w, c))
    x, y = draw(n, h, w, c), draw(n, h, w, c)
    kept = (K.codes, K.scales, V.codes, V.scales, A.codes, A.scales, y)
    before = [t.clone() for t in kept]
    launches = sige.sige_launch_count()
    for where in (none, tail):
        sige.sige_qcache_write(x, K, **where)
        sige.sige_qcache_read(K, y, **where)
        sige.sige_qlinear(A, wt, None, y, **where)
        sige.sige_attention_qcache(x, K, V, 2, y, **where)
        sige.sige_attention_sparse_q(x, where["idx"], where["count"], 0, 4, wt, wt, None, 2, K, V, y, wk=wt, wv=wt)
        with pytest.raises((ValueError, sige.SigeError)):
            sige.sige_qcache_write(x, K, **dict(where, capacity=1))
        with pytest.raises((ValueError, sige.SigeError)):
            sige.sige_qcache_write(x, K, **dict(where, block=0))
    torch.cuda.synchronize()
    assert sige.sige_launch_count() == launches
    assert all(torch.equal(a, b) for a, b in zip(kept, before))
