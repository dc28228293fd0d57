"""The quantised cache on the GPU against its oracle (oracle/qcache.py).

Codes and scales are compared bit for bit: the format defines them exactly (a
float32 scale, the exact quotient rounded with ties to even).  Reading back is
one float32 product (2^-24) and one rounding to the map's dtype.
"""
import numpy as np
import pytest
import torch

import spatially_sparse_incremental_b200 as sige
from helpers import bits
from oracle import qcache as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = ("s8", "e4m3", "s4")
DTYPES = (torch.bfloat16, torch.float32)


def tile_list(rng, H, W, b, frac=0.3):
    every = [(h, w) for h in range(0, H, b) for w in range(0, W, b)]
    keep = rng.random(len(every)) < frac
    keep[rng.integers(len(every))] = True
    idx = np.array([t for t, k in zip(every, keep) if k], dtype=np.int32)
    d = torch.zeros((len(every), 2), dtype=torch.int32)
    d[:len(idx)] = torch.from_numpy(idx)
    return idx, dict(idx=d.to(DEV), count=torch.tensor([len(idx)], dtype=torch.int32, device=DEV), capacity=len(every),
                     block=b)


def random_map(rng, n, h, w, c, dtype):
    x = rng.normal(size=(n, h, w, c)) * np.exp(rng.normal(size=c)) * np.exp(3 * rng.normal(size=(n, h, w, 1)))
    x[rng.random((n, h, w)) < 0.05] = 0
    return torch.from_numpy(x).to(dtype)


def random_cache(rng, n, h, w, c, group, fmt):
    """A cache of random normals: (device QCache, oracle code values, oracle scales)."""
    q, s = oq.quantise(rng.normal(size=(n, h, w, c)).astype(np.float32), group, fmt)
    codes = torch.from_numpy(oq.stored(q, fmt)).view(
        {"s8": torch.int8, "e4m3": torch.float8_e4m3fn, "s4": torch.uint8}[fmt])
    return sige.QCache(codes.to(DEV), torch.from_numpy(s).to(DEV), fmt), q, s


def byte_view(cache):
    return cache.codes.cpu().view(torch.uint8).numpy()



def check_write(x, group, fmt, idx=None, where=None, b=1, seed=0):
    rng = np.random.default_rng(seed)
    n, h, w, c = x.shape
    cache, _, _ = random_cache(rng, n, h, w, c, group, fmt)
    before, sbefore = byte_view(cache).copy(), cache.scales.cpu().numpy().copy()
    sige.sige_qcache_write(x.to(DEV), cache, **(where or {}))
    torch.cuda.synchronize()
    q, s = oq.quantise(x.float().numpy(), group, fmt)
    tok = oq.tokens(idx, b, h, w)
    want, swant = before.reshape(n, h * w, -1).copy(), sbefore.reshape(n, h * w, -1).copy()
    want[:, tok] = oq.stored(q, fmt).reshape(n, h * w, -1)[:, tok]
    swant[:, tok] = s.reshape(n, h * w, -1)[:, tok]
    got = byte_view(cache).reshape(n, h * w, -1)
    if fmt == "e4m3":   # -0 and 0 are the same value
        got, want = np.where(got == 128, 0, got), np.where(want == 128, 0, want)
    assert np.array_equal(cache.scales.cpu().numpy().reshape(n, h * w, -1), swant, equal_nan=True)
    assert np.array_equal(got, want)
    return cache


SHAPES = [
    (1, 16, 16, 320, 40), (2, 13, 11, 128, 128), (1, 9, 7, 1280, 1280), (1, 5, 6, 64, 8), (3, 4, 5, 24, 24),
    (1, 3, 3, 4096, 2048), (1, 2, 2, 5120, 2560), (1, 7, 5, 36, 12), (1, 5, 5, 30, 10), (1, 1, 1, 16, 16), (2, 6, 3, 200, 2),
    (1, 4, 4, 1024, 512), (1, 33, 31, 96, 32),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,h,w,c,group", SHAPES)
def test_write_whole_map(n, h, w, c, group, dtype, fmt):
    check_write(random_map(np.random.default_rng(h * w + c), n, h, w, c, dtype), group, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,h,w,c,group,b", [(1, 16, 16, 320, 40, 4), (2, 13, 11, 128, 128, 4), (2, 9, 7, 30, 10, 2),
                                             (1, 8, 8, 64, 32, 1), (3, 17, 23, 48, 16, 8), (1, 20, 20, 16, 16, 64)])
def test_write_at_tiles(n, h, w, c, group, b, fmt):
    rng = np.random.default_rng(b + c)
    idx, where = tile_list(rng, h, w, b)
    check_write(random_map(rng, n, h, w, c, torch.bfloat16), group, fmt, idx, where, b)


def test_write_group_of_one():
    """Every element its own scale: codes are +-127 (or 0)."""
    check_write(random_map(np.random.default_rng(5), 1, 4, 5, 9, torch.float32), 1, "s8")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("group", [8, 6])
def test_write_special_values(fmt, group):
    """Infinities, NaN, subnormals, the largest floats, exact ties, in the vector
    form (groups of 8) and the other (groups of 6)."""
    big, tiny = 3.4028234663852886e38, 1e-45
    rows = [[0.0] * 8, [-0.0] * 8, [np.inf] + [1.0] * 7, [1.0, -np.inf] + [2.0] * 6, [np.nan] + [1.0] * 7, [np.nan, np.inf] * 4,
            [tiny] * 8, [1e-37, 1e-38, 0, 0, 0, 0, 0, 0], [1.5e-36, 1e-37, -1e-36, 0, 0, 0, 0, 0], [1e-36] * 8, [big, -big, 1.0, 0, 0, 0, 0, 0],
            [127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 125.5, 126.5], [7.0, 0.5, 1.5, 2.5, -3.5, -4.5, 5.5, 6.5],
            [14.0, 1.0, 3.0, 5.0, -7.0, -9.0, 11.0, 13.0], [448.0, 208.0, 17.0, 19.0, 0.0009765625, 0.0029296875, -21.0, 1.0625],
            [449.0, 1.0, 2.0, 3.0, 4.0, 5.0, 6.0, 7.0], [1.0000001, 0.5, 0.25, 0.49999997, 1e-10, -1e-10, 0.003937008, 0.0039370083]]
    x = torch.tensor([r[:group] for r in rows], dtype=torch.float32).view(1, 1, len(rows), group)
    cache = check_write(x, group, fmt)
    back = sige.sige_qcache_read(cache, dtype=torch.float32).cpu().view(len(rows), group)
    assert torch.isnan(back[2:6]).all() and torch.isfinite(back[6:10]).all() and not back[:2].any()


@pytest.mark.parametrize("fmt", ["s8", "s4"])
def test_write_near_ties(fmt):
    """Values within a few float32 steps of every tie k + 1/2 of many scales: the
    exact quotient decides."""
    rng = np.random.default_rng(11)
    qm = oq.QMAX[fmt]
    m = rng.uniform(0.5, 4.0, size=(4000, 1)).astype(np.float32)
    s = m / np.float32(qm)
    k = rng.integers(-int(qm), int(qm), size=(4000, 15))
    v = ((k + 0.5) * s.astype(np.float64)).astype(np.float32)
    for _ in range(2):
        v = np.where(rng.random(v.shape) < 0.4, np.nextafter(v, np.float32(0)), v)
        v = np.where(rng.random(v.shape) < 0.4, np.nextafter(v, np.float32(9)), v)
    x = np.concatenate([m, np.clip(v, -m, m)], 1)
    check_write(torch.from_numpy(x).view(1, 40, 100, 16), 16, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("off", [1, 4, 8])
def test_write_and_read_unaligned(fmt, off):
    """Maps and codes that start off the vector form's alignment."""
    rng = np.random.default_rng(off)
    n, h, w, c, group = 1, 6, 5, 64, 16
    x = random_map(rng, n, h, w, c, torch.bfloat16)
    buf = torch.empty(x.numel() + off, dtype=torch.bfloat16, device=DEV)
    xd = buf[off:].view(n, h, w, c)
    xd.copy_(x)
    cb = c // 2 if fmt == "s4" else c
    raw = torch.zeros(n * h * w * cb + off, dtype=torch.uint8, device=DEV)
    store = {"s8": torch.int8, "e4m3": torch.float8_e4m3fn, "s4": torch.uint8}[fmt]
    cache = sige.QCache(raw[off:].view(store).view(n, h, w, cb), torch.zeros((n, h, w, c // group), device=DEV), fmt)
    sige.sige_qcache_write(xd, cache)
    ref = sige.sige_qcache_write(x.to(DEV), sige.qcache_empty(n, h, w, c, fmt, group))
    assert torch.equal(cache.codes.view(torch.uint8), ref.codes.view(torch.uint8))
    assert torch.equal(cache.scales, ref.scales)
    assert not raw[:off].any()
    y = torch.zeros(x.numel() + off, dtype=torch.bfloat16, device=DEV)
    sige.sige_qcache_read(cache, y[off:].view(n, h, w, c))
    assert torch.equal(y[off:], sige.sige_qcache_read(ref).view(-1)) and not y[:off].any()


@pytest.mark.parametrize("n,h,w,c,group", [(2, 5, 6, 64, 32), (1, 4, 7, 30, 10)])
@pytest.mark.parametrize("silu", [False, True])
def test_write_with_transform(n, h, w, c, group, silu):
    """GroupNorm affine (+ SiLU) before the codes.  The float32 transform is off
    by at most 2^-22 of the terms' magnitudes (one fma; __expf and __fdividef
    add 2^-21 (2 + |t|)), so a code is at most that plus half a step from the
    exact value, and a scale that far, relatively, from the exact one."""
    rng = np.random.default_rng(c)
    x = random_map(rng, n, h, w, c, torch.bfloat16).clamp(-50, 50)
    gs, gh = rng.normal(size=(n, c)).astype(np.float32), rng.normal(size=(n, c)).astype(np.float32)
    cache = sige.qcache_empty(n, h, w, c, "s8", group)
    sige.sige_qcache_write(x.to(DEV), cache, gn_scale=torch.from_numpy(gs).to(DEV), gn_shift=torch.from_numpy(gh).to(DEV),
                           silu=silu)
    prod = x.double().numpy() * gs[:, None, None].astype(np.float64)
    t = prod + gh[:, None, None]
    err = (np.abs(prod) + np.abs(gh[:, None, None])) * 2.0 ** -23
    if silu:
        err = err * 1.2 + np.abs(t) * (2 + np.abs(t)) * 2.0 ** -21
        t = t / (1 + np.exp(-t))
    s = cache.scales.double().cpu().numpy()
    m = np.abs(t).reshape(n, h, w, -1, group).max(-1)
    em = err.reshape(n, h, w, -1, group).max(-1)
    assert (np.abs(127 * s - m) <= em + m * 2.0 ** -23).all()
    back = cache.codes.double().cpu().numpy() * np.repeat(s, group, -1)
    assert (np.abs(back - t) <= err + np.repeat(s, group, -1) * (0.5 + 2.0 ** -20)).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,h,w,c,group", [(1, 16, 16, 320, 40), (2, 13, 11, 30, 10), (1, 5, 6, 64, 64), (1, 1, 1, 2, 2)])
def test_read(n, h, w, c, group, dtype, fmt):
    rng = np.random.default_rng(c + group)
    cache, q, s = random_cache(rng, n, h, w, c, group, fmt)
    want = torch.from_numpy((q.reshape(*s.shape, -1).astype(np.float32) * s[..., None]).reshape(q.shape)).to(dtype)
    assert torch.equal(sige.sige_qcache_read(cache, dtype=dtype).cpu(), want)
    # the listed tiles only
    idx, where = tile_list(rng, h, w, 4)
    y0 = random_map(rng, n, h, w, c, dtype)
    y = y0.to(DEV)
    sige.sige_qcache_read(cache, y, **where)
    tok = torch.from_numpy(oq.tokens(idx, 4, h, w))
    ref = y0.clone().view(n, h * w, c)
    ref[:, tok] = want.view(n, h * w, c)[:, tok]
    assert torch.equal(bits(y).view(-1), bits(ref).view(-1))


def test_lists_that_are_short_long_or_out_of_the_map():
    """A count of zero, one above the capacity, tiles outside the map or listed
    twice: only in-image pixels of the first `capacity` tiles are touched."""
    rng = np.random.default_rng(21)
    n, h, w, c = 2, 10, 10, 32
    x = random_map(rng, n, h, w, c, torch.bfloat16)
    full = sige.sige_qcache_write(x.to(DEV), sige.qcache_empty(n, h, w, c, "s8", 16))
    tiles = torch.tensor([[4, 4], [4, 4], [8, 8], [-4, 0], [0, -1], [12, 0], [0, 400], [0, 0]], dtype=torch.int32, device=DEV)
    for count, cap, listed in ((0, 8, []), (-3, 8, []), (99, 3, [(4, 4), (8, 8)]), (8, 8, [(4, 4), (8, 8), (0, 0)])):
        cache = sige.QCache(torch.full((n, h, w, c), 77, dtype=torch.int8, device=DEV),
                            torch.full((n, h, w, 2), 5.0, device=DEV), "s8")
        y = torch.full((n, h, w, c), 3.0, dtype=torch.bfloat16, device=DEV)
        where = dict(idx=tiles, count=torch.tensor([count], dtype=torch.int32, device=DEV), capacity=cap, block=4)
        sige.sige_qcache_write(x.to(DEV), cache, **where)
        sige.sige_qcache_read(full, y, **where)
        hit = torch.zeros((h, w), dtype=torch.bool, device=DEV)
        for a, b in listed:
            hit[a:a + 4, b:b + 4] = True
        assert torch.equal(cache.codes[:, hit], full.codes[:, hit]) and (cache.codes[:, ~hit] == 77).all()
        assert torch.equal(cache.scales[:, hit], full.scales[:, hit]) and (cache.scales[:, ~hit] == 5).all()
        assert torch.equal(y[:, hit], sige.sige_qcache_read(full)[:, hit]) and (y[:, ~hit] == 3).all()


def test_offsets_past_32_bits():
    """A map of more than 2^31 elements: the last pixels land where they belong."""
    n, h, w, c = 1, 1, 1 << 20, 2304
    x = torch.zeros((n, h, w, c), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    x[:, :, -3:] = torch.randn((n, h, 3, c), generator=g, device=DEV).to(torch.bfloat16)
    cache = sige.qcache_empty(n, h, w, c, "s8", 8)
    sige.sige_qcache_write(x, cache)
    small = sige.sige_qcache_write(x[:, :, -3:].contiguous(), sige.qcache_empty(n, h, 3, c, "s8", 8))
    assert torch.equal(cache.codes[:, :, -3:], small.codes) and torch.equal(cache.scales[:, :, -3:], small.scales)
    assert not cache.codes[:, :, -100:-3].any()
    sige.sige_qcache_read(cache, x.fill_(1.0))
    assert torch.equal(x[:, :, -3:], sige.sige_qcache_read(small)) and not x[:, :, -100:-3].any()


def test_streams_and_graphs():
    """The calls on a stream of their own and in a captured graph replayed on
    new values give what the eager calls give."""
    rng = np.random.default_rng(31)
    n, h, w, c = 1, 32, 32, 320
    x = random_map(rng, n, h, w, c, torch.bfloat16).to(DEV)
    _, where = tile_list(rng, h, w, 4)
    ref = sige.sige_qcache_write(x, sige.qcache_empty(n, h, w, c, "e4m3", 40))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache = sige.qcache_empty(n, h, w, c, "e4m3", 40)
    sige.sige_qcache_write(x, cache, stream=side)
    y = sige.sige_qcache_read(cache, stream=side)
    side.synchronize()
    assert torch.equal(cache.codes.view(torch.uint8), ref.codes.view(torch.uint8))
    assert torch.equal(y, sige.sige_qcache_read(ref))
    graph = torch.cuda.CUDAGraph()
    out = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        sige.sige_qcache_write(x, cache, **where)
        sige.sige_qcache_read(cache, out, **where)
    x.copy_(random_map(rng, n, h, w, c, torch.bfloat16))
    graph.replay()
    eager = sige.sige_qcache_read(sige.sige_qcache_write(x, sige.qcache_empty(n, h, w, c, "e4m3", 40)), torch.zeros_like(x),
                                  **where)
    torch.cuda.synchronize()
    assert torch.equal(out, eager)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [8, 16, 24, 32, 56, 72, 80, 168, 320, 640, 1000, 1280, 2040, 2048])
def test_write_group_widths(group, dtype, fmt):
    """Every split of a group over lanes and vectors, two groups a pixel; half of
    a group's largest magnitude, the commonest near tie of bf16 maps, in each."""
    rng = np.random.default_rng(group)
    x = random_map(rng, 1, 5, 7, 2 * group, dtype)
    g = x.view(-1, group)
    g[:, group // 2] = g.abs().amax(1) / 2
    check_write(x, group, fmt)


@pytest.mark.parametrize("fmt", ["s8", "s4"])
@pytest.mark.parametrize("shift", [-119, -118, -117, -60, 60, 124])
def test_write_near_ties_of_extreme_scales(fmt, shift):
    """The near ties of test_write_near_ties with scales from 2^-126 up to the
    largest: shifts by a power of two, exact but for subnormal elements."""
    rng = np.random.default_rng(12)
    qm = oq.QMAX[fmt]
    m = rng.uniform(1.0, 2.0, size=(2000, 1)).astype(np.float32)
    s = m / np.float32(qm)
    k = rng.integers(-int(qm), int(qm), size=(2000, 15))
    v = ((k + 0.5) * s.astype(np.float64)).astype(np.float32)
    v = np.where(rng.random(v.shape) < 0.4, np.nextafter(v, np.float32(0)), v)
    x = np.ldexp(np.concatenate([m, np.clip(v, -m, m)], 1), shift).astype(np.float32)
    check_write(torch.from_numpy(x).view(1, 20, 100, 16), 16, fmt)


def test_more_groups_than_32_bits_count():
    """More than 2^31 groups and vectors in the map, few of them listed: the
    last tile's, with a transform whose channels follow from the group."""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    h, w, c = 1024, 1024, 18432
    rng = np.random.default_rng(5)
    small = random_map(rng, 1, 2, 2, c, torch.bfloat16).clamp(-50, 50).to(DEV)
    x = torch.empty((1, h, w, c), dtype=torch.bfloat16, device=DEV)
    x[:, -2:, -2:] = small
    gn = dict(gn_scale=torch.from_numpy(rng.normal(size=(1, c)).astype(np.float32)).to(DEV),
              gn_shift=torch.from_numpy(rng.normal(size=(1, c)).astype(np.float32)).to(DEV))
    where = dict(idx=torch.tensor([[h - 2, w - 2]], dtype=torch.int32, device=DEV),
                 count=torch.ones(1, dtype=torch.int32, device=DEV), capacity=1, block=2)
    cache = sige.sige_qcache_write(x, sige.qcache_empty(1, h, w, c, "s8", 8), **where, **gn)
    ref = sige.sige_qcache_write(small, sige.qcache_empty(1, 2, 2, c, "s8", 8), **gn)
    assert torch.equal(cache.codes[:, -2:, -2:], ref.codes) and torch.equal(cache.scales[:, -2:, -2:], ref.scales)
    sige.sige_qcache_read(cache, x, **where)
    assert torch.equal(x[:, -2:, -2:], sige.sige_qcache_read(ref))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [2, 4, 6, 10, 12, 20, 44, 90, 100, 250, 510, 516, 1020, 1028])
def test_narrow_accesses(group, dtype, fmt):
    """Groups that four, two or no elements at once divide: written and read,
    whole and at tiles."""
    rng = np.random.default_rng(group)
    x = random_map(rng, 2, 7, 6, 3 * group, dtype)
    cache = check_write(x, group, fmt)
    idx, where = tile_list(rng, 7, 6, 2)
    check_write(x, group, fmt, idx, where, 2)
    values = torch.from_numpy(oq.values(*oq.quantise(x.float().numpy(), group, fmt)).astype(np.float32)).to(dtype)
    assert torch.equal(sige.sige_qcache_read(cache, dtype=dtype).cpu(), values.view(x.shape))
