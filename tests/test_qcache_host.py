"""Host-side checks of the quantised cache's calls: sizes, refusals before any
device work (fake pointers: nothing is launched), and the binding's checks."""
import ctypes

import pytest
import torch

import spatially_sparse_incremental_b200 as sige


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build_library()
    return sige.lib()


X, CODES, SCALES, IDX, CNT = (ctypes.c_void_p(0x10000000 * k) for k in range(1, 6))
OUT, WS, B, W, SW = (ctypes.c_void_p(0x10000000 * k) for k in range(6, 11))


def _td(n=1, h=16, w=16, c=320, dt=sige.BF16, layout=sige.NHWC):
    return sige.TensorDesc(n, h, w, c, dt, layout)


def _qd(n=1, h=16, w=16, c=320, fmt=sige.Q_S8, group=40):
    return sige.QCacheDesc(n, h, w, c, fmt, group)


def test_sizes(L):
    assert sige.sige_qcache_code_bytes(_qd(2, 3, 5, 24, sige.Q_S8, 8)) == 2 * 3 * 5 * 24
    assert sige.sige_qcache_code_bytes(_qd(2, 3, 5, 24, sige.Q_S4, 8)) == 2 * 3 * 5 * 12
    assert sige.sige_qcache_scales(_qd(2, 3, 5, 24, sige.Q_E4M3, 8)) == 2 * 3 * 5 * 3
    big = _qd(64, 4096, 4096, 1280, sige.Q_E4M3, 1280)              # past 32 bits
    assert sige.sige_qcache_code_bytes(big) == 64 * 4096 * 4096 * 1280
    for bad in (_qd(group=0), _qd(group=33), _qd(c=0), _qd(fmt=3), _qd(fmt=-1), _qd(c=9, fmt=sige.Q_S4, group=3),
                _qd(n=1 << 16, h=1 << 16), _qd(w=-1)):
        assert sige.sige_qcache_code_bytes(bad) == 0 and sige.sige_qcache_scales(bad) == 0
    assert L.sige_qcache_code_bytes(None) == 0


def _rw(L, write, **kw):
    a = dict(x=X, xd=_td(), gs=None, gh=None, silu=0, block=4, idx=IDX, cnt=CNT, cap=16, codes=CODES, scales=SCALES,
             cd=_qd())
    a.update(kw)
    xd = ctypes.byref(a["xd"]) if a["xd"] is not None else None
    cd = ctypes.byref(a["cd"]) if a["cd"] is not None else None
    if write:
        return L.sige_qcache_write(a["x"], xd, a["gs"], a["gh"], a["silu"], a["block"], a["idx"], a["cnt"], a["cap"],
                                   a["codes"], a["scales"], cd, None)
    return L.sige_qcache_read(a["codes"], a["scales"], cd, a["block"], a["idx"], a["cnt"], a["cap"], a["x"], xd, None)


@pytest.mark.parametrize("write", [True, False])
def test_cache_refusals(L, write):
    bad = [dict(x=None), dict(xd=None), dict(codes=None), dict(scales=None), dict(cd=None), dict(cnt=None),
           dict(cap=-1), dict(block=0), dict(idx=ctypes.c_void_p(0x1004)), dict(cd=_qd(group=48)),
           dict(cd=_qd(h=15)), dict(cd=_qd(n=2)), dict(cd=_qd(fmt=7)), dict(codes=X), dict(scales=X), dict(scales=CODES),
           dict(x=ctypes.c_void_p(0x10000001)), dict(scales=ctypes.c_void_p(0x30000002)),
           dict(codes=ctypes.c_void_p(0x10000000 + 16 * 16 * 320 * 2 - 1))]
    for kw in bad:
        assert _rw(L, write, **kw) == sige.ERR_INVALID_ARG, kw
    for kw in (dict(xd=_td(dt=sige.U8)), dict(xd=_td(layout=sige.NCHW)), dict(block=65),
               dict(cd=_qd(c=9, group=3, fmt=sige.Q_S4), xd=_td(c=9)), dict(cap=1 << 27)):
        assert _rw(L, write, **kw) == sige.ERR_UNSUPPORTED, kw
    n0 = sige.sige_launch_count()
    assert _rw(L, write, cap=0) == sige.OK
    assert sige.sige_launch_count() == n0
    if write:
        assert _rw(L, True, gs=B) == sige.ERR_INVALID_ARG
        assert _rw(L, True, gh=B) == sige.ERR_INVALID_ARG


def test_qlinear_refusals(L):
    def call(**kw):
        a = dict(a=CODES, sa=SCALES, ad=_qd(group=320), w=W, sw=SW, wd=_qd(n=64, h=1, w=1, group=320), bias=None,
                 block=4, idx=IDX, cnt=CNT, cap=16, res=None, y=OUT, yd=_td(c=64), ws=WS, wsb=256)
        a.update(kw)
        r = lambda d: ctypes.byref(d) if d is not None else None
        return L.sige_qlinear(a["a"], a["sa"], r(a["ad"]), a["w"], a["sw"], r(a["wd"]), a["bias"], a["block"], a["idx"],
                              a["cnt"], a["cap"], a["res"], a["y"], r(a["yd"]), a["ws"], a["wsb"], None)
    for kw in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(y=None), dict(yd=None), dict(ad=None),
               dict(wd=None), dict(cnt=None), dict(cap=-1), dict(block=0), dict(idx=ctypes.c_void_p(0x1004)),
               dict(wd=_qd(n=64, h=2, w=1, group=320)), dict(wd=_qd(n=64, h=1, w=1, c=160, group=160)),
               dict(yd=_td(c=65)), dict(yd=_td(h=8, c=64)), dict(y=CODES), dict(res=OUT), dict(y=SW),
               dict(y=ctypes.c_void_p(0x60000001)), dict(bias=ctypes.c_void_p(0x70000002))):
        assert call(**kw) == sige.ERR_INVALID_ARG, kw
    for kw in (dict(ad=_qd(group=40)), dict(ad=_qd(group=320, fmt=sige.Q_E4M3)), dict(yd=_td(c=64, dt=sige.U8)),
               dict(wd=_qd(n=64, h=1, w=1, group=320, fmt=sige.Q_S4)), dict(yd=_td(c=64, layout=sige.NCHW)),
               dict(block=65), dict(ad=_qd(c=131072, group=131072), wd=_qd(n=64, h=1, w=1, c=131072, group=131072))):
        assert call(**kw) == sige.ERR_UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(wsb=255), dict(ws=ctypes.c_void_p(0x70000008))):
        assert call(**kw) == sige.ERR_WORKSPACE, kw
    assert call(cap=0) == sige.OK


def test_attention_qcache_refusals(L):
    def call(**kw):
        a = dict(q=X, qd=_td(), k=CODES, ks=SCALES, kd=_qd(h=77, w=1), v=W, vs=SW, vd=_qd(h=77, w=1), kc=None, heads=8,
                 block=4, idx=IDX, cnt=CNT, cap=16, o=OUT, ws=WS, wsb=256)
        a.update(kw)
        r = lambda d: ctypes.byref(d) if d is not None else None
        return L.sige_attention_qcache(a["q"], r(a["qd"]), a["k"], a["ks"], r(a["kd"]), a["v"], a["vs"], r(a["vd"]),
                                       a["kc"], a["heads"], a["block"], a["idx"], a["cnt"], a["cap"], a["o"], a["ws"],
                                       a["wsb"], None)
    for kw in (dict(q=None), dict(qd=None), dict(k=None), dict(ks=None), dict(kd=None), dict(v=None), dict(vs=None),
               dict(vd=None), dict(o=None), dict(heads=0), dict(heads=3), dict(cnt=None), dict(cap=-1), dict(block=0),
               dict(kd=_qd(h=76, w=1)), dict(kd=_qd(n=2, h=77, w=1)), dict(vd=_qd(n=2, h=77, w=1)),
               dict(kd=_qd(h=77, w=1, c=160)), dict(o=X), dict(o=W), dict(kc=ctypes.c_void_p(0x70000002))):
        assert call(**kw) == sige.ERR_INVALID_ARG, kw
    for kw in (dict(heads=1), dict(kd=_qd(h=77, w=1, group=20)), dict(vd=_qd(h=77, w=1, group=8)),
               dict(qd=_td(dt=sige.F32)), dict(qd=_td(layout=sige.NCHW)), dict(block=65)):
        assert call(**kw) == sige.ERR_UNSUPPORTED, kw
    assert call(ws=None) == sige.ERR_WORKSPACE
    assert call(wsb=16) == sige.ERR_WORKSPACE
    assert call(cap=0) == sige.OK
    assert sige.sige_attention_qcache_path(257, 8) == sige.ERR_UNSUPPORTED
    assert sige.sige_attention_qcache_path(0, 8) == sige.ERR_INVALID_ARG


def test_binding_refusals():
    codes, scales = torch.zeros((1, 4, 4, 16), dtype=torch.int8), torch.zeros((1, 4, 4, 2))
    c = sige.QCache(codes, scales, "s8")
    assert c.shape == (1, 4, 4, 16) and c.group == 8
    s4 = sige.QCache(codes.view(torch.uint8), scales, "s4")
    assert s4.shape == (1, 4, 4, 32) and s4.group == 16
    for args in ((codes, scales, "s5"), (codes, scales, "e4m3"), (codes, scales.double(), "s8"),
                 (codes, scales[:, :3], "s8"), (codes, scales.transpose(1, 2), "s8"),
                 (codes, torch.zeros((1, 4, 4, 3)), "s8"), (codes[0], scales[0], "s8")):
        with pytest.raises(ValueError):
            sige.QCache(*args)
    for kw in (dict(group=5), dict(group=0), dict(format="s4", group=1)):
        with pytest.raises(ValueError):
            sige.qcache_empty(1, 4, 4, 16, device="cpu", **kw)
    x = torch.zeros((1, 4, 4, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sige.sige_qcache_write(x, c)                                   # host tensors
    with pytest.raises(ValueError, match="fit"):
        sige.sige_qcache_write(x[:, :3], c)
    with pytest.raises(ValueError):
        sige.sige_qcache_write(x, c, idx=torch.zeros((2, 2)), count=torch.zeros(1), capacity=2)
    idx = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="capacity"):
        sige.sige_qcache_read(c, x, idx=idx, count=torch.zeros(1, dtype=torch.int32), capacity=3)
    with pytest.raises(ValueError):
        sige.sige_qcache_read(c, x, idx=idx, capacity=2)               # no count
    with pytest.raises(ValueError):
        sige.sige_qlinear(c, c, bias=torch.zeros(3))
    with pytest.raises(ValueError):
        sige.sige_attention_qcache(x, c, c, 2, key_counts=torch.zeros(2, dtype=torch.int32))


def test_counts_near_the_end_of_32_bits(L):
    """Channels or keys so many that a tile past the last would leave 32 bits are
    refused, whatever the addresses."""
    most = 2 ** 31 - 1
    r = ctypes.byref
    a, w, y = _qd(n=1, h=1, w=1, c=16, group=16), _qd(n=most, h=1, w=1, c=16, group=16), _td(n=1, h=1, w=1, c=most)
    assert L.sige_qlinear(CODES, SCALES, r(a), W, SW, r(w), None, 1, None, None, 0, None, OUT, r(y), WS, 256,
                          None) == sige.ERR_UNSUPPORTED
    q, k = _td(n=1, h=1, w=1, c=16), _qd(n=1, h=most, w=1, c=16, group=16)
    assert L.sige_attention_qcache(X, r(q), CODES, SCALES, r(k), W, SW, r(k), None, 1, 1, None, None, 0, OUT, WS, 256,
                                   None) == sige.ERR_UNSUPPORTED


def test_outputs_in_an_operand_are_refused(L):
    """An output over the list, its count, the affine, the key counts or the
    workspace: refused like one over any other operand."""
    r = ctypes.byref
    at = lambda p, k: ctypes.c_void_p(p.value + k)
    xb, cb, sb = 16 * 16 * 320 * 2, 16 * 16 * 320, 16 * 16 * 8 * 4
    for kw in (dict(gs=at(CODES, cb - 4), gh=B), dict(gs=B, gh=at(SCALES, -4 * 320 + 4)), dict(gs=SCALES, gh=B), dict(idx=at(CODES, 8)),
               dict(idx=at(CODES, -8 * 16 + 8)), dict(cnt=at(SCALES, sb - 4)), dict(cnt=CODES), dict(idx=SCALES)):
        assert _rw(L, True, **kw) == sige.ERR_INVALID_ARG, kw
    for kw in (dict(idx=at(X, xb - 8)), dict(idx=at(X, -8)), dict(cnt=X)):
        assert _rw(L, False, **kw) == sige.ERR_INVALID_ARG, kw
    assert _rw(L, False, idx=at(CODES, 8), cap=0) == sige.OK      # (operands may share memory)
    lin = lambda **k: L.sige_qlinear(CODES, SCALES, r(_qd(group=320)), W, SW, r(_qd(n=64, h=1, w=1, group=320)), None, 4,
                                     k.get("idx", IDX), k.get("cnt", CNT), 16, None, OUT, r(_td(c=64)), k.get("ws", WS), 256, None)
    yb = 16 * 16 * 64 * 2
    for kw in (dict(idx=OUT), dict(idx=at(OUT, yb - 8)), dict(cnt=at(OUT, 4)), dict(ws=at(OUT, yb - 16)), dict(ws=at(OUT, -240))):
        assert lin(**kw) == sige.ERR_INVALID_ARG, kw
    kd = _qd(h=77, w=1)
    att = lambda **k: L.sige_attention_qcache(X, r(_td()), CODES, SCALES, r(kd), W, SW, r(kd), k.get("kc"), 8, 4, k.get("idx", IDX),
                                              k.get("cnt", CNT), 16, OUT, k.get("ws", WS), 256, None)
    for kw in (dict(kc=OUT), dict(kc=at(OUT, xb - 4)), dict(idx=at(OUT, -120)), dict(cnt=OUT), dict(ws=OUT)):
        assert att(**kw) == sige.ERR_INVALID_ARG, kw


def test_sizes_past_32_bits_are_refused():
    """Sizes that an int32 would take modulo 2^32 (5 pixels of 2^32 + 5)."""
    at = lambda shape, dt: torch.empty(shape, dtype=dt, device="meta")
    for shape in ((1, 1, 2 ** 32 + 5, 1), (2 ** 32 + 1, 1, 1, 2), (1, 2 ** 31, 1, 8), (1, 1, 1, 2 ** 32 + 16)):
        with pytest.raises(ValueError, match="32 bits"):
            sige.QCache(at(shape, torch.int8), at((*shape[:3], 1), torch.float32), "s8")
        with pytest.raises(ValueError, match="32 bits"):
            sige.qcache_empty(*shape, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        sige.QCache(at((1, 1, 1, 2 ** 30), torch.uint8), at((1, 1, 1, 1), torch.float32), "s4")   # 2^31 channels
    c = sige.QCache(torch.zeros((1, 4, 4, 16), dtype=torch.int8), torch.zeros((1, 4, 4, 1)), "s8")
    x = torch.zeros((1, 4, 4, 16), dtype=torch.bfloat16)
    idx, cnt = torch.zeros((2, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="32 bits"):
        sige.sige_qcache_write(x, c, idx=idx, count=cnt, capacity=2, block=2 ** 32 + 4)
    with pytest.raises(ValueError, match="32 bits"):
        sige.sige_attention_qcache(at((1, 2 ** 32 + 4, 1, 16), torch.bfloat16), c, c, 2)
    with pytest.raises(ValueError, match="32 bits"):
        sige.sige_attention_qcache(x, c, c, 2 ** 32 + 2)
