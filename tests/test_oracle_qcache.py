"""Pins of the quantised cache's oracle (oracle/qcache.py): worked values, ties,
the e4m3 format against torch's CPU conversion, and bounds of the rounding."""
import numpy as np
import pytest
import torch

from oracle import qcache as oq


def test_integer_codes_by_hand():
    # m = 127: scale 1, codes the values rounded with ties to even
    t = np.array([[127.0, 0.5, 1.5, -0.5, -2.5, 2.5, 126.49999, -127.0]])
    q, s = oq.quantise(t, 8, "s8")
    assert s.tolist() == [[1.0]]
    assert q.tolist() == [[127, 0, 2, 0, -2, 2, 126, -127]]
    # 4 bits: m = 14 -> scale 2
    q, s = oq.quantise(np.array([[14.0, 1.0, 3.0, -5.0]]), 4, "s4")
    assert s.tolist() == [[2.0]] and q.tolist() == [[7, 0, 2, -2]]
    assert oq.stored(q, "s4").tolist() == [[0x07, 0xE2]]


def test_groups_zeros_and_poison():
    t = np.array([[1.0, 2.0, 0.0, 0.0, np.inf, 1.0, np.nan, 1.0, 1e-40, 1e-41]])
    for fmt in ("s8", "e4m3", "s4"):
        q, s = oq.quantise(t, 2, fmt)
        assert s[0, 1] == 0 and np.isnan(s[0, 2]) and np.isnan(s[0, 3]) and s[0, 4] == 0
        assert not q[0, 2:].any()
        v = oq.values(q, s)
        assert not v[0, 2:4].any() and np.isnan(v[0, 4:8]).all()


def test_e4m3_matches_torch():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 20000), 2.0 ** rng.uniform(-12, 8.8, 20000), np.arange(-448, 449) / 2,
                        np.arange(512) * 2.0 ** -11]).astype(np.float32)
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn)
    got = oq.e4m3_round(v)
    assert np.array_equal(got, ref.float().numpy().astype(np.float64))
    plus = got != 0
    assert np.array_equal(oq.stored(got[plus], "e4m3"), ref.view(torch.uint8).numpy()[plus])


@pytest.mark.parametrize("fmt,step", [("s8", 0.5), ("s4", 0.5), ("e4m3", None)])
def test_rounding_is_half_a_step(fmt, step):
    rng = np.random.default_rng(1)
    t = (rng.normal(size=(50, 48)) * np.exp(rng.normal(size=(50, 1)) * 4)).astype(np.float32).astype(np.float64)
    q, s = oq.quantise(t, 16, fmt)
    d = np.abs(oq.values(q, s) - t).reshape(50, 3, 16)
    S = s.astype(np.float64)[..., None]
    if step:
        assert (d <= step * S * (1 + 2 ** -20)).all()
        assert np.abs(q).max() == oq.QMAX[fmt]
    else:
        # half a step of 3 mantissa bits, or half the subnormal spacing
        assert (d <= np.maximum(np.abs(t).reshape(50, 3, 16) * 2.0 ** -4, S * 2.0 ** -10)).all()
        m = np.abs(t).reshape(50, 3, 16).max(-1)
        assert (m <= 448 * s).all() and (m > 224 * s).all()


def test_qlinear_is_the_product_of_values():
    rng = np.random.default_rng(2)
    a, w = rng.integers(-127, 128, (5, 33)), rng.integers(-127, 128, (7, 33))
    sa, sw = rng.random(5), rng.random(7)
    ref = (a * sa[:, None]) @ (w * sw[:, None]).T + 1.0
    assert np.allclose(oq.qlinear(a, sa, w, sw, bias=np.ones(7)), ref, rtol=1e-12)


def test_attention_counts():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(4, 6)), rng.normal(size=(9, 6)), rng.normal(size=(9, 8))
    o, _ = oq.attention(q, k, v, 2, 5)
    ref, _ = oq.attention(q, k[:5], v[:5], 2)
    assert np.array_equal(o, ref)
    assert not oq.attention(q, k, v, 2, 0)[0].any()
    o, _ = oq.attention(q, k, v, 2, 1)
    assert np.allclose(o, np.broadcast_to(v[0], o.shape))
    t = torch.nn.functional.scaled_dot_product_attention(
        *(torch.from_numpy(x).reshape(1, x.shape[0], 2, -1).transpose(1, 2) for x in (q, k, v)))
    assert np.allclose(oq.attention(q, k, v, 2)[0], t.transpose(1, 2).reshape(4, 8).numpy(), atol=1e-12)
