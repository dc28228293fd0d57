"""What is measured of the quantised cache and the operators that read it.

Three operators, as a user of the sparse engine calls them:

  cache      an activation map is written into a cache of 8- or 4-bit codes
             (one float32 scale per group of channels of a pixel), at the
             listed tiles or whole, and read back the same way;
  linear     a projection of a cached map (8-bit integers, one scale per
             token) with 8-bit weights (one scale per output channel), at the
             listed tiles of a cached output or on the whole map;
  attention  the tokens under the listed tiles (or all) attend to a key and a
             value cache held in codes.

``run`` computes them in plain torch; with ``own`` set it makes the calls of
this repository's package instead.
"""
import math

import torch

own = False

QMAX = {"s8": 127.0, "s4": 7.0}
FORMATS = ("s8", "e4m3", "s4")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one small edit of a Stable-Diffusion latent map: 25 tiles of 4x4 pixels of a key map with a scale per head
        # (8 heads of 40) are written into the cache and restored into the working map
        dict(name="cache-sd64-tiles", op="cache", n=1, h=64, w=64, c=320, group=40, fmt="s8", dtype="bf16", tiles=25, block=4),
        # caching one conv output of a 256x256 DDPM layer, a scale per pixel
        dict(name="cache-ddpm256-map", op="cache", n=1, h=256, w=256, c=128, group=128, fmt="s8", dtype="bf16", tiles=-1, block=1),
        # the same layer at four images, 8-bit floats, a scale per 32 channels: the largest cache
        dict(name="cache-ddpm256-batch4", op="cache", n=4, h=256, w=256, c=128, group=32, fmt="e4m3", dtype="bf16", tiles=-1, block=1),
        # a ragged float32 map in 4 bits
        dict(name="cache-ragged-f32-s4", op="cache", n=2, h=37, w=53, c=200, group=40, fmt="s4", dtype="f32", tiles=-1, block=1),
        # a query projection at 16x16: 20 one-pixel tiles against 1280 x 1280 weights (latency and the weights' read)
        dict(name="linear-sd16-tiles", op="linear", n=1, h=16, w=16, c=1280, c_out=1280, dtype="bf16", tiles=20, block=1, bias=False, residual=False),
        # the output projection at 64x64 after one small edit, with bias and residual
        dict(name="linear-sd64-tiles", op="linear", n=1, h=64, w=64, c=320, c_out=320, dtype="bf16", tiles=25, block=4, bias=True, residual=True),
        # the second feed-forward product of the 64x64 level on four whole maps
        dict(name="linear-sd64-map", op="linear", n=4, h=64, w=64, c=1280, c_out=320, dtype="bf16", tiles=-1, block=1, bias=True, residual=True),
        # the first feed-forward product of the 32x32 level on sixteen whole maps: the largest product
        dict(name="linear-sd32-map16", op="linear", n=16, h=32, w=32, c=640, c_out=5120, dtype="bf16", tiles=-1, block=1, bias=True, residual=False),
        # odd sizes throughout, float32 output
        dict(name="linear-odd-f32", op="linear", n=1, h=13, w=11, c=74, c_out=51, dtype="f32", tiles=-1, block=1, bias=True, residual=False),
        # self-attention of the 400 tokens of a small edit over the 4096 cached keys
        dict(name="attn-sd64-tiles", op="attention", n=1, h=64, w=64, heads=8, dh=40, dv=40, keys=4096, fmt="s8", tiles=25, block=4, ragged=False),
        # the whole map of two images, 8-bit floats
        dict(name="attn-sd64-map", op="attention", n=2, h=64, w=64, heads=8, dh=40, dv=40, keys=4096, fmt="e4m3", tiles=-1, block=4, ragged=False),
        # cross-attention of a padded batch: contexts of 0 to 77 tokens, heads of 80
        dict(name="attn-sd32-cross", op="attention", n=3, h=32, w=32, heads=8, dh=80, dv=80, keys=77, fmt="s8", tiles=-1, block=4, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _tiles(rng, h, w, block):
    """-1 (the whole map) or a number of tiles, from one to a third of the grid."""
    grid = -(-h // block) * -(-w // block)
    return -1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, grid // 3))


def draw(rng):
    op = rng.choice(("cache", "linear", "attention"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    block = rng.choice((1, 2, 4, 8))
    if op == "cache":
        group = 2 * _log_int(rng, 4, 160)
        c = group * rng.choice((1, 1, 2, 4, 8))
        n = rng.choice((1, 2, 3, 4))
        most = max(16, (1 << 25) // (n * c))
        h = _log_int(rng, 3, min(256, math.isqrt(most)))
        w = _log_int(rng, 3, min(256, most // h))
        return dict(op=op, n=n, h=h, w=w, c=c, group=group, fmt=rng.choice(FORMATS), dtype=dtype,
                    tiles=_tiles(rng, h, w, block), block=block)
    if op == "linear":
        n = rng.choice((1, 1, 2, 4, 16))
        h, w = _log_int(rng, 1, 64 if n <= 4 else 32), _log_int(rng, 1, 64 if n <= 4 else 32)
        unit = rng.choice((16, 16, 16, 1))
        c = unit * _log_int(rng, 2, 1280 // unit if unit > 1 else 320)
        c_out = rng.choice((1, 8)) * _log_int(rng, 8, 640)
        return dict(op=op, n=n, h=h, w=w, c=c, c_out=c_out, dtype=dtype, tiles=_tiles(rng, h, w, block), block=block,
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    n = rng.choice((1, 1, 2))
    h, w = _log_int(rng, 2, 64), _log_int(rng, 2, 64)
    dh = 8 * rng.randint(1, 5) if rng.random() < 0.6 else rng.choice((64, 80, 100, 128, 160))
    heads = rng.choice((1, 2, 4, 8) if dh <= 40 else (1, 2))
    return dict(op=op, n=n, h=h, w=w, heads=heads, dh=dh, dv=dh, keys=_log_int(rng, 1, 4096), fmt=rng.choice(FORMATS),
                tiles=_tiles(rng, h, w, block), block=block, ragged=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _map(g, *shape):
    """Activations as a layer leaves them: normal, channels of unequal size, a few pixels without any signal."""
    x = torch.randn(shape, generator=g, device="cuda") * torch.exp(0.7 * torch.randn(shape[-1], generator=g, device="cuda"))
    return x * (torch.rand(shape[:-1], generator=g, device="cuda") > 0.01).unsqueeze(-1)


def _tile_list(g, case):
    """(idx, n_tiles, capacity): the list in row-major order with the grid's capacity, as the mask reduction leaves it."""
    h, w, b = case["h"], case["w"], case["block"]
    gh, gw = -(-h // b), -(-w // b)
    if case["tiles"] < 0:
        return None, 0, 0
    m = min(case["tiles"], gh * gw)
    t = torch.randperm(gh * gw, generator=g, device="cuda")[:m].sort().values
    idx = torch.zeros((gh * gw, 2), dtype=torch.int32, device="cuda")
    idx[:m, 0] = (t // gw * b).int()
    idx[:m, 1] = (t % gw * b).int()
    return idx, m, gh * gw


def prepare(case, seed):
    g = _generator(seed)
    idx, m, cap = _tile_list(g, case)
    s = dict(case=case, idx=idx, m=m, cap=cap,
             count=torch.tensor([m], dtype=torch.int32, device="cuda"),
             workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))   # kept by a user from call to call
    n, h, w = case["n"], case["h"], case["w"]
    if case["op"] == "cache":
        c, dt = case["c"], DTYPES[case["dtype"]]
        s["x"] = _map(g, n, h, w, c).to(dt)
        s["codes"], s["scales"] = _quantise(_map(g, n, h, w, c), case["group"], case["fmt"])   # the original's cache
        s["y"] = _map(g, n, h, w, c).to(dt)                                                  # the working map
    elif case["op"] == "linear":
        c, co, dt = case["c"], case["c_out"], DTYPES[case["dtype"]]
        s["a"] = _quantise(_map(g, n, h, w, c), c, "s8")
        s["w"] = _quantise(torch.randn((co, 1, 1, c), generator=g, device="cuda") / math.sqrt(c), c, "s8")
        s["bias"] = 0.1 * torch.randn(co, generator=g, device="cuda") if case["bias"] else None
        s["residual"] = torch.randn((n, h, w, co), generator=g, device="cuda").to(dt) if case["residual"] else None
        s["y"] = torch.randn((n, h, w, co), generator=g, device="cuda").to(dt)                # the cached output
    else:
        d, dv, keys = case["heads"] * case["dh"], case["heads"] * case["dv"], case["keys"]
        s["q"] = torch.randn((n, h, w, d), generator=g, device="cuda").to(torch.bfloat16)
        s["k"] = _quantise(torch.randn((n, keys, 1, d), generator=g, device="cuda"), case["dh"], case["fmt"])
        s["v"] = _quantise(torch.randn((n, keys, 1, dv), generator=g, device="cuda"), case["dv"], case["fmt"])
        s["o"] = torch.randn((n, h, w, dv), generator=g, device="cuda").to(torch.bfloat16)
        if case["ragged"]:
            # one context of each length at the ends, the others between them
            lens = torch.randint(0, keys + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
            lens[0] = keys
            if n > 1:
                lens[1] = 0
            s["lens"] = lens
        else:
            s["lens"] = None
    return s


# ------------------------------------------------------------------ the plain form

def _scale(amax, fmt):
    """The float32 scale of groups of largest magnitude ``amax``."""
    if fmt == "e4m3":
        m, e = torch.frexp(amax)                       # 448 = 0.875 * 2^9
        s = torch.exp2((e - 9 + (m > 0.875)).double()).float()
    else:
        s = amax / torch.full_like(amax, QMAX[fmt])
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _quantise(x, group, fmt):
    """Codes as they are stored (int8, float8, or two 4-bit codes to a byte) and scales of a float32 map [N, H, W, C]."""
    n, h, w, c = x.shape
    t = x.float().view(n, h, w, c // group, group)
    s = _scale(t.abs().amax(-1), fmt)
    q = torch.where(s > 0, 1.0, 0.0).unsqueeze(-1) * t.double() / torch.where(s > 0, s, torch.ones_like(s)).double().unsqueeze(-1)
    q = q.view(n, h, w, c)
    if fmt == "e4m3":
        return q.float().to(torch.float8_e4m3fn), s
    q = q.round().clamp(-QMAX[fmt], QMAX[fmt]).to(torch.int8)
    if fmt == "s4":
        q = q.view(n, h, w, c // 2, 2).to(torch.uint8) & 15
        q = q[..., 0] | (q[..., 1] << 4)
    return q, s


def _values(codes, scales, fmt):
    """The float32 values that codes stand for, [..., C]."""
    if fmt == "s4":
        two = torch.stack((codes & 15, codes >> 4), -1).view(*codes.shape[:-1], -1).to(torch.int8)
        codes = torch.where(two > 7, two - 16, two)
    c = codes.float()
    return (c.view(*scales.shape, -1) * scales.unsqueeze(-1)).view(c.shape)


def _tokens(s):
    """Flat token ids [T] (of all batch items) under the tile list."""
    case = s["case"]
    n, h, w, b = case["n"], case["h"], case["w"], case["block"]
    if s["idx"] is None:
        return None
    o = torch.arange(b, device="cuda")
    y = s["idx"][: s["m"], 0].long()[:, None, None] + o[None, :, None]
    x = s["idx"][: s["m"], 1].long()[:, None, None] + o[None, None, :]
    t = (y * w + x)[(y < h) & (x < w)]
    return (torch.arange(n, device="cuda")[:, None] * (h * w) + t[None]).reshape(-1)


def _run_cache(s):
    case, tok = s["case"], _tokens(s)
    n, h, w, c = s["x"].shape
    x = s["x"].view(n * h * w, 1, 1, c)
    codes, scales, y = (s[k].view(n * h * w, 1, 1, -1) for k in ("codes", "scales", "y"))
    if tok is not None:
        x = x[tok]
    new_codes, new_scales = _quantise(x, case["group"], case["fmt"])
    if tok is None:
        codes.copy_(new_codes)
        scales.copy_(new_scales)
        y.copy_(_values(codes, scales, case["fmt"]).to(y.dtype))
    else:
        codes.view(torch.uint8)[tok] = new_codes.view(torch.uint8)
        scales[tok] = new_scales
        y[tok] = _values(codes.view(torch.uint8)[tok].view(codes.dtype), scales[tok], case["fmt"]).to(y.dtype)
    return dict(scales=s["scales"], y=s["y"])


def _run_linear(s):
    tok = _tokens(s)
    n, h, w, co = s["y"].shape
    a, sa = s["a"][0].view(n * h * w, -1), s["a"][1].view(n * h * w, 1)
    y = s["y"].view(n * h * w, co)
    if tok is not None:
        a, sa = a[tok], sa[tok]
    # a sum of 1024 products of 8-bit integers stays below 2^24: in parts of so many channels float32 sums are exact
    parts = [p for p in range(0, a.shape[1], 1024)]
    acc = sum((a[:, p:p + 1024].float() @ s["w"][0].view(co, -1)[:, p:p + 1024].float().T).double() for p in parts)
    r = (acc * sa.double() * s["w"][1].view(1, co).double()).float()
    if s["bias"] is not None:
        r = r + s["bias"]
    if s["residual"] is not None:
        res = s["residual"].view(n * h * w, co)
        r = r + (res if tok is None else res[tok]).float()
    if tok is None:
        y.copy_(r.to(y.dtype))
    else:
        y[tok] = r.to(y.dtype)
    return s["y"]


def _run_attention(s):
    case, tok = s["case"], _tokens(s)
    n, h, w, d = s["q"].shape
    heads, keys = case["heads"], case["keys"]
    q = s["q"].view(n * h * w, d)
    q = (q if tok is None else q[tok]).float().view(n, -1, heads, case["dh"]).transpose(1, 2)
    k = _values(*s["k"], case["fmt"]).view(n, keys, heads, case["dh"]).transpose(1, 2)
    v = _values(*s["v"], case["fmt"]).view(n, keys, heads, case["dv"]).transpose(1, 2)
    p = q @ k.transpose(2, 3) / math.sqrt(case["dh"])
    if s["lens"] is not None:
        gone = torch.arange(keys, device="cuda")[None, :] >= s["lens"][:, None]
        p = p.masked_fill(gone[:, None, None, :], -math.inf)
    m = p.amax(-1, keepdim=True)
    p = torch.exp(p - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.transpose(1, 2).reshape(-1, heads * case["dv"]).to(torch.bfloat16)
    flat = s["o"].view(n * h * w, -1)
    if tok is None:
        flat.copy_(o)
    else:
        flat[tok] = o
    return s["o"]


# ------------------------------------------------------------------ the package's calls

def _run_own(s):
    import spatially_sparse_incremental_b200 as sige

    case = s["case"]
    where = dict(idx=s["idx"], count=s["count"], capacity=s["cap"], block=case["block"]) if s["idx"] is not None else {}
    if case["op"] == "cache":
        cache = sige.QCache(s["codes"], s["scales"], case["fmt"])
        sige.sige_qcache_write(s["x"], cache, **where)
        sige.sige_qcache_read(cache, s["y"], **where)
        return dict(scales=s["scales"], y=s["y"])
    if case["op"] == "linear":
        return sige.sige_qlinear(sige.QCache(*s["a"], "s8"), sige.QCache(*s["w"], "s8"), s["bias"], s["y"],
                                   residual=s["residual"], workspace=s["workspace"], **where)
    k, v = sige.QCache(*s["k"], case["fmt"]), sige.QCache(*s["v"], case["fmt"])
    return sige.sige_attention_qcache(s["q"], k, v, case["heads"], s["o"], key_counts=s["lens"], workspace=s["workspace"],
                                      **where)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _run_cache(state) if op == "cache" else _run_linear(state) if op == "linear" else _run_attention(state)


# ------------------------------------------------------------------ work and exact values

def _n_tokens(case):
    """Tokens of a pass (clipped edge tiles counted whole where they are listed)."""
    n, h, w, b = case["n"], case["h"], case["w"], case["block"]
    return n * h * w if case["tiles"] < 0 else n * min(h * w, case["tiles"] * b * b)


def work(case):
    t = _n_tokens(case)
    if case["op"] == "cache":
        e = 2 if case["dtype"] == "bf16" else 4
        code = 0.5 if case["fmt"] == "s4" else 1.0
        c = case["c"]
        return dict(bytes=t * (2 * c * e + 2 * (c * code + 4 * c / case["group"])), flops=0)
    if case["op"] == "linear":
        e = 2 if case["dtype"] == "bf16" else 4
        c, co = case["c"], case["c_out"]
        return dict(bytes=t * (c + 4) + co * (c + 4) + t * co * e * (1 + bool(case["residual"])) + 4 * co * bool(case["bias"]),
                    flops=2 * t * c * co)
    d, dv, keys = case["heads"] * case["dh"], case["heads"] * case["dv"], case["keys"]
    code = 0.5 if case["fmt"] == "s4" else 1.0
    return dict(bytes=t * 2 * (d + dv) + case["n"] * keys * ((d + dv) * code + 8 * case["heads"]),
                flops=2 * t * keys * (d + dv))


def exact(case, seed):
    """The operators' values in 64 bits, from their definitions, token by token of the batch items."""
    s = prepare(case, seed)
    n, h, w, b = case["n"], case["h"], case["w"], case["block"]
    active = torch.ones((h, w), dtype=torch.bool, device="cuda")
    if s["idx"] is not None:
        active.zero_()
        for y0, x0 in s["idx"][: s["m"]].tolist():
            active[y0:y0 + b, x0:x0 + b] = True

    def decode(codes, fmt):
        if fmt != "s4":
            return codes.double()
        low, high = (codes % 16).double(), torch.div(codes, 16, rounding_mode="floor").double()
        both = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.float64, device="cuda")
        both[..., 0::2], both[..., 1::2] = low, high
        return both - 16.0 * (both >= 8)

    if case["op"] == "cache":
        scales, y = s["scales"].clone(), s["y"].double()
        for i in range(n):
            t = s["x"][i][active].double().unflatten(-1, (-1, case["group"]))
            top = t.abs().max(-1).values
            if case["fmt"] == "e4m3":
                step = torch.pow(2.0, torch.ceil(torch.log2(top / 448.0))).float().double()   # a power of two, exactly
                step = torch.where(top > 448.0 * step, 2 * step, torch.where(top <= 224.0 * step, step / 2, step))
            else:
                step = (top / QMAX[case["fmt"]]).float().double()
            step = torch.where((top > 0) & (step >= 2.0 ** -126), step, torch.zeros_like(step))
            u = torch.where(step[..., None] > 0, t / step[..., None], torch.zeros_like(t))
            if case["fmt"] == "e4m3":
                # spacing 2^(e-3) of normal values 2^e .., 2^-9 below 2^-6
                grid = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6))) - 3).float().double()
                u = torch.round(u / grid) * grid
            else:
                u = torch.round(u)
            scales[i][active] = step.float()
            y[i][active] = (u * step[..., None]).flatten(-2)
        return dict(scales=scales, y=y)
    if case["op"] == "linear":
        y = s["y"].double()
        wd = s["w"][0].double().reshape(case["c_out"], -1) * s["w"][1].double().reshape(-1, 1)
        for i in range(n):
            r = (s["a"][0][i][active].double() * s["a"][1][i][active].double()) @ wd.T
            if s["bias"] is not None:
                r += s["bias"].double()
            if s["residual"] is not None:
                r += s["residual"][i][active].double()
            y[i][active] = r
        return y
    o = s["o"].double()
    for i in range(n):
        length = case["keys"] if s["lens"] is None else int(s["lens"][i])
        rows = torch.zeros((int(active.sum()), case["heads"] * case["dv"]), dtype=torch.float64, device="cuda")
        for j in range(case["heads"] if length else 0):
            at, av = slice(j * case["dh"], (j + 1) * case["dh"]), slice(j * case["dv"], (j + 1) * case["dv"])
            k = decode(s["k"][0][i, :length, 0], case["fmt"])[:, at] * s["k"][1][i, :length, 0, j:j + 1].double()
            v = decode(s["v"][0][i, :length, 0], case["fmt"])[:, av] * s["v"][1][i, :length, 0, j:j + 1].double()
            rows[:, av] = torch.softmax(s["q"][i][active][:, at].double() @ k.T / math.sqrt(case["dh"]), -1) @ v
        o[i][active] = rows
    return o
