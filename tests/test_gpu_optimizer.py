"""GPU parity of the global gradient norm and of the AdamW step against
float64 (oracle.training).

Bounds, with e = 2^-24 (half a step of fp32): m is two products and a sum of
constants that are themselves rounded, at most 4e (|beta1 m| + |(1 - beta1) g|);
v likewise at most 6e of itself; the update u = lr m / (1 - beta1^t) / (sqrt(v /
(1 - beta2^t)) + eps) adds at most 16e |u| (a quotient to 2 ulp, a root, five
products and sums, and half of v's error) to what m's error makes of it; p adds
3e (|p| + |u|).  A 16-bit parameter is off by half a step of its type more:
that is relative to the value for normal numbers, and 2^-25 for fp16 values
below 2^-14, whose step is 2^-24 throughout."""
import math

import numpy as np
import pytest

from oracle import training as TR

pytestmark = pytest.mark.gpu

BAD_IDS, INVALID = 8, 1
E = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 0.0}
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8)


@pytest.fixture(scope="module", autouse=True)
def built():
    from hstu_sequential_transducer_layer_b200.build import build
    build()


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def _ws(n):
    import torch
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")


def _np(x):
    return x.detach().double().cpu().numpy()


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("sizes", [[], [0], [1], [3, 0, 5], [4096], [4097, 8191, 7],
                                   [300000, 1, 77777], [5] * 300, [3] * 600])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_norm(sizes, dtype):
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    g = [torch.randn(n, device="cuda").to(_dt(dtype)) for n in sizes]
    lst = H.GradTensors([dict(grad=x) for x in g])
    out, ws = torch.full((2,), -1.0, device="cuda"), _ws(H.hstu_grad_norm_workspace_size())
    for max_norm in (0.5, 1e9):
        H.hstu_grad_norm(lst, max_norm, out, ws)
        n, c = TR.grad_norm([_np(x) for x in g], max_norm)
        got = out.tolist()
        # fp64 sums: only the rounding to fp32 shows
        assert abs(got[0] - n) <= 1.01 * E * n and abs(got[1] - c) <= 1.01 * E * c
        assert H.hstu_read_status(ws) == 0


def test_norm_extremes_and_rows():
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    out, ws = torch.zeros(2, device="cuda"), _ws(H.hstu_grad_norm_workspace_size())
    big = torch.tensor([3e30, 4e30], device="cuda")
    small = torch.tensor([3e-30, 4e-30], device="cuda")
    for x, n in ((big, 5e30), (small, 5e-30)):           # squares beyond fp32's range
        H.hstu_grad_norm(H.GradTensors([dict(grad=x)]), 1.0, out, ws)
        assert abs(float(out[0]) / n - 1) < 1e-6
        assert abs(float(out[1]) - min(1.0, 1 / n)) <= 1e-6 * min(1.0, 1 / n)
    H.hstu_grad_norm(H.GradTensors([dict(grad=torch.zeros(9, device="cuda"))]), 1.0, out, ws)
    assert out.tolist() == [0.0, 1.0]
    H.hstu_grad_norm(H.GradTensors([dict(grad=big)]), math.inf, out, ws)
    assert float(out[1]) == 1.0
    for x in (math.nan, math.inf, -math.inf):
        bad = torch.ones(10000, device="cuda")
        bad[7777] = x
        H.hstu_grad_norm(H.GradTensors([dict(grad=bad), dict(grad=big)]), 1.0, out, ws)
        assert math.isnan(float(out[1])) and not math.isfinite(float(out[0]))
    # only the first n_rows rows count; a count outside [0, rows] is cut
    rows = torch.randn(100, 33, device="cuda")
    rows[60:] = math.nan
    n = torch.zeros(1, dtype=torch.int64, device="cuda")
    lst = H.GradTensors([dict(grad=rows, n_rows=n), dict(grad=big[:1] * 0 + 2)])
    for k in (0, 1, 59, 60, -4):
        n.fill_(k)
        H.hstu_grad_norm(lst, 1.0, out, ws)
        want = TR.grad_norm([_np(rows[:max(k, 0)]), np.array([2.0])], 1.0)
        assert abs(float(out[0]) - want[0]) <= 1.01 * E * want[0]
    n.fill_(1 << 60)
    H.hstu_grad_norm(lst, 1.0, out, ws)
    assert math.isnan(float(out[0]))                      # all 100 rows, the NaN ones among them


# ---------------------------------------------------------------- AdamW
def _bounds(p, g, m, v, step, wd, gs, h=HYPER):
    """(p, m, v) in float64 and how far fp32 may be from each."""
    rp, rm, rv = TR.adamw(p, g, m, v, step, h["lr"], h["beta1"], h["beta2"], h["eps"], wd, gs)
    dm = 4 * E * (np.abs(h["beta1"] * m) + np.abs((1 - h["beta1"]) * g * gs))
    den = np.sqrt(rv / (1 - h["beta2"] ** step)) + h["eps"]
    unit = h["lr"] / (1 - h["beta1"] ** step) / den
    u = unit * np.abs(rm)
    dp = unit * dm + 16 * E * u + 3 * E * (np.abs(p) + u)
    return rp, rm, rv, dp, dm, 6 * E * rv


def _make(n, param, grad, master, bits, seed, shape=None, zero=False):
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda s: torch.randn(*(shape or (n,)), device="cuda", generator=g) * s  # noqa: E731
    p = r(1.0)
    t = dict(param=p.to(_dt(param)), grad=r(0.1).to(_dt(grad)))
    if master:
        t["master"] = p.clone()
    if bits == 32:
        t["m"], t["v"] = r(0.02) * (not zero), (r(0.02) * (not zero)).square()
    else:
        s = shape or (n,)
        k = H.state_scales(s)
        code = lambda top: torch.randint(0, top, s, device="cuda", generator=g)  # noqa: E731
        sign = code(2) * 128
        t["m"] = ((code(0x7E) + sign) * (not zero)).to(torch.uint8)
        t["v"] = (code(0x7E) * (not zero)).to(torch.uint8)
        for q, e in (("m_scale", 118), ("v_scale", 117)):
            t[q] = (torch.randint(e - 2, e + 3, (k,), device="cuda", generator=g)
                    * (not zero)).to(torch.uint8)
    return t


def _copy(t):
    return {k: (x.clone() if hasattr(x, "clone") else x) for k, x in t.items()}


@pytest.mark.parametrize("shape", [(256 * 9,), (256 * 9 + 101,), (40, 257), (40, 512)])
def test_states_are_not_contracted(shape):
    """fp32 m and v equal products and sums that are rounded one by one, bit for bit."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    t = _make(0, "f32", "f32", False, 32, 3, shape=shape)
    if len(shape) == 2:
        t["row_ids"] = torch.arange(shape[0], device="cuda")
        t["n_rows"] = torch.tensor([shape[0]], device="cuda")
    g, m, v = (t[k].cpu().numpy() for k in ("grad", "m", "v"))
    ws = _ws(256)
    H.hstu_adamw_step(H.AdamWTensors([t]), ws, step=2, **HYPER)
    assert H.hstu_read_status(ws) == 0
    f = np.float32
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    rm = m * f(b1) + g * f(1 - b1)
    rv = v * f(b2) + g * g * f(1 - b2)
    assert rm.dtype == f and rv.dtype == f
    np.testing.assert_array_equal(t["m"].cpu().numpy(), rm)
    np.testing.assert_array_equal(t["v"].cpu().numpy(), rv)


def _blocks(x, rows=None):
    """Array [blocks, 256] of a tensor (of each row of it), zeros behind the end."""
    x = x.reshape(1, -1) if rows is None else x.reshape(rows, -1)
    n = -(-x.shape[1] // 256) * 256
    return np.pad(x, ((0, 0), (0, n - x.shape[1]))).reshape(-1, 256)


def _check(old, new, step, gs, ordinal, seed, hyper=HYPER, name="bf16"):
    """One dense tensor: new against the oracle's step of old."""
    import torch
    wd = old.get("weight_decay", 0.0)
    p = _np(old["master"] if "master" in old else old["param"])
    g = _np(old["grad"])
    if old["m"].dtype == torch.float32:
        m, v = _np(old["m"]), _np(old["v"])
    else:
        co = {k: old[k].view(torch.uint8).cpu().numpy() for k in ("m", "v", "m_scale", "v_scale")}
        m = TR.decode(_blocks(co["m"]), co["m_scale"]).ravel()[:p.size]
        v = TR.decode(_blocks(co["v"]), co["v_scale"]).ravel()[:p.size] ** 2
    rp, rm, rv, dp, dm, dv = _bounds(p, g, m, v, step, wd, gs, hyper)
    if "master" in new:
        assert (np.abs(_np(new["master"]) - rp) <= dp).all()
    assert (np.abs(_np(new["param"]) - rp) <= dp * 1.01 + HALF[name] * np.abs(rp) + TINY[name]).all()
    if "copy_f16" in new:
        want = new["param"].float().clamp(-65504, 65504).half()
        assert torch.equal(new["copy_f16"], want)
    if old["m"].dtype == torch.float32:
        assert (np.abs(_np(new["m"]) - rm) <= dm).all() and (np.abs(_np(new["v"]) - rv) <= dv).all()
        return
    nb = -(-p.size // 256)
    cm, sm, cr, sr = TR.adamw_step_8bit(
        _blocks(co["m"]), co["m_scale"], _blocks(co["v"]), co["v_scale"], _blocks(g).astype(np.float32),
        seed, step, ordinal, np.arange(nb), hyper["beta1"], hyper["beta2"], np.float32(gs))
    for k, want in (("m", cm), ("v", cr)):
        np.testing.assert_array_equal(new[k].view(torch.uint8).cpu().numpy(), want.ravel()[:p.size])
    np.testing.assert_array_equal(new["m_scale"].cpu().numpy(), sm)
    np.testing.assert_array_equal(new["v_scale"].cpu().numpy(), sr)


SIZES = [1, 3, 255, 256, 257, 2047, 2048, 2051, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", [("bf16", "f32", True), ("bf16", "bf16", False),
                                               ("f32", "f32", False), ("f16", "f16", True),
                                               ("f32", "bf16", False), ("f16", "f32", False),
                                               ("bf16", "f32", False)])
def test_adamw_step(bits, param, grad, master):
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    ts = []
    for i, n in enumerate(SIZES):
        t = _make(n, param, grad, master, bits, seed=i)
        t["weight_decay"] = 0.1 * (i % 2)
        if i % 3 != 1:
            t["copy_f16"] = torch.zeros(n, dtype=torch.float16, device="cuda")
        ts.append(t)
    old = [_copy(t) for t in ts]
    lst, ws = H.AdamWTensors(ts), _ws(256)
    gs = torch.tensor([0.37], device="cuda")
    for step in (1, 12345):
        H.hstu_adamw_step(lst, ws, step=step, grad_scale=gs, seed=99, **HYPER)
        assert H.hstu_read_status(ws) == 0
        for i, t in enumerate(ts):
            _check(old[i], t, step, float(gs), i, 99, name=param)
        old = [_copy(t) for t in ts]


def test_adamw_first_step_from_zeros_and_large_values():
    """Zero states; then gradients and parameters over many magnitudes (a
    parameter beyond fp16's range saturates its fp16 copy)."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    for bits in (32, 8):
        t = _make(3000, "bf16", "f32", True, bits, 3, zero=True)
        t["grad"] *= torch.exp(torch.linspace(-18, 18, 3000, device="cuda"))
        t["grad"][:256] = 0
        t["master"][5], t["param"][5] = 1e6, 1e6
        t["copy_f16"] = torch.zeros(3000, dtype=torch.float16, device="cuda")
        old = _copy(t)
        H.hstu_adamw_step(H.AdamWTensors([t]), _ws(256), step=1, **HYPER)
        _check(old, t, 1, 1.0, 0, 0)
        assert float(t["copy_f16"][5]) == 65504.0


def test_many_tensors():
    """More tensors than one launch takes, empty ones among them."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    ts = [_make(1 + 37 * (i % 9), "bf16", "f32", True, 8 if i % 2 else 32, i) for i in range(600)]
    for i in (0, 100, 300, 599):
        ts[i] = {k: x[:0].contiguous() for k, x in ts[i].items()}
    old = [_copy(t) for t in ts]
    lst, ws = H.AdamWTensors(ts), _ws(256)
    H.hstu_adamw_step(lst, ws, step=7, seed=5, **HYPER)
    for i, t in enumerate(ts):
        if t["param"].numel():
            _check(old[i], t, 7, 1.0, i, 5)
    H.hstu_adamw_step(H.AdamWTensors([]), ws, step=1, lr=1e-3)
    assert H.hstu_read_status(ws) == 0


@pytest.mark.parametrize("tail", [0, 5, 256 * 3, 256 * 7 + 255])
def test_large_tensors(tail):
    """Lists large enough for a warp to take several consecutive blocks at a
    time: blocks at the start, at the end (whole and not) and all over a large
    8-bit tensor, with small tensors of either width around it."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    n = 20_000_000 - 20_000_000 % 2048 + tail
    ts = [_make(700, "bf16", "f32", True, 8, 1), _make(n, "bf16", "f32", True, 8, 2),
          _make(5000, "f32", "f32", False, 32, 3), _make(2000, "bf16", "bf16", False, 8, 4)]
    old = [_copy(t) for t in ts]
    ws = _ws(256)
    H.hstu_adamw_step(H.AdamWTensors(ts), ws, step=9, seed=8, **HYPER)
    assert H.hstu_read_status(ws) == 0
    for i in (0, 2, 3):
        _check(old[i], ts[i], 9, 1.0, i, 8, name="f32" if i == 2 else "bf16")
    nb = -(-n // 256)
    rng = np.random.default_rng(tail)
    pick = np.unique(np.concatenate([np.arange(40), np.arange(nb - 40, nb), rng.integers(0, nb, 2000)]))
    at = (pick[:, None] * 256 + np.arange(256)).ravel()
    live = at < n
    idx = torch.from_numpy(np.minimum(at, n - 1)).cuda()

    def cut(t, k):
        x = t[k].view(torch.uint8)[idx] if k in ("m", "v") else t[k][idx]
        x = x.cpu().numpy() if k in ("m", "v") else _np(x)
        return np.where(live, x, 0).reshape(-1, 256)
    o, t = old[1], ts[1]
    sc = {k: o[k].cpu().numpy()[pick] for k in ("m_scale", "v_scale")}
    cm, sm, cr, sr = TR.adamw_step_8bit(cut(o, "m"), sc["m_scale"], cut(o, "v"), sc["v_scale"],
                                        cut(o, "grad").astype(np.float32), 8, 9, 1, pick,
                                        HYPER["beta1"], HYPER["beta2"])
    np.testing.assert_array_equal(cut(t, "m").ravel()[live], cm.ravel()[live])
    np.testing.assert_array_equal(cut(t, "v").ravel()[live], cr.ravel()[live])
    np.testing.assert_array_equal(t["m_scale"].cpu().numpy()[pick], sm)
    np.testing.assert_array_equal(t["v_scale"].cpu().numpy()[pick], sr)
    m, r = TR.decode(cut(o, "m"), sc["m_scale"]), TR.decode(cut(o, "v"), sc["v_scale"])
    rp, _, _, dp, _, _ = _bounds(cut(o, "master"), cut(o, "grad"), m, r ** 2, 9, 0.0, 1.0)
    assert (np.abs(cut(t, "master") - rp) <= dp).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("R,d,U,cap", [(1, 1, 1, 1), (9, 50, 0, 4), (9, 50, 9, 9), (300, 257, 77, 90),
                                       (300, 256, 77, 300), (1000, 8, 400, 401), (64, 1024, 33, 50)])
def test_touched_rows(R, d, U, cap, bits):
    """Rows of a table: those of the list as the dense step would, every other
    row's parameter and state as before."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    t = _make(0, "bf16", "f32", True, bits, R + d, shape=(R, d))
    rng = np.random.default_rng(R)
    rows = np.sort(rng.permutation(R)[:U])
    t["grad"] = torch.full((cap, d), math.nan, device="cuda")
    t["grad"][:U] = torch.randn(U, d, device="cuda") * 0.1
    t["row_ids"] = torch.full((cap,), -1, dtype=torch.int64, device="cuda")
    t["row_ids"][:U] = torch.from_numpy(rows).cuda()
    t["n_rows"] = torch.tensor([U], device="cuda")
    t["weight_decay"], t["copy_f16"] = 0.1, torch.zeros(R, d, dtype=torch.float16, device="cuda")
    old = _copy(t)
    ws = _ws(256)
    dense = _make(100, "f32", "f32", False, bits, 1)      # the table is the list's second tensor
    H.hstu_adamw_step(H.AdamWTensors([dense, t]), ws, step=4, seed=11, **HYPER)
    assert H.hstu_read_status(ws) == 0
    rest = np.setdiff1d(np.arange(R), rows)
    nb = -(-d // 256)
    for k in ("param", "master", "m", "v", "copy_f16"):
        assert torch.equal(t[k].view(R, d)[rest], old[k].view(R, d)[rest])
    if U == 0:
        return
    g = _np(t["grad"][:U])
    p = _np(old["master"])[rows]
    if bits == 32:
        m, v = _np(old["m"])[rows], _np(old["v"])[rows]
    else:
        cod = {k: old[k].cpu().numpy() for k in ("m", "v", "m_scale", "v_scale")}
        at = (rows[:, None] * nb + np.arange(nb)).ravel()
        wide = {k: _blocks(cod[k][rows], U) for k in ("m", "v")}
        dec = lambda k: TR.decode(wide[k], cod[k + "_scale"][at]).reshape(U, -1)[:, :d]  # noqa: E731
        m, v = dec("m"), dec("v") ** 2
    rp, rm, rv, dp, dm, dv = _bounds(p, g, m, v, 4, 0.1, 1.0)
    assert (np.abs(_np(t["master"])[rows] - rp) <= dp).all()
    assert (np.abs(_np(t["param"])[rows] - rp) <= dp * 1.01 + 2.0 ** -8 * np.abs(rp)).all()
    if bits == 32:
        assert (np.abs(_np(t["m"])[rows] - rm) <= dm).all()
        assert (np.abs(_np(t["v"])[rows] - rv) <= dv).all()
        return
    cm, sm, cr, sr = TR.adamw_step_8bit(wide["m"], cod["m_scale"][at], wide["v"], cod["v_scale"][at],
                                        _blocks(g, U).astype(np.float32), 11, 4, 1, at,
                                        HYPER["beta1"], HYPER["beta2"])
    cut = lambda c: c.reshape(U, -1)[:, :d]  # noqa: E731
    np.testing.assert_array_equal(t["m"].cpu().numpy()[rows], cut(cm))
    np.testing.assert_array_equal(t["v"].cpu().numpy()[rows], cut(cr))
    np.testing.assert_array_equal(t["m_scale"].cpu().numpy()[at], sm)
    np.testing.assert_array_equal(t["v_scale"].cpu().numpy()[at], sr)
    others = np.setdiff1d(np.arange(R * nb), at)
    assert torch.equal(t["m_scale"][others], old["m_scale"][others])


@pytest.mark.parametrize("bits", [32, 8])
def test_tables_of_all_types_in_one_list(bits):
    """Touched rows of tables with and without masters: the bits that a dense
    step gives these rows (with rows of 512 the blocks of 256 are the same)."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    R, d, U = 700, 512, 260
    types = [("bf16", "f32", False), ("bf16", "bf16", False), ("f32", "f32", False),
             ("bf16", "f32", True), ("f16", "f32", False)]
    gen = torch.Generator(device="cuda").manual_seed(5)
    sparse, dense, rows = [], [], []
    for i, (p, g, master) in enumerate(types):
        t = _make(0, p, g, master, bits, 10 + i, shape=(R, d))
        dense.append(_copy(t))
        ids = torch.randperm(R, device="cuda", generator=gen)[:U].sort().values
        t["grad"], t["row_ids"] = t["grad"][ids].contiguous(), ids
        t["n_rows"] = torch.tensor([U], device="cuda")
        sparse.append(t)
        rows.append(ids)
    ws = _ws(256)
    for ts in (sparse, dense):
        H.hstu_adamw_step(H.AdamWTensors(ts), ws, step=3, seed=2, **HYPER)
        assert H.hstu_read_status(ws) == 0
    for t, o, ids in zip(sparse, dense, rows):
        for k in ("param", "master", "m", "v"):
            if k in t:
                assert torch.equal(t[k].view(R, d)[ids].view(torch.uint8), o[k].view(R, d)[ids].view(torch.uint8))
        if bits == 8:
            for k in ("m_scale", "v_scale"):
                assert torch.equal(t[k].view(R, 2)[ids], o[k].view(R, 2)[ids])


@pytest.mark.parametrize("n", [0, 2])
def test_row_count_of_another_size_is_refused(n):
    """An empty count has a null address, which would mean a dense gradient."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    t = _make(0, "f32", "f32", False, 32, 1, shape=(10, 16))
    t["row_ids"] = torch.arange(10, device="cuda")
    t["n_rows"] = torch.zeros(n, dtype=torch.int64, device="cuda")
    with pytest.raises(H.HstuError):
        H.AdamWTensors([t])
    with pytest.raises(H.HstuError):
        H.GradTensors([dict(grad=t["grad"], n_rows=t["n_rows"])])


@pytest.mark.parametrize("bits,d", [(32, 16), (8, 16), (8, 512), (32, 512), (8, 7)])
def test_bad_rows_are_skipped_and_reported(bits, d):
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    for ids, n, good in (([1, 5, 20], 3, [1, 5]), ([-1, 3, 4], 3, [3, 4]), ([2, 2, 6], 3, [2, 6]),
                         ([7, 3, 8], 3, [7, 8]), ([1, 2, 3], 4, [1, 2, 3]), ([1, 2, 3], -1, [])):
        t = _make(0, "f32", "f32", False, bits, 1, shape=(10, d))
        t["grad"] = torch.ones(3, d, device="cuda")
        t["row_ids"] = torch.tensor(ids, device="cuda")
        t["n_rows"] = torch.tensor([n], device="cuda")
        old, ws = _copy(t), _ws(256)
        H.hstu_adamw_step(H.AdamWTensors([t]), ws, step=1, **HYPER)
        assert H.hstu_read_status(ws) == BAD_IDS, ids
        changed = (t["param"] != old["param"]).any(1).nonzero().flatten().tolist()
        assert changed == good, (ids, changed)
        t["row_ids"].copy_(torch.tensor([0, 4, 9], device="cuda"))
        t["n_rows"].fill_(3)
        H.hstu_adamw_step(H.AdamWTensors([t]), ws, step=2, **HYPER)
        assert H.hstu_read_status(ws) == 0


def test_step_is_skipped_when_the_scale_is_not_finite():
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    for bits in (32, 8):
        t = _make(1000, "bf16", "f32", True, bits, 2)
        old, lst, ws = _copy(t), H.AdamWTensors([t]), _ws(256)
        for x in (math.nan, math.inf, -math.inf):
            H.hstu_adamw_step(lst, ws, step=1, lr=1.0, grad_scale=torch.tensor([x], device="cuda"))
        zero = torch.zeros(1, dtype=torch.int64, device="cuda")
        H.hstu_adamw_step(lst, ws, step=zero, lr=1.0)
        assert H.hstu_read_status(ws) == INVALID
        for k, x in old.items():
            assert torch.equal(t[k], x)


def test_not_finite_gradients_stay_in_their_element():
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    for bits in (32, 8):
        t = _make(512, "f32", "f32", False, bits, 2)
        t["grad"][7], t["grad"][300] = math.nan, math.inf
        clean = _copy(t)
        clean["grad"][7], clean["grad"][300] = 0, 0
        ws = _ws(256)
        H.hstu_adamw_step(H.AdamWTensors([t]), ws, step=3, seed=1, **HYPER)
        H.hstu_adamw_step(H.AdamWTensors([clean]), ws, step=3, seed=1, **HYPER)
        assert torch.isnan(t["param"][7]) and torch.isnan(t["param"][300])
        keep = torch.ones(512, dtype=torch.bool, device="cuda")
        keep[7] = keep[300] = False
        for k in ("param", "m", "v"):
            assert torch.equal(t[k][keep], clean[k][keep])
        if bits == 8:
            assert (t["m"][~keep] & 0x7F == 0x7F).all() and (t["v"][~keep] == 0x7F).all()


def test_fp16_copy_is_what_the_conversion_gives():
    """The copy of each new bf16 parameter, bit for bit as hstu_bf16_to_f16:
    values beyond fp16's range, subnormals, zeros, NaN; whole blocks and the
    end of a tensor."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    n = 1000
    p = torch.exp(torch.linspace(-40, 40, n, device="cuda")) * \
        torch.tensor([1.0, -1.0], device="cuda").repeat(n // 2)
    p[3], p[4], p[998] = math.nan, 0.0, math.nan
    z = lambda: torch.zeros(n, device="cuda")  # noqa: E731
    t = dict(param=p.bfloat16(), master=p.clone(), grad=z(), m=z(), v=z(),
             copy_f16=torch.zeros(n, dtype=torch.float16, device="cuda"))
    H.hstu_adamw_step(H.AdamWTensors([t]), _ws(256), step=1, **HYPER)
    want = torch.zeros_like(t["copy_f16"])
    H.hstu_bf16_to_f16(t["param"], want)
    assert torch.equal(t["copy_f16"].view(torch.int16), want.view(torch.int16))
    assert torch.isnan(want[3]) and torch.isnan(want[998]) and float(want[n - 4]) == 65504.0


def test_small_second_moments_keep_moving():
    """v moves by 1e-3 of itself per step, far less than a code step s <= 2^-3 of
    its root: under rounding to nearest it would stand still.  100 steps with
    one gradient, then 1500 with none for half of the elements: their mean v
    falls to 0.999^1500 = 0.22 of what it was.  The stored root r is right in
    the mean; its variance, s^2 q (1 - q) r^2 per step for a move of q code
    steps, biases v = r^2 upwards: while v grows linearly q = 1 / (2 t s), and
    a bias of step t weighs t / 100 at step 100, so at most s / 2 = 6.3%; while
    it falls q = 5e-4 / s, so at most 1500 * 5e-4 s = 9.4%; together (factors)
    under 17%.  The mean over 2^15 elements with a spread of at most 100% adds
    5 / 2^7.5 = 2.8%."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    n = 1 << 16
    t = _make(n, "f32", "f32", False, 8, 0, zero=True)
    t["grad"].fill_(0.5)
    lst, ws = H.AdamWTensors([t]), _ws(256)
    v = 0.0
    for step in range(1, 1601):
        if step == 101:
            t["grad"][n // 2:] = 0.0
        H.hstu_adamw_step(lst, ws, step=step, lr=1e-3, seed=17)
        v = 0.999 * v + (0.001 * 0.25 if step <= 100 else 0.0)
    scale = torch.exp2(t["v_scale"].float() - 127).repeat_interleave(256)
    r = t["v"].view(torch.float8_e4m3fn).float() * scale
    mean = float(r[n // 2:].double().square().mean())
    assert -0.028 <= mean / v - 1 <= 0.20, (mean, v)


def test_captured_step_reads_step_and_rate_from_the_device():
    """A captured norm and step, replayed with a step counter, a rate and
    gradients that change on the device, equals the eager steps."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    ts = [_make(n, "bf16", "f32", True, b, n) for n, b in ((5000, 32), (777, 8), (1, 32))]
    eager = [_copy(t) for t in ts]
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.zeros(1, device="cuda")
    out, out2 = torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda")
    nws, ws = _ws(H.hstu_grad_norm_workspace_size()), _ws(256)
    lst, elst = H.AdamWTensors(ts), H.AdamWTensors(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        H.hstu_grad_norm(lst, 0.5, out, nws)
        H.hstu_adamw_step(lst, ws, lr=lr, step=step, grad_scale=out[1:], seed=4)
    g = torch.Generator(device="cuda").manual_seed(0)
    for k in range(1, 5):
        lr.fill_(2.0 ** -k)
        for a, b in zip(ts, eager):
            a["grad"].normal_(generator=g)
            b["grad"].copy_(a["grad"])
        graph.replay()
        H.hstu_grad_norm(elst, 0.5, out2, nws)
        H.hstu_adamw_step(elst, ws, lr=2.0 ** -k, step=k, grad_scale=out2[1:], seed=4)
        torch.cuda.synchronize()
        assert H.hstu_read_status(ws) == 0 and torch.equal(out, out2)
        for a, b in zip(ts, eager):
            for q in a:
                assert torch.equal(a[q], b[q]), q
    del graph


def test_lists_on_two_streams_at_once():
    """Two lists, each with its own workspace, on two streams."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    ts = [[_make(300_000, "bf16", "f32", True, b, b)] for b in (8, 32)]
    old = [[_copy(t[0])] for t in ts]
    lst, ws = [H.AdamWTensors(t) for t in ts], [_ws(256), _ws(256)]
    out, nws = [torch.zeros(2, device="cuda") for _ in ts], \
        [_ws(H.hstu_grad_norm_workspace_size()) for _ in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    for k in range(2):
        H.hstu_grad_norm(lst[k], 1.0, out[k], nws[k], stream=streams[k])
        H.hstu_adamw_step(lst[k], ws[k], step=1, grad_scale=out[k][1:], seed=2, stream=streams[k],
                          **HYPER)
    torch.cuda.synchronize()
    for k in range(2):
        _check(old[k][0], ts[k][0], 1, float(out[k][1]), 0, 2)


def test_offsets_past_32_bits():
    """A table of more than 2^31 elements: its last rows."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    R, d = 2_200_000, 1024
    z = lambda dt: torch.zeros(R, d, dtype=dt, device="cuda")  # noqa: E731
    t = dict(param=z(torch.bfloat16), m=z(torch.uint8), v=z(torch.uint8),
             m_scale=torch.zeros(R * 4, dtype=torch.uint8, device="cuda"),
             v_scale=torch.zeros(R * 4, dtype=torch.uint8, device="cuda"),
             grad=torch.ones(3, d, device="cuda"),
             row_ids=torch.tensor([0, R - 2, R - 1], device="cuda"),
             n_rows=torch.tensor([3], device="cuda"))
    ws = _ws(256)
    H.hstu_adamw_step(H.AdamWTensors([t]), ws, step=1, lr=0.5)
    assert H.hstu_read_status(ws) == 0
    want = torch.tensor(-0.5, dtype=torch.bfloat16)
    for r in (0, R - 2, R - 1):
        assert (t["param"][r] == want).all() and (t["m_scale"][4 * r:4 * r + 4] > 0).all()
    assert not t["param"][1:R - 2].any() and not t["m"][1:R - 2].any()


def test_norm_of_few_rows_in_a_large_buffer():
    """Rows in use at the start of a buffer of more than 2^31 elements: what lies behind them does not
    count, however far behind; with every row in use all of it does."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    R, d = 2_200_000, 1024
    rows = torch.full((R, d), 2.0, dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(1, dtype=torch.int64, device="cuda")
    lst = H.GradTensors([dict(grad=rows, n_rows=n), dict(grad=torch.full((9,), 2.0, device="cuda"))])
    out, ws = torch.zeros(2, device="cuda"), _ws(H.hstu_grad_norm_workspace_size())
    for k in (0, 1, 100, R - 1, R):
        n.fill_(k)
        H.hstu_grad_norm(lst, 1.0, out, ws)
        want = 2.0 * math.sqrt(k * d + 9)          # every square and sum is exact
        assert H.hstu_read_status(ws) == 0
        assert abs(float(out[0]) - want) <= 1.01 * E * want
        assert abs(float(out[1]) - 1 / want) <= 1.01 * E / want


@pytest.mark.parametrize("n", [0, 1000, 2_000_000])
def test_norm_after_a_failed_call_is_nan(n):
    """In one launch and in two, and with nothing to add up: any status word but HSTU_OK gives NaN, and
    the AdamW step behind it changes nothing."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    t = _make(n, "bf16", "f32", True, 32, 1)
    old, lst = _copy(t), H.AdamWTensors([t] if n else [])
    out, ws, ows = torch.zeros(2, device="cuda"), _ws(H.hstu_grad_norm_workspace_size()), _ws(256)
    after = torch.zeros(64, dtype=torch.int32, device="cuda")
    for word in (5, 6, 7, -1):
        after[0] = word
        H.hstu_grad_norm_after(lst, 1.0, after, out, ws)
        assert torch.isnan(out).all() and H.hstu_read_status(ws) == 0
        H.hstu_adamw_step(lst, ows, step=1, grad_scale=out[1:], **HYPER)
        assert all(torch.equal(t[k], x) for k, x in old.items())
    after[0], after[1:] = 0, 9                     # the rest of a workspace means nothing
    H.hstu_grad_norm_after(lst, 1.0, after, out, ws)
    plain = torch.zeros(2, device="cuda")
    H.hstu_grad_norm(lst, 1.0, plain, ws)
    assert torch.equal(out, plain) and torch.isfinite(out).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capacity", [(0, 0), (4, 0), (0, 4)])
def test_row_list_without_entries(bits, capacity):
    """A row gradient that has no room for a row (of an empty batch): the table stays as it is, the other
    tensors of the list are updated, and a count above its room is reported."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    rows, ids = capacity
    t, dense = _make(0, "bf16", "f32", True, bits, 1, shape=(10, 48)), _make(100, "f32", "f32", False, bits, 2)
    t["grad"] = torch.full((rows, 48), math.nan, device="cuda")
    t["row_ids"] = torch.zeros(ids, dtype=torch.int64, device="cuda")
    t["n_rows"] = torch.zeros(1, dtype=torch.int64, device="cuda")
    old, old_dense = _copy(t), _copy(dense)
    lst, ws = H.AdamWTensors([t, dense]), _ws(256)
    out, nws = torch.zeros(2, device="cuda"), _ws(H.hstu_grad_norm_workspace_size())
    H.hstu_grad_norm(lst, 1e9, out, nws)
    want = TR.grad_norm([_np(dense["grad"])], 1e9)[0]
    assert abs(float(out[0]) - want) <= 1.01 * E * want and float(out[1]) == 1.0
    H.hstu_adamw_step(lst, ws, step=2, seed=3, **HYPER)
    assert H.hstu_read_status(ws) == 0
    assert all(torch.equal(t[k], old[k]) for k in ("param", "master", "m", "v"))
    _check(old_dense, dense, 2, 1.0, 1, 3, name="f32")
    t["n_rows"].fill_(1)
    H.hstu_adamw_step(lst, ws, step=3, seed=3, **HYPER)
    assert H.hstu_read_status(ws) == BAD_IDS
    assert all(torch.equal(t[k], old[k]) for k in ("param", "master", "m", "v"))
