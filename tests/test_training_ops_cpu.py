"""CPU checks of the training-side operators: the oracle against differences,
torch and closed forms, and what the C ABI and its binding refuse before
anything is launched."""
import ctypes
import math

import numpy as np
import pytest

import hstu_sequential_transducer_layer_b200 as H
from hstu_sequential_transducer_layer_b200 import binding as B
from oracle import training as TR


@pytest.fixture(scope="module", autouse=True)
def built():
    from hstu_sequential_transducer_layer_b200.build import build
    build()


# ---------------------------------------------------------------- oracle
def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(0)
    ids = np.array([2, 0, 2, 5, -1, 4, 2, 9])     # 5: pad, -1 and 9: outside
    E, W = rng.standard_normal((5, 3)), rng.standard_normal((8, 3))
    g, a, n = TR.embed_bwd(ids, W, 5, 1.7, pad=5)
    assert n.tolist() == [1, 0, 3, 0, 1]
    h = 1e-3                                       # the lookup is linear: differences are exact
    for r in range(5):
        for c in range(3):
            up, dn = E.copy(), E.copy()
            up[r, c] += h
            dn[r, c] -= h
            d = ((TR.embed_fwd(ids, up, 1.7, 5) - TR.embed_fwd(ids, dn, 1.7, 5)) * W).sum() / (2 * h)
            assert abs(d - g[r, c]) < 1e-9


def test_adamw_oracle_is_torch_adamw():
    import torch
    rng = np.random.default_rng(1)
    p0 = rng.standard_normal(50)
    t = torch.tensor(p0, dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([t], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.3)
    p, m, v = p0, np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.standard_normal(50)
        t.grad = torch.tensor(g)
        opt.step()
        p, m, v = TR.adamw(p, g, m, v, step, 3e-3, 0.8, 0.95, 1e-6, 0.3)
    assert np.abs(p - t.detach().numpy()).max() < 1e-13


def test_norm_oracle():
    n, c = TR.grad_norm([np.array([3.0]), np.zeros(0), np.array([[0.0, 4.0]])], 1.0)
    assert n == 5.0 and c == 0.2
    assert TR.grad_norm([np.array([3.0])], 10.0) == (3.0, 1.0)
    assert TR.grad_norm([np.zeros(4)], 1.0) == (0.0, 1.0)
    assert math.isnan(TR.grad_norm([np.array([np.inf])], 1.0)[1])
    assert math.isnan(TR.grad_norm([np.array([1.0, np.nan])], 1.0)[1])


def test_e4m3_table_is_torch():
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(TR._E4M3, t)


def test_codes_follow_the_definition():
    """The float32 form of the encoding against real arithmetic: every value
    within one grid step, and almost all equal (a float32 product may fall on
    the other side of a rounding border)."""
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((40, 256)) * np.exp(rng.uniform(-12, 2, (40, 256)))).astype(np.float32)
    x[3, 5], x[4] = 0.0, 0.0
    x[5] *= np.float32(1e-30)
    x[6] *= np.float32(1e30)
    r = rng.integers(0, 65536, x.shape).astype(np.uint32)
    c, s = TR.encode_f32(x, r)
    q, k = TR.round_states(x, r)
    assert (s.astype(int) - 127 == k).all()
    got = TR.decode(c, s) / np.exp2(k)[:, None]
    assert (got != q).mean() < 1e-3
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -6))) - 3)
    assert (np.abs(got - q) <= step).all()
    assert np.abs(got).max() <= 256                      # never saturates


def test_rounding_is_unbiased():
    """The mean of the stored value over all 2^16 random numbers is the value,
    to 2 / 2^16 of a code step."""
    r = np.arange(65536, dtype=np.uint32)[None, :]
    for y in (200.3, 17.77, 0.3, 2.0 ** -6 * 0.77, 2.0 ** -9 * 0.3):
        x = np.full((1, 65536), y)
        x[0, 0] = 255.0                                  # fixes the scale at 2^0
        q, k = TR.round_states(x, r)
        assert k[0] == 0
        step = 2.0 ** (max(math.floor(math.log2(y)), -6) - 3)
        assert abs(q[0, 1:].mean() - y) <= step * 2 / 65536


def test_random_numbers_differ_by_seed_step_tensor_and_block():
    base = TR.random16(7, 3, 0, [0, 1])
    assert not np.array_equal(base[0][0], base[0][1])
    for other in (TR.random16(8, 3, 0, [0]), TR.random16(7, 4, 0, [0]), TR.random16(7, 3, 1, [0]),
                  TR.random16(7, 3, 0, [1 << 32])):
        assert (other[0][0] == base[0][0]).mean() < 0.05
    many = np.concatenate([x.ravel() for x in TR.random16(1, 1, 0, np.arange(256))])
    assert abs(many.mean() - 32767.5) < 5 * 65536 / math.sqrt(12 * many.size)


# ---------------------------------------------------------------- refusals
def test_embedding_refusals():
    L = B.lib()
    n0 = H.hstu_launch_count()
    fwd = lambda **k: L.hstu_embed_fwd(
        k.get("T", 10), k.get("ids", 0x1000), k.get("tab", 0x2000), k.get("dt", 0),
        k.get("R", 100), k.get("d", 64), k.get("ldt", 64), -1, k.get("s", 1.0),
        k.get("out", 0x3000), k.get("odt", 0), k.get("ldo", 64), k.get("ws", 0x10000),
        k.get("wsb", 256), None)
    for bad in (dict(T=-1), dict(T=1 << 31), dict(R=0), dict(R=1 << 31), dict(d=0), dict(ldt=63),
                dict(ldo=63), dict(dt=3), dict(odt=-1), dict(s=math.nan), dict(s=math.inf),
                dict(ldt=1 << 32), dict(ldo=1 << 32),
                dict(ids=None), dict(tab=None), dict(out=None), dict(tab=0x2008), dict(out=0x3002),
                dict(ids=0x1008)):
        assert fwd(**bad) == 1, bad
    assert fwd(ws=None) == 3 and fwd(ws=0x10010) == 3 and fwd(wsb=255) == 3
    need = L.hstu_embed_bwd_workspace_size(10, 100, 64)
    assert need > 0 and need % 256 == 0
    assert L.hstu_embed_bwd_workspace_size(-1, 100, 64) == 0
    assert L.hstu_embed_bwd_workspace_size(10, 0, 64) == 0
    assert L.hstu_embed_bwd_workspace_size(10, 100, 0) == 0
    assert L.hstu_embed_bwd_workspace_size(1 << 31, 100, 64) == 0
    assert L.hstu_embed_bwd_workspace_size(1000, 100, 64) > need
    bwd = lambda **k: L.hstu_embed_bwd(
        k.get("T", 10), k.get("ids", 0x1000), k.get("dY", 0x2000), k.get("dt", 0), k.get("ldy", 64),
        k.get("R", 100), k.get("d", 64), -1, k.get("s", 1.0), k.get("acc", 0), k.get("dE", 0x3000),
        k.get("odt", 1), k.get("ldo", 64), k.get("ws", 0x10000), k.get("wsb", need), None)
    for bad in (dict(T=-1), dict(R=0), dict(d=0), dict(ldy=63), dict(ldo=10), dict(dt=7),
                dict(odt=9), dict(acc=2), dict(s=math.nan), dict(ids=None), dict(dY=None),
                dict(dE=None), dict(dE=0x3008), dict(dY=0x2004), dict(T=0, dE=None)):
        assert bwd(**bad) == 1, bad
    assert bwd(wsb=need - 1) == 3 and bwd(ws=0x10080) == 3
    rows = lambda **k: L.hstu_embed_bwd_rows(
        k.get("T", 10), 0x1000, 0x2000, 0, 64, 100, 64, -1, 1.0, k.get("ri", 0x4000),
        k.get("out", 0x3000), 1, 64, k.get("n", 0x5000), k.get("ws", 0x10000), k.get("wsb", need),
        None)
    for bad in (dict(ri=None), dict(n=None), dict(out=None), dict(ri=0x4008), dict(n=0x5008)):
        assert rows(**bad) == 1, bad
    assert rows(wsb=0) == 3
    ids = lambda out: L.hstu_sl_embed_ids(2, 10, 8, 0x1000, 0x2000, 0x3000, 7, 0x4000, 100, 0x5000,
                                          8, 64, 0x6000, 0x7000, 0x8000, out, 0x10000, 128, None)
    assert ids(None) == 1 and ids(0x9000) == 3
    assert ids(0x9008) == 1
    assert H.hstu_launch_count() == n0


def _tensor(**k):
    t = B.AdamWTensor()
    for f, x in dict(dict(n=256, grad=0x1000, grad_dtype=1, param=0x2000, param_dtype=0, m=0x3000,
                          v=0x4000, state_bits=32), **k).items():
        setattr(t, f, x)
    return t


def test_optimizer_refusals():
    L = B.lib()
    n0 = H.hstu_launch_count()
    ws = 0x10000

    def step(t=None, n=1, w=ws, wb=256, **k):
        a = B.AdamWArgs(1e-3, 0.9, 0.999, 1e-8, 1, None, None, None, 0)
        for f, x in k.items():
            setattr(a, f, x)
        return L.hstu_adamw_step(ctypes.byref(a), ctypes.byref(t or _tensor()), n, w, wb, None)

    for bad in (dict(step=0), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(eps=0.0), dict(eps=1e-39),
                dict(eps=math.nan), dict(lr=math.inf), dict(beta2=math.nan)):
        assert step(**bad) == 1, bad
    rows = dict(row_ids=0x5000, n_rows=0x6000, row_len=64, max_rows=10)
    for bad in (dict(n=-1), dict(grad=None), dict(param=None), dict(m=None), dict(v=None),
                dict(grad=0x1004), dict(param=0x2002), dict(master=0x7004), dict(copy_f16=0x7002),
                dict(m=0x3008), dict(v=0x4004), dict(grad_dtype=5), dict(param_dtype=-1),
                dict(state_bits=16), dict(state_bits=8), dict(state_bits=8, m_scale=0x7001),
                dict(weight_decay=math.nan), dict(row_ids=0x5000), dict(n_rows=0x6000, row_len=64),
                dict(rows, row_len=0), dict(rows, row_len=48), dict(rows, max_rows=-1),
                dict(rows, row_ids=0x5008), dict(rows, n_rows=0x6004)):
        assert step(_tensor(**bad)) == 1, bad
    assert step(n=-1) == 1 and step(n=5000) == 2
    assert step(w=None) == 3 and step(w=ws + 8) == 3 and step(wb=128) == 3
    assert step(_tensor(**dict(rows, max_rows=0x7fffffff, row_len=1 << 20, n=1 << 30))) == 2
    wn = L.hstu_grad_norm_workspace_size()
    norm = lambda t=None, n=1, mx=1.0, out=0x8000, w=ws, wb=wn: L.hstu_grad_norm(
        ctypes.byref(t or _tensor()), n, mx, out, w, wb, None)
    for bad in (dict(mx=0.0), dict(mx=math.nan), dict(mx=-1.0), dict(out=None), dict(out=0x8004),
                dict(n=-1), dict(t=_tensor(grad=None)), dict(t=_tensor(grad_dtype=4)),
                dict(t=_tensor(grad=0x1008)), dict(t=_tensor(n_rows=0x6000, row_len=0))):
        assert norm(**bad) == 1, bad
    assert norm(wb=wn - 1) == 3 and norm(w=ws + 16) == 3 and norm(n=5000) == 2
    assert H.hstu_launch_count() == n0


def test_state_scales():
    assert H.state_scales((1,)) == 1 and H.state_scales((256,)) == 1 and H.state_scales((257,)) == 2
    assert H.state_scales((10, 50)) == 10 and H.state_scales((10, 512)) == 20


def test_binding_refuses_host_tensors():
    import torch
    ids = torch.zeros(4, dtype=torch.int64)
    tab, out = torch.zeros(8, 16), torch.zeros(4, 16)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(B.HstuError):
        H.hstu_embed_fwd(ids, tab, out, ws)
    with pytest.raises(B.HstuError):
        H.GradTensors([dict(grad=torch.zeros(4))])


def test_norm_after_refusals():
    L = B.lib()
    n0 = H.hstu_launch_count()
    wn = L.hstu_grad_norm_workspace_size()
    norm = lambda after=0x20000, n=1, mx=1.0, out=0x8000, w=0x10000, wb=wn: L.hstu_grad_norm_after(
        ctypes.byref(_tensor()), n, mx, after, out, w, wb, None)
    for bad in (dict(after=0x20010), dict(after=4), dict(n=-1), dict(mx=0.0), dict(out=None),
                dict(out=0x8004)):
        assert norm(**bad) == 1, bad
    assert norm(wb=wn - 1) == 3 and norm(w=None) == 3 and norm(n=5000) == 2
    assert H.hstu_launch_count() == n0
