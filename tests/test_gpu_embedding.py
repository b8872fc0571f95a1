"""GPU parity of the embedding lookup with scaling and of its gradient against
float64 (oracle.training).

Bounds: a lookup is one fp32 product rounded to the output type, so it is off
by at most 2^-24 and half a step of the type, relative to the value.  A
gradient element is n fp32 additions, the product with the scale and the
output's rounding: at most (n + 2) 2^-24 of the sum of the magnitudes, and half
a step of the type (accumulating adds one more fp32 addition).  Small integers
with a power-of-two scale are exact."""
import math

import numpy as np
import pytest

from oracle import training as TR

pytestmark = pytest.mark.gpu

BAD_IDS = 8
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}       # half a step of fp16's smallest values


@pytest.fixture(scope="module", autouse=True)
def built():
    from hstu_sequential_transducer_layer_b200.build import build
    build()


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def _ws(n):
    import torch
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")     # never clean


def _strided(rows, cols, ld, dt, fill=float("nan")):
    """A [rows, cols] view with row stride ld, and its whole buffer."""
    import torch
    buf = torch.full((max(rows, 1), ld), fill, dtype=dt, device="cuda")
    return buf[:rows, :cols], buf


def _tokens(T, R, seed, kind):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        return rng.integers(0, R, T)
    if kind == "one":
        return np.full(T, R - 1)
    if kind == "few":                      # half of the tokens on the last 3 rows
        a = rng.integers(0, R, T)
        a[1::2] = R - 1 - rng.integers(0, min(3, R), len(a[1::2]))
        return a
    return np.arange(T) % R                # every row once (or evenly)


# ---------------------------------------------------------------- lookup
@pytest.mark.parametrize("T,R,d,pad_ld", [
    (0, 5, 8, 0), (1, 1, 1, 0), (1, 8, 256, 0), (37, 100, 50, 0), (5, 9, 1024, 8), (300, 64, 257, 3),
    (1000, 33, 8, 0), (999, 1000, 100, 4), (64, 7, 2056, 0), (70001, 500, 8, 8)])
@pytest.mark.parametrize("src,out", [("bf16", "bf16"), ("f32", "bf16"), ("f16", "f32"), ("f32", "f16")])
def test_lookup(T, R, d, pad_ld, src, out):
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    g = torch.Generator(device="cuda").manual_seed(T + d)
    tab, _ = _strided(R, d, d + pad_ld, _dt(src))
    tab.copy_(torch.randn(R, d, device="cuda", generator=g))
    y, buf = _strided(T, d, d + 2 * pad_ld, _dt(out), fill=7.0)
    ids = _tokens(T, R, T, "uniform")
    if T > 4:
        ids[3] = 2 % R                     # the padding's row
    scale = math.sqrt(d) if T % 2 else 0.5
    pad = 2 % R if T > 4 else -1
    ws = _ws(H.hstu_embed_workspace_size())
    H.hstu_embed_fwd(torch.from_numpy(ids).cuda(), tab, y, ws, scale=scale, pad_id=pad)
    assert H.hstu_read_status(ws) == 0
    ref = TR.embed_fwd(ids, tab.double().cpu().numpy(), np.float64(np.float32(scale)), pad)
    got = y.double().cpu().numpy()
    assert (np.abs(got - ref) <= (HALF[out] + 2.0 ** -23) * np.abs(ref) + TINY[out]).all()
    assert not got[ids == pad].any()
    if pad_ld and T:                       # the gaps between rows are left alone
        assert (buf[:, d:] == 7.0).all()


@pytest.mark.parametrize("T", [9, 70000])
def test_lookup_bad_ids(T):
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    tab = torch.randn(10, 16, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(0, 10, (T,), device="cuda")
    ids[2], ids[5], ids[7], ids[8] = 10, -3, 1 << 40, 99
    y = torch.full((T, 16), 3.0, device="cuda", dtype=torch.bfloat16)
    ws = _ws(256)
    H.hstu_embed_fwd(ids, tab, y, ws, pad_id=99)
    assert H.hstu_read_status(ws) == BAD_IDS
    bad = (ids < 0) | (ids >= 10)
    assert not y[bad].any() and torch.equal(y[~bad], tab[ids[~bad]])
    ids.clamp_(0, 9)                       # the next call on the same workspace is clean again
    H.hstu_embed_fwd(ids, tab, y, ws)
    assert H.hstu_read_status(ws) == 0 and torch.equal(y, tab[ids])


# ---------------------------------------------------------------- gradient
def _gradient(ids, dY, R, scale=1.0, pad=-1, out="f32", compact=False, start=None, ld=None,
              accumulate=False):
    """(status, dense gradient float64, row ids, whole output buffer)."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    T, d = dY.shape
    t = torch.from_numpy(np.asarray(ids, np.int64)).cuda()
    ws = _ws(H.hstu_embed_bwd_workspace_size(T, R, d))
    ld = ld or d
    if compact:
        cap = min(T, R)
        rows, buf = _strided(cap, d, ld, _dt(out), fill=-5.0)
        row_ids = torch.full((cap,), -9, dtype=torch.int64, device="cuda")
        n = torch.full((1,), -1, dtype=torch.int64, device="cuda")
        H.hstu_embed_bwd_rows(t, dY, R, row_ids, rows, n, ws, scale=scale, pad_id=pad)
        st, U = H.hstu_read_status(ws), int(n)
        r = row_ids.cpu().numpy()
        assert (r[U:] == -9).all() and (buf[U:] == -5.0).all()     # behind the last: as it was
        assert (np.diff(r[:U]) > 0).all()
        dense = np.zeros((R, d))
        dense[r[:U]] = rows[:U].double().cpu().numpy()
        return st, dense, r[:U], buf
    g, buf = _strided(R, d, ld, _dt(out), fill=-5.0)
    if start is not None:
        g.copy_(start)
    H.hstu_embed_bwd(t, dY, g, ws, scale=scale, pad_id=pad, accumulate=accumulate)
    return H.hstu_read_status(ws), g.double().cpu().numpy(), None, buf


@pytest.mark.parametrize("compact", [False, True])
@pytest.mark.parametrize("T,R,d,kind", [
    (0, 5, 8, "uniform"), (1, 1, 1, "one"), (1, 1000000, 64, "one"), (2, 3, 8, "one"),
    (16, 1, 8, "one"), (17, 4, 50, "few"), (127, 9, 64, "few"), (128, 128, 264, "each"),
    (129, 2, 8, "few"), (700, 3, 257, "uniform"), (1500, 100000, 100, "few"),
    (5000, 40, 72, "few"), (8192, 8, 64, "uniform"), (8193, 2000000, 8, "uniform"),
    (9001, 1, 16, "one"), (20011, 1500, 136, "few"), (70001, 1 << 22, 8, "few")])
def test_gradient(T, R, d, kind, compact):
    import torch
    ids = _tokens(T, R, T + R, kind)
    dt = ("bf16", "f16", "f32")[T % 3]
    dY = torch.randn(T, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T)) \
        .to(_dt(dt))
    scale, pad = 1.25, (int(ids[T // 2]) if T > 100 and kind != "one" else -1)
    if R * d > 1 << 25 and not compact:
        R = int(ids.max()) + 1
        if R * d > 1 << 26:
            pytest.skip("the dense form of this table is tested by its rows")
    st, got, rows, _ = _gradient(ids, dY, R, scale, pad, compact=compact)
    assert st == 0
    ref, mag, n = TR.embed_bwd(ids, dY.double().cpu().numpy(), R, scale, pad)
    tol = (n[:, None] + 2) * 2.0 ** -24 * mag + 2.0 ** -24 * np.abs(ref)
    assert (np.abs(got - ref) <= tol).all()
    if compact:
        np.testing.assert_array_equal(rows, np.flatnonzero(n))


@pytest.mark.parametrize("compact", [False, True])
@pytest.mark.parametrize("T,R,d,kind", [
    (131072, 1000, 8, "few"), (131073, 3000000, 8, "few"), (140000, 2, 50, "few"),
    (262145, 70000, 16, "each"), (300001, 1, 8, "one"), (400000, 1 << 25, 8, "uniform")])
def test_gradient_of_many_tokens(T, R, d, kind, compact):
    """Around and beyond the 131,072 tokens that one cluster of blocks sorts."""
    import torch
    if not compact and R * d > 1 << 26:
        R = 100000
    ids = _tokens(T, R, T, kind)
    dY = torch.randn(T, d, device="cuda", generator=torch.Generator("cuda").manual_seed(T)) \
        .to(torch.bfloat16)
    pad = int(ids[7]) if kind == "few" else -1
    st, got, rows, _ = _gradient(ids, dY, R, 2.0, pad, compact=compact)
    assert st == 0
    keep = ids != pad
    y = 2.0 * dY.double().cpu().numpy()[keep]
    touched, at = np.unique(ids[keep], return_inverse=True)
    ref, mag, n = np.zeros((len(touched), d)), np.zeros((len(touched), d)), np.bincount(at)
    np.add.at(ref, at, y)
    np.add.at(mag, at, np.abs(y))
    tol = (n[:, None] + 2) * 2.0 ** -24 * mag + 2.0 ** -24 * np.abs(ref)
    assert (np.abs(got[touched] - ref) <= tol).all()
    assert not np.delete(got, touched, axis=0).any()
    if compact:
        np.testing.assert_array_equal(rows, touched)
    if T % 2:
        ids[T // 3] = R + 5
        assert _gradient(ids, dY, R, 2.0, pad, compact=compact)[0] == BAD_IDS


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,ld", [(40, 40), (40, 48), (41, 43), (512, 512)])
def test_gradient_output_types_and_accumulation(out, d, ld):
    import torch
    T, R = 900, 77
    ids = _tokens(T, R, 5, "few")
    dY = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    ref, mag, n = TR.embed_bwd(ids, dY.double().cpu().numpy(), R, 0.75)
    tol = (n[:, None] + 2) * 2.0 ** -24 * mag
    st, got, _, buf = _gradient(ids, dY, R, 0.75, out=out, ld=ld)
    assert st == 0 and (np.abs(got - ref) <= tol * 1.01 + HALF[out] * np.abs(ref) + TINY[out]).all()
    assert (buf[:, d:] == -5.0).all()
    start = torch.randn(R, d, device="cuda").to(_dt(out))
    s = start.double().cpu().numpy()
    st, got, _, _ = _gradient(ids, dY, R, 0.75, out=out, ld=ld, start=start, accumulate=True)
    total = s + ref
    assert st == 0
    assert (np.abs(got - total) <= tol * 1.01 + 2.0 ** -23 * (np.abs(s) + np.abs(ref)) +
            HALF[out] * np.abs(total) + TINY[out]).all()
    assert (got[n == 0] == s[n == 0]).all()


def test_gradient_of_integers_is_exact_and_repeats_bitwise():
    import torch
    T, R, d = 30011, 700, 264
    ids = _tokens(T, R, 8, "few")
    rng = np.random.default_rng(8)
    dY = rng.integers(-3, 4, (T, d)).astype(np.float32)
    ref = np.zeros((R, d))
    np.add.at(ref, ids, dY)
    st, got, _, _ = _gradient(ids, torch.from_numpy(dY).cuda(), R, 0.5)
    np.testing.assert_array_equal(got, 0.5 * ref)
    x = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    first = _gradient(ids, x, R, 0.3)[1]
    for _ in range(3):
        np.testing.assert_array_equal(_gradient(ids, x, R, 0.3)[1], first)
    np.testing.assert_array_equal(_gradient(ids, x, R, 0.3, compact=True)[1], first)


def test_gradient_input_strides():
    import torch
    T, R, d = 300, 20, 24
    ids = _tokens(T, R, 1, "few")
    for ld in (24, 32, 27):
        dY, _ = _strided(T, d, ld, torch.float16)
        dY.copy_(torch.randn(T, d, device="cuda"))
        ref, mag, n = TR.embed_bwd(ids, dY.double().cpu().numpy(), R, 1.0)
        st, got, _, _ = _gradient(ids, dY, R)
        assert st == 0 and (np.abs(got - ref) <= (n[:, None] + 2) * 2.0 ** -24 * mag).all()


def test_gradient_of_a_broadcast_input_is_refused():
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    dY = torch.ones(1, 8, device="cuda").expand(4, 8)
    with pytest.raises(H.HstuError):
        H.hstu_embed_bwd(ids, dY, torch.zeros(3, 8, device="cuda"),
                         _ws(H.hstu_embed_bwd_workspace_size(4, 3, 8)))


@pytest.mark.parametrize("T", [40, 9000])
def test_gradient_bad_and_dropped_ids(T):
    import torch
    ids = np.arange(T) % 7
    ids[[3, T - 1]] = 7
    ids[8] = -1
    ids[10] = 1 << 35
    dY = torch.randn(T, 16, device="cuda")
    for compact in (False, True):
        st, got, _, _ = _gradient(ids, dY, 7, pad=-1, compact=compact)     # -1: padding, 7: bad
        assert st == BAD_IDS
        ref, mag, n = TR.embed_bwd(ids, dY.double().cpu().numpy(), 7, 1.0, -1)
        assert (np.abs(got - ref) <= (n[:, None] + 2) * 2.0 ** -24 * mag).all()
        # every token dropped
        st, got, rows, _ = _gradient(np.full(T, 5), dY, 7, pad=5, compact=compact)
        assert st == 0 and not got.any() and (rows is None or rows.size == 0)


def test_nan_stays_in_its_row():
    import torch
    dY = torch.ones(50, 8, device="cuda")
    dY[20, 3] = float("nan")
    dY[21, 4] = float("inf")
    ids = np.arange(50) % 5
    _, got, _, _ = _gradient(ids, dY, 5)
    assert np.isnan(got[0, 3]) and np.isinf(got[1, 4])
    got[0, 3] = got[1, 4] = 10.0
    assert (got == 10.0).all()


def test_offsets_past_32_bits():
    """A table, and a gradient, of more than 2^32 bytes and 2^31 elements: rows
    at its end (the gradient's other rows are zero)."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    R, d = 2_200_000, 1024
    tab = torch.zeros(R, d, dtype=torch.bfloat16, device="cuda")
    last = torch.tensor([R - 1, 0, R - 2, R - 1], device="cuda")
    tab[R - 2], tab[R - 1], tab[0] = 2.0, 3.0, 4.0
    y = torch.empty(4, d, dtype=torch.bfloat16, device="cuda")
    ws = _ws(256)
    H.hstu_embed_fwd(last, tab, y, ws, scale=2.0)
    assert y[:, 0].tolist() == [6.0, 8.0, 4.0, 6.0] and H.hstu_read_status(ws) == 0
    tab.fill_(1.0)
    ws = _ws(H.hstu_embed_bwd_workspace_size(4, R, d))
    H.hstu_embed_bwd(last, y, tab, ws)
    assert (tab[R - 1] == 12.0).all() and (tab[R - 2] == 4.0).all() and (tab[0] == 8.0).all()
    assert not tab[1:R - 2].any()


def test_another_stream_and_captured_replay():
    """The calls run on the stream they are given, and a captured lookup and
    gradient give the same again on new ids."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    T, R, d = 3000, 50, 64
    tab = torch.randn(R, d, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(0, R, (T,), device="cuda")
    y = torch.empty(T, d, device="cuda", dtype=torch.bfloat16)
    g = torch.empty(R, d, device="cuda")
    row_ids = torch.zeros(R, dtype=torch.int64, device="cuda")
    rows, n = torch.zeros(R, d, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = _ws(H.hstu_embed_bwd_workspace_size(T, R, d))
    fws = _ws(256)

    def both():
        H.hstu_embed_fwd(ids, tab, y, fws, scale=2.0)
        H.hstu_embed_bwd(ids, y, g, ws, scale=2.0)
        H.hstu_embed_bwd_rows(ids, y, R, row_ids, rows, n, ws, scale=2.0)

    def check():
        torch.cuda.synchronize()
        want = torch.zeros(R, d, dtype=torch.float64, device="cuda").index_add_(
            0, ids, 4.0 * tab[ids].double())
        count = torch.bincount(ids, minlength=R)[:, None]
        tol = (count + 2) * 2.0 ** -24 * 4.0 * tab.double().abs() * count
        assert ((g - want).abs() <= tol).all()
        U = int(n)
        assert row_ids[:U].tolist() == ids.unique().tolist()
        assert torch.equal(rows[:U], g[row_ids[:U]])
        assert H.hstu_read_status(ws) == 0 and H.hstu_read_status(fws) == 0
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        both()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in (3, 40, 50):
        ids.copy_(torch.randint(0, k, (T,), device="cuda"))
        graph.replay()
        check()
    del graph


def test_two_gradients_at_once():
    """Two streams, each with its own workspace."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    T, R, d = 20000, 300, 256
    s = [torch.cuda.Stream() for _ in range(2)]
    ids = [torch.randint(0, R, (T,), device="cuda") for _ in s]
    dY = [torch.randint(-2, 3, (T, d), device="cuda").float() for _ in s]
    g = [torch.empty(R, d, device="cuda") for _ in s]
    ws = [_ws(H.hstu_embed_bwd_workspace_size(T, R, d)) for _ in s]
    torch.cuda.synchronize()
    for _ in range(5):
        for k in range(2):
            H.hstu_embed_bwd(ids[k], dY[k], g[k], ws[k], stream=s[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(g[k], torch.zeros_like(g[k]).index_add_(0, ids[k], dY[k]))


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,ld", [(40, 40), (40, 48), (41, 43), (512, 520), (1, 9)])
@pytest.mark.parametrize("T", [1, 900, 9001])
def test_touched_rows_output_types_and_strides(T, d, ld, out):
    """The touched rows in each type and with gaps behind the rows: the sums as in the dense form, the gaps
    and the rows behind the last one left alone (checked by _gradient, and the gaps here)."""
    import torch
    R = 77
    ids = _tokens(T, R, 5, "few")
    dt = _dt(("bf16", "f16", "f32")[(T + d) % 3])
    dY = torch.randn(T, d, device="cuda", generator=torch.Generator("cuda").manual_seed(d)).to(dt)
    ref, mag, n = TR.embed_bwd(ids, dY.double().cpu().numpy(), R, 0.75)
    st, got, rows, buf = _gradient(ids, dY, R, 0.75, out=out, ld=ld, compact=True)
    assert st == 0
    np.testing.assert_array_equal(rows, np.flatnonzero(n))
    tol = (n[:, None] + 2) * 2.0 ** -24 * mag
    assert (np.abs(got - ref) <= tol * 1.01 + HALF[out] * np.abs(ref) + TINY[out]).all()
    assert (buf[:, d:] == -5.0).all()
