"""The training-side operators together, as HSTUTrainer runs them: raw streams
-> hstu_sl_embed_ids -> the stack's gradients -> the gradient of the touched
table rows -> the clipping norm -> the AdamW step, several times over, each
result against float64 on what the step before it left."""
import numpy as np
import pytest

import hstu_workloads as hw
from gpu_util import TOL, relerr, rmserr, runner_for
from oracle import hstu_backward as BW
from oracle import stochastic_length as SL
from oracle import training as TR

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from hstu_sequential_transducer_layer_b200.build import build
    build()


def _streams(seed, lengths=(200, 1, 90, 0, 301), d=128, n_content=60, n_actions=8):
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    rs = hw.raw_stream("train", list(lengths), d, n_content, n_actions, seed=seed)
    # The generator draws one timestamp for an empty user too, so the user behind it would start
    # with that one, 1,327,867,846 s before its own: more than the 2^30 s that the stack takes.
    # One token a minute instead.
    rs.raw_timestamps = np.concatenate([60 * np.arange(n) for n in lengths]).astype(np.int64)
    dev = [torch.from_numpy(x).cuda() for x in (rs.raw_offsets, rs.raw_ids, rs.raw_timestamps)]
    k = [SL.keep_count(int(n)) for n in np.diff(rs.raw_offsets)]
    return rs, dev, sum(k), max(k)


def _embed(rs, dev, T, table, n_content):
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    off = torch.empty(rs.B + 1, dtype=torch.int64, device="cuda")
    X = torch.empty(T, table.shape[1], dtype=torch.bfloat16, device="cuda")
    ts = torch.empty(T, dtype=torch.int64, device="cuda")
    ids = torch.full((T,), -7, dtype=torch.int64, device="cuda")
    ws = torch.empty(H.hstu_sl_embed_workspace_size(), dtype=torch.uint8, device="cuda")
    H.hstu_sl_embed_ids(rs.B, rs.R, rs.max_raw_len, *dev, rs.sl_seed, table[:n_content],
                        table[n_content:], off, X, ts, ids, ws)
    return off, X, ts, ids, H.hstu_read_status(ws)


def test_ids_of_the_kept_tokens():
    """The ids name the rows that were copied: looking them up again gives X,
    and everything else is what hstu_sl_embed writes; a bad id gives -1."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    rs, dev, T, _ = _streams(3)
    table = torch.randn(68, 128, device="cuda").to(torch.bfloat16)
    off, X, ts, ids, st = _embed(rs, dev, T, table, 60)
    assert st == 0 and int(ids.min()) >= 0 and int(ids.max()) < 68
    Y = torch.empty_like(X)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    H.hstu_embed_fwd(ids, table, Y, ws)
    assert torch.equal(X, Y) and H.hstu_read_status(ws) == 0
    o2, X2, t2 = torch.empty_like(off), torch.empty_like(X), torch.empty_like(ts)
    H.hstu_sl_embed(rs.B, rs.R, rs.max_raw_len, *dev, rs.sl_seed, table[:60], table[60:], o2, X2, t2, ws)
    assert torch.equal(off, o2) and torch.equal(X, X2) and torch.equal(ts, t2)
    for u in range(rs.B):                       # the oracle's positions
        pos = SL.kept_positions(rs.sl_seed, u, int(np.diff(rs.raw_offsets)[u]))
        want = [int(rs.raw_ids[rs.raw_offsets[u] + p]) + 60 * (p & 1) for p in pos]
        assert ids[int(off[u]):int(off[u + 1])].tolist() == want
    dev[1][200] = 60                            # the only token of user 1, a content position
    _, X, _, ids, st = _embed(rs, dev, T, table, 60)
    at = int(off[1])
    assert st == 8 and int(ids[at]) == -1 and not X[at].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps(bits):
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    dims = hw.LayerDims(128, 2, 64, 64, 64, 128, 3, 2, 1e-6, hw.BF16)
    w = hw.custom("train", [1], dims, n_layers=2, seed=21)
    r = runner_for(w)
    table = torch.randn(68, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) \
        .to(torch.bfloat16)
    tr = H.HSTUTrainer(r, table, max_tokens=400, state_bits=bits, lr=1e-2, weight_decay=0.1,
                       max_norm=0.5, seed=3)
    rng = np.random.default_rng(0)
    for k in range(1, 4):
        rs, dev, T, max_len = _streams(30 + k)
        off, X, ts, ids, st = _embed(rs, dev, T, table, 60)
        assert st == 0
        dY = r.to_device(hw.round_to_bf16(rng.standard_normal((T, 128)).astype(np.float32)))
        old = [{q: x.clone() for q, x in t.items() if hasattr(x, "clone")} for t in tr.tensors]
        weights = [{q: w_[q].double().cpu().numpy() for q in w_ if not q.endswith("_f16")}
                   for w_ in r.weights]
        dX = tr.step(off, X, ts, dY, max_len, ids=ids, embed_scale=2.0)
        torch.cuda.synchronize()
        assert tr.status() == 0
        # the stack's gradients from the weights the last step left (their fp16 copies included)
        ref, gref = BW.stack_bwd(X.double().cpu().numpy(), off.cpu().numpy(), ts.cpu().numpy(), weights,
                                 dims, dY.double().cpu().numpy())
        assert rmserr(dX.double().cpu().numpy(), ref) <= TOL[hw.BF16]
        for l in range(2):
            for q in gref[l]:
                if q != "dX":
                    assert rmserr(tr.grads[l][q].double().cpu().numpy(), gref[l][q]) <= TOL[hw.BF16], q
        # the touched rows from the GPU's own dX
        g, mag, n = TR.embed_bwd(ids.cpu().numpy(), dX.double().cpu().numpy(), 68, 2.0)
        U = int(tr.n_rows)
        assert tr.row_ids[:U].tolist() == np.flatnonzero(n).tolist()
        rows = tr.row_grad[:U].double().cpu().numpy()
        assert (np.abs(rows - g[n > 0]) <= ((n[:, None] + 2) * E * mag)[n > 0]).all()
        # norm and clip factor from the GPU's own gradients
        norm, c = TR.grad_norm([x.double().cpu().numpy() for l in tr.grads for x in l.values()] + [rows], 0.5)
        assert abs(float(tr.norm[0]) - norm) <= 1.01 * E * norm
        gs = float(tr.norm[1])
        assert abs(gs - c) <= 1.01 * E * c and c < 1
        # the update; the table's untouched rows stay
        for t, o in zip(tr.tensors, old):
            wide = (o["master"] if "master" in o else o["param"]).double().cpu().numpy()
            grad = t["grad"].double().cpu().numpy()
            if bits == 32:
                m, v = (o[q].double().cpu().numpy() for q in ("m", "v"))
            else:
                d = t["param"].shape[-1] if "row_ids" in t else t["param"].numel()
                nb = -(-d // 256)
                pad = lambda x: torch.nn.functional.pad(x.view(torch.uint8).reshape(-1, d), (0, nb * 256 - d)) \
                    .reshape(-1, 256).cpu().numpy()
                m, v = (TR.decode(pad(o[q]), o[q + "_scale"].cpu().numpy()).reshape(-1, nb * 256)[:, :d]
                        .reshape(wide.shape) for q in ("m", "v"))
                v = v ** 2
            if "row_ids" in t:
                full = np.zeros_like(wide)
                full[n > 0] = rows
                grad = full
            p, _, _ = TR.adamw(wide, grad.reshape(wide.shape), m, v, k, 1e-2, 0.9, 0.999, 1e-8,
                               t["weight_decay"], gs)
            if "row_ids" in t:
                p[n == 0] = wide[n == 0]
                assert torch.equal(t["param"][n == 0], o["param"][n == 0])
            new = (t["master"] if "master" in t else t["param"]).double().cpu().numpy()
            # a step is at most lr (1 - beta1) / sqrt(1 - beta2) = 0.032 at any time, its terms good to
            # 2^-18 of that (m may cancel to 1/16 of its terms), and p to 2^-22
            assert (np.abs(new - p) <= 0.032 * 2.0 ** -18 + 2.0 ** -22 * np.abs(p)).all()
            if "master" in t:
                assert torch.equal(t["param"], t["master"].to(t["param"].dtype))
            if t.get("copy_f16") is not None:
                assert torch.equal(t["copy_f16"], t["param"].half())
    with pytest.raises(H.HstuError):
        tr.step(off, X, ts, dY, max_len)


def test_trainer_without_a_table():
    """Two hundred steps of one layer with 8-bit states run through and keep
    every weight finite."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    dims = hw.LayerDims(128, 2, 64, 64, 64, 128, 3, 2, 1e-6, hw.BF16)
    w = hw.custom("fit", [60, 7, 33], dims, seed=4)
    r = runner_for(w)
    off, ts, X = r.to_device(w.offsets, "i64"), r.to_device(w.timestamps, "i64"), r.to_device(w.X)
    target = torch.roll(X, 1, 0)
    tr = H.HSTUTrainer(r, lr=3e-3, state_bits=8)
    for _ in range(200):
        Y = r.stack(off, X, ts, w.max_len)
        tr.step(off, X, ts, (Y - target).contiguous(), w.max_len)
    torch.cuda.synchronize()
    assert tr.status() == 0
    for t in tr.tensors:
        assert torch.isfinite(t["param"]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_failed_backward_pass_changes_nothing(bits):
    """A batch with a user whose timestamps span more than the stack takes, and one whose offsets do not
    end at its rows, as the first step and behind a good one: weights, masters, copies, states and table
    stay as they are, status() tells why, and the next good step runs."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    dims = hw.LayerDims(128, 2, 64, 64, 64, 128, 3, 2, 1e-6, hw.BF16)
    w = hw.custom("failed", [60, 7, 33], dims, n_layers=2, seed=5)
    r = runner_for(w)
    table = torch.randn(40, 128, device="cuda").to(torch.bfloat16)
    tr = H.HSTUTrainer(r, table, max_tokens=100, state_bits=bits, lr=1e-2, table_decay=0.1)
    off, ts, X = r.to_device(w.offsets, "i64"), r.to_device(w.timestamps, "i64"), r.to_device(w.X)
    dY = torch.randn(100, 128, device="cuda").to(torch.bfloat16)
    ids = torch.arange(100, device="cuda") % 37
    late, short = ts.clone(), off.clone()
    late[5] += 1 << 31
    short[-1] -= 1
    keep = lambda: [{q: x.clone() for q, x in t.items() if hasattr(x, "clone")}  # noqa: E731
                    for t in tr.tensors]

    def same(old):
        return [all(torch.equal(t[q].view(torch.uint8), o[q].view(torch.uint8)) for q in o
                    if q not in ("grad", "row_ids", "n_rows")) for t, o in zip(tr.tensors, old)]
    for k in range(2):
        for o, t, want in ((off, late, 7), (short, ts, 5)):
            old = keep()
            tr.step(o, X, t, dY, w.max_len, ids=ids)
            assert tr.status() == want
            assert all(same(old)) and torch.isnan(tr.norm).all()
        old = keep()
        tr.step(off, X, ts, dY, w.max_len, ids=ids)
        assert tr.status() == 0 and torch.isfinite(tr.norm).all()
        assert not any(same(old))


@pytest.mark.parametrize("handle", [False, True])
def test_steps_on_a_stream_of_their_own(handle):
    """Two steps queued behind a pause of another stream, the second on a batch that makes the workspace
    grow, dX dropped each time: what the current stream allocates meanwhile, of those very sizes, is not
    written by them, and the weights are those of the same steps on the current stream."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    dims = hw.LayerDims(128, 2, 64, 64, 64, 128, 3, 2, 1e-6, hw.BF16)
    batches = [hw.custom("streams", n, dims, n_layers=2, seed=9) for n in ([60, 7, 33], [260, 301, 40])]
    runners = [runner_for(batches[0]) for _ in range(2)]
    trainers = [H.HSTUTrainer(r, torch.ones(50, 128, dtype=torch.bfloat16, device="cuda"), max_tokens=601)
                for r in runners]
    inputs = [(runners[0].to_device(w.offsets, "i64"), runners[0].to_device(w.X),
               runners[0].to_device(w.timestamps, "i64"), runners[0].to_device(w.X[::-1]), w.max_len,
               torch.arange(w.T, device="cuda") % 50) for w in batches]
    for off, X, ts, dY, longest, ids in inputs:
        trainers[0].step(off, X, ts, dY, longest, ids=ids)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for r, tr in ((runners[1], trainers[1]),):
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)               # cycles: a tenth of a second
        sizes = []
        for off, X, ts, dY, longest, ids in inputs:
            tr.step(off, X, ts, dY, longest, ids=ids, stream=side.cuda_stream if handle else side)
            sizes += [X.numel() * 2, r._bws.numel()]
        paused = not side.query()
        others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    assert paused
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in others)
    assert trainers[1].status(side) == 0
    for a, b in zip(trainers[0].tensors, trainers[1].tensors):
        for q in a:
            if hasattr(a[q], "clone"):
                assert torch.equal(a[q], b[q]), q


def test_outputs_belong_to_the_stream_of_the_call():
    """The same for the runner's other calls: what they return, once dropped, is not handed to the current
    stream while the call may still write it."""
    import torch
    dims = hw.LayerDims(128, 2, 64, 64, 64, 128, 3, 2, 1e-6, hw.BF16)
    w = hw.custom("streams", [60, 7, 33], dims, n_layers=2, seed=9)
    r = runner_for(w)
    off, X, ts = r.to_device(w.offsets, "i64"), r.to_device(w.X), r.to_device(w.timestamps, "i64")
    want = r.stack(off, X, ts, w.max_len)
    torch.cuda.synchronize()
    r.workspace(0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    r.stack(off, X, ts, w.max_len, stream=side)                     # dropped
    r.workspace(r._ws.numel() + 4096)                               # replaced while it is in use
    got = r.stack(off, X, ts, w.max_len, stream=side)
    paused = not side.query()
    others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda")
              for n in (X.numel() * 2, r._ws.numel() - 4096) for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    assert paused
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in others)
    assert torch.equal(got, want)


@pytest.mark.parametrize("with_table", [False, True])
def test_status_before_the_first_step(with_table):
    """No call has failed yet, whatever the memory of the workspaces held before."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    dims = hw.LayerDims(128, 2, 64, 64, 64, 128, 3, 2, 1e-6, hw.BF16)
    r = runner_for(hw.custom("fresh", [5], dims, seed=4))
    for n in (256, 1 << 16, 1 << 20, 1 << 22):              # given back to the allocator at once
        torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    table = torch.zeros(50, 128, dtype=torch.bfloat16, device="cuda") if with_table else None
    assert H.HSTUTrainer(r, table, max_tokens=100).status() == 0


def test_step_of_an_empty_batch():
    """No tokens: no gradient, so a step without weight decay changes no weight."""
    import torch
    import hstu_sequential_transducer_layer_b200 as H
    dims = hw.LayerDims(128, 2, 64, 64, 64, 128, 3, 2, 1e-6, hw.BF16)
    r = runner_for(hw.custom("empty", [5], dims, seed=4))
    table = torch.randn(50, 128, device="cuda").to(torch.bfloat16)
    tr = H.HSTUTrainer(r, table, max_tokens=10, weight_decay=0.0)
    old = [t["param"].clone() for t in tr.tensors]
    z = lambda *s: torch.zeros(*s, dtype=torch.int64, device="cuda")  # noqa: E731
    X = torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda")
    for off in (z(1), z(4)):
        dX = tr.step(off, X, z(0), X, 1, ids=z(0))
        assert dX.shape == X.shape and tr.status() == 0 and int(tr.n_rows) == 0
        assert tr.norm.tolist() == [0.0, 1.0]
    assert all(torch.equal(t["param"], o) for t, o in zip(tr.tensors, old))
