"""Cases of the training-side operators: embedding lookup with scaling, its gradient by sorted tokens, the global
gradient norm and the AdamW step over many tensors (states in 32 or in 8 bits, dense tensors or touched table rows).

Where `own` is false, run() computes them with elementary torch operations; where it is true, with the library's entry
points.  Sizes come from the workloads of hstu_workloads.py (the 8-layer d = 1024 stack, the single d = 256 layer, the
long-history batch) or are generic."""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 256          # elements that share a scale in the 8-bit states
GAMMA = 0x9E3779B97F4A7C15
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one user, a new event arriving while serving: latency only
        dict(name="lookup_single", op="lookup", tokens=1, rows=1000, actions=8, d=256, table="bf16", out="bf16",
             scale=16.0, pad=False),
        # the kept tokens of the full 8-layer batch (128 users after Stochastic Length) from its 1M-row table
        dict(name="lookup_batch", op="lookup", tokens=38070, rows=1000000, actions=8, d=1024, table="bf16",
             out="bf16", scale=32.0, pad=False),
        # a small public-dataset-sized catalog: odd width, fp32 table, padded ids
        dict(name="lookup_odd", op="lookup", tokens=20011, rows=3953, actions=0, d=50, table="f32", out="bf16",
             scale=math.sqrt(50.0), pad=True),
        # gradient of lookup_batch's table as touched rows: half of the tokens fall on 8 action rows
        dict(name="gradient_rows_batch", op="gradient", tokens=38070, rows=1000000, actions=8, d=1024, dy="bf16",
             out="f32", scale=32.0, pad=False, compact=True, accumulate=False),
        # the long-history batch into a dense gradient of a mid-size catalog
        dict(name="gradient_dense_catalog", op="gradient", tokens=82351, rows=65536, actions=0, d=512, dy="bf16",
             out="f32", scale=1.0, pad=False, compact=False, accumulate=False),
        # one user's actions added into an 8-row table's gradient: few rows, many tokens each
        dict(name="gradient_actions", op="gradient", tokens=3271, rows=8, actions=0, d=256, dy="f16", out="f32",
             scale=16.0, pad=True, compact=False, accumulate=True),
        # gradients of the single d = 256 layer
        dict(name="norm_layer", op="norm", layers=1, d_model=256, heads=4, d_head=64, grad="f32", rows=0),
        # gradients of the 8-layer stack with the touched table rows
        dict(name="norm_stack", op="norm", layers=8, d_model=1024, heads=8, d_head=128, grad="f32", rows=11003),
        # the single d = 256 layer's update, bf16 weights with fp32 masters
        dict(name="adamw_layer", op="adamw", layers=1, d_model=256, heads=4, d_head=64, param="bf16", grad="f32",
             master=True, copy=True, bits=32, step=3),
        # the 8-layer stack's update
        dict(name="adamw_stack", op="adamw", layers=8, d_model=1024, heads=8, d_head=128, param="bf16", grad="f32",
             master=True, copy=True, bits=32, step=1000),
        # the same with 8-bit states
        dict(name="adamw_stack_8bit", op="adamw", layers=8, d_model=1024, heads=8, d_head=128, param="bf16",
             grad="f32", master=True, copy=True, bits=8, step=1000),
        # touched rows of a bf16 table, 8-bit states
        dict(name="adamw_rows_8bit", op="adamw_rows", rows=200000, d=512, touched=14011, cap=38070, param="bf16",
             grad="f32", master=False, bits=8, step=57),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "gradient", "gradient", "norm", "adamw", "adamw", "adamw_rows"])
    wide = rng.choice([8, 50, 64, 100, 128, 200, 256, 257, 512, 768, 1000, 1024])
    if op == "lookup":
        return dict(op=op, tokens=_log(rng, 1, 40000), rows=_log(rng, 8, 1000000), actions=rng.choice([0, 8]),
                    d=wide, table=rng.choice(["bf16", "f16", "f32"]), out=rng.choice(["bf16", "f16", "f32"]),
                    scale=rng.choice([1.0, math.sqrt(wide)]), pad=rng.random() < 0.5)
    if op == "gradient":
        tokens, rows = _log(rng, 1, 80000), _log(rng, 8, 1000000)
        return dict(op=op, tokens=tokens, rows=rows, actions=rng.choice([0, 8]), d=wide,
                    dy=rng.choice(["bf16", "f16", "f32"]), out=rng.choice(["f32", "f32", "bf16"]),
                    scale=rng.choice([1.0, math.sqrt(wide)]), pad=rng.random() < 0.5,
                    compact=rows > 70000 or rng.random() < 0.5, accumulate=False)
    if op == "norm":
        return dict(op=op, layers=rng.randint(1, 8), d_model=rng.choice([64, 256, 512, 1024]), heads=rng.choice([2, 4, 8]),
                    d_head=rng.choice([64, 128]), grad=rng.choice(["f32", "bf16"]), rows=rng.choice([0, _log(rng, 1, 10000)]))
    if op == "adamw":
        bits = rng.choice([32, 8])
        return dict(op=op, layers=rng.randint(1, 8), d_model=rng.choice([64, 192, 256, 512, 1024]),
                    heads=rng.choice([2, 4, 8]), d_head=rng.choice([64, 128]),
                    param=rng.choice(["bf16", "f16", "f32"]), grad=rng.choice(["f32", "bf16"]),
                    master=rng.random() < 0.5, copy=rng.random() < 0.5, bits=bits, step=_log(rng, 1, 100000))
    rows = _log(rng, 8, 150000)
    cap = _log(rng, 1, 30000)
    return dict(op=op, rows=rows, d=min(wide, 512), touched=rng.randint(0, min(cap, rows)), cap=cap,
                param=rng.choice(["bf16", "f32"]), grad=rng.choice(["f32", "bf16"]), master=rng.random() < 0.5,
                bits=rng.choice([32, 8]), step=_log(rng, 1, 100000))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ids(case, g):
    """Zipf(1.1) content ids under a fixed permutation; with an action table behind the catalog, odd positions are its
    rows; with padding one token in 16 is the pad id 0."""
    T, R = case["tokens"], case["rows"]
    p = torch.arange(1, R + 1, device="cuda", dtype=torch.float64).pow(-1.1).cumsum(0)
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * p[-1]
    ids = torch.searchsorted(p, u).clamp_(max=R - 1)
    odd = 0x9E3779B1
    while math.gcd(odd, R) != 1:
        odd += 2
    ids = (ids * odd + 12345) % R
    if case["actions"]:
        a = torch.randint(0, case["actions"], (T,), generator=g, device="cuda") + R
        ids = torch.where(torch.arange(T, device="cuda") % 2 == 1, a, ids)
    if case["pad"]:
        ids = torch.where(torch.rand(T, generator=g, device="cuda") < 1 / 16, torch.zeros_like(ids), ids)
    return ids


def _tensors(case):
    """(elements, decayed) of a stack's parameters, those of the fp32 bias tables last."""
    d, h, e = case["d_model"], case["heads"], case["d_head"]
    F, hdv = 4 * h * e, h * e
    dense = [(F * d, True), (d * hdv, True)] * case["layers"]
    plain = [(F, False), (d, False), (hdv, False), (hdv, False)] * case["layers"]
    bias = [(h * 128, False), (h * 128, False)] * case["layers"]
    return dense + plain, bias


def _offsets(sizes):
    """Start of each tensor in a flat buffer, every one at a multiple of BLOCK, and the buffer's length."""
    at, o = [], 0
    for n, _ in sizes:
        at.append(o)
        o += -(-n // BLOCK) * BLOCK
    return at, o


def _live(sizes, total):
    """Truth value per flat element: inside a tensor (not the gap behind it)."""
    at, _ = _offsets(sizes)
    m = np.zeros(total // BLOCK, np.int64) + BLOCK
    for (n, _), o in zip(sizes, at):
        if n % BLOCK:
            m[(o + n) // BLOCK] = n % BLOCK
    e = torch.arange(BLOCK, device="cuda")
    return (e < torch.from_numpy(m).cuda()[:, None]).reshape(-1)


def _group(sizes, first, g, case, param, copy):
    """One flat buffer set for tensors `sizes`, the first of them number `first` of the step's list."""
    at, n = _offsets(sizes)
    live = _live(sizes, n)
    r = lambda s: torch.randn(n, generator=g, device="cuda") * s * live  # noqa: E731
    p = r(0.05)
    q = dict(sizes=sizes, at=at, first=first, grad=r(1e-3).to(DT[case["grad"]]),
             param=p.to(param), decayed=sum(-(-k // BLOCK) * BLOCK for k, w in sizes if w),
             master=p if case["master"] and param != torch.float32 else None)
    q["copy"] = torch.zeros(q["decayed"], dtype=torch.float16, device="cuda") if copy and q["decayed"] else None
    blocks = [-(-k // BLOCK) for k, _ in sizes]
    q["ordinal"] = torch.repeat_interleave(torch.arange(first, first + len(sizes)), torch.tensor(blocks)).cuda()
    q["block"] = torch.from_numpy(np.concatenate([np.arange(b) for b in blocks])).cuda()
    _moments(q, r(2e-4), (r(1e-3).square() * 0.5), case, n // BLOCK, BLOCK)
    return q


def _moments(q, m, v, case, blocks, width):
    if case["bits"] == 32:
        q["m"], q["v"] = m, v
        return
    z = torch.full((blocks, width), 0x8000, dtype=torch.int64, device="cuda")
    q["m"], q["m_scale"] = _encode(m.view(blocks, width), z)
    q["v"], q["v_scale"] = _encode(v.sqrt().view(blocks, width), z)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case, seed=seed)
    op = case["op"]
    if op in ("lookup", "gradient"):
        s["ids"] = _ids(case, g)
        T, R, d = case["tokens"], case["rows"] + case["actions"], case["d"]
        if op == "lookup":
            s["table"] = torch.empty(R, d, dtype=DT[case["table"]], device="cuda").normal_(generator=g)
            s["out"] = torch.empty(T, d, dtype=DT[case["out"]], device="cuda")
        else:
            s["dY"] = (torch.randn(T, d, generator=g, device="cuda") * 0.1).to(DT[case["dy"]])
            if case["compact"]:
                cap = min(T, R)
                s["row_ids"] = torch.full((cap,), -1, dtype=torch.int64, device="cuda")
                s["grad"] = torch.zeros(cap, d, dtype=DT[case["out"]], device="cuda")
                s["count"] = torch.zeros(1, dtype=torch.int64, device="cuda")
            else:
                s["grad"] = torch.zeros(R, d, dtype=DT[case["out"]], device="cuda")
    elif op == "norm":
        a, b = _tensors(case)
        s["sizes"] = a + b
        s["at"], n = _offsets(s["sizes"])
        s["grad"] = (torch.randn(n, generator=g, device="cuda") * 1e-3 * _live(s["sizes"], n)).to(DT[case["grad"]])
        if case["rows"]:
            s["rows"] = torch.randn(case["rows"], case["d_model"], generator=g, device="cuda") * 1e-3
            s["count"] = torch.tensor([case["rows"]], device="cuda")
        s["out"] = torch.empty(2, device="cuda")
    elif op == "adamw":
        a, b = _tensors(case)
        s["groups"] = [_group(a, 0, g, case, DT[case["param"]], case["copy"]),
                       _group(b, len(a), g, case, torch.float32, False)]
        s["grad_scale"] = torch.rand(1, generator=g, device="cuda") * 0.5 + 0.5
    else:
        R, d, U = case["rows"], case["d"], case["touched"]
        nb = -(-d // BLOCK)
        pick = torch.randperm(R, generator=g, device="cuda")[:U].sort()[0]
        s["row_ids"] = torch.full((case["cap"],), -1, dtype=torch.int64, device="cuda")
        s["row_ids"][:U] = pick
        s["count"] = torch.tensor([U], device="cuda")
        grad = torch.zeros(case["cap"], d, device="cuda")
        grad[:U].normal_(std=1e-3, generator=g)
        s["grad"] = grad.to(DT[case["grad"]])
        p = torch.randn(R, d, generator=g, device="cuda")
        s["param"] = p.to(DT[case["param"]])
        s["master"] = p if case["master"] and case["param"] != "f32" else None
        m = torch.randn(R, d, generator=g, device="cuda") * 2e-4
        v = torch.randn(R, d, generator=g, device="cuda").square() * 5e-7
        if case["bits"] == 8:
            m, v = (torch.nn.functional.pad(x, (0, nb * BLOCK - d)) for x in (m, v))
        _moments(s, m, v, case, R * nb, BLOCK)
        if case["bits"] == 8:
            s["m"], s["v"] = (x.view(R, nb * BLOCK)[:, :d].contiguous() for x in (s["m"], s["v"]))
        s["grad_scale"] = torch.rand(1, generator=g, device="cuda") * 0.5 + 0.5
    if own:
        _plan(s)
    return s


# ------------------------------------------------------------------ the library's calls
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)
DECAY = 0.1
MAX_NORM = 1.0


def _plan(s):
    """What a training program keeps: the workspace and, for the tensor lists, the list laid out once."""
    import hstu_sequential_transducer_layer_b200 as H
    s["H"] = H
    case, op = s["case"], s["case"]["op"]
    ws = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    if op == "lookup":
        s["ws"] = ws(H.hstu_embed_workspace_size())
    elif op == "gradient":
        s["ws"] = ws(H.hstu_embed_bwd_workspace_size(case["tokens"], case["rows"] + case["actions"], case["d"]))
    elif op == "norm":
        ts = [dict(grad=s["grad"][o:o + n]) for (n, _), o in zip(s["sizes"], s["at"])]
        if case["rows"]:
            ts.append(dict(grad=s["rows"], n_rows=s["count"]))
        s["list"] = H.GradTensors(ts)
        s["ws"] = ws(H.hstu_grad_norm_workspace_size())
    elif op == "adamw":
        ts = []
        for q in s["groups"]:
            for (n, w), o in zip(q["sizes"], q["at"]):
                e = slice(o, o + n)
                t = dict(param=q["param"][e], grad=q["grad"][e], weight_decay=DECAY if w else 0.0)
                if q["master"] is not None:
                    t["master"] = q["master"][e]
                if q["copy"] is not None and w:
                    t["copy_f16"] = q["copy"][e]
                b = slice(o // BLOCK, -(-(o + n) // BLOCK))
                for k in ("m", "v"):
                    t[k] = q[k].view(-1)[e]
                    if case["bits"] == 8:
                        t[k + "_scale"] = q[k + "_scale"][b]
                ts.append(t)
        s["list"] = H.AdamWTensors(ts)
        s["ws"] = ws(H.hstu_adamw_workspace_size())
    else:
        t = {k: s[k] for k in ("param", "grad", "m", "v", "m_scale", "v_scale", "row_ids") if k in s}
        if s["master"] is not None:
            t["master"] = s["master"]
        s["list"] = H.AdamWTensors([dict(t, n_rows=s["count"], weight_decay=DECAY)])
        s["ws"] = ws(H.hstu_adamw_workspace_size())


def _own(s):
    H, case, op = s["H"], s["case"], s["case"]["op"]
    if op == "lookup":
        H.hstu_embed_fwd(s["ids"], s["table"], s["out"], s["ws"], scale=case["scale"], pad_id=0 if case["pad"] else -1)
    elif op == "gradient":
        pad = 0 if case["pad"] else -1
        if case["compact"]:
            H.hstu_embed_bwd_rows(s["ids"], s["dY"], case["rows"] + case["actions"], s["row_ids"], s["grad"], s["count"],
                                  s["ws"], scale=case["scale"], pad_id=pad)
        else:
            H.hstu_embed_bwd(s["ids"], s["dY"], s["grad"], s["ws"], scale=case["scale"], pad_id=pad,
                             accumulate=case["accumulate"])
    elif op == "norm":
        H.hstu_grad_norm(s["list"], MAX_NORM, s["out"], s["ws"])
    else:
        H.hstu_adamw_step(s["list"], s["ws"], step=case["step"], seed=s["seed"], grad_scale=s["grad_scale"], **HYPER)


# ------------------------------------------------------------------ the plain forms
def _lowbias(x):
    """The 32-bit integer mix x ^= x >> 16; x *= 0x7feb352d; x ^= x >> 15; x *= 0x846ca68b; x ^= x >> 16, in int64."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & M32
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & M32
    return x ^ (x >> 16)


def _shr(x, k):
    return (x >> k) & ((1 << (64 - k)) - 1)


def _i64(c):
    return c - (1 << 64) if c >= 1 << 63 else c


def _random(seed, step, ordinal, block):
    """Two 16-bit numbers for each element of each block of a tensor (`ordinal` in the step's list): SplitMix64 output
    number step * 2^20 + ordinal + 1 from state `seed` keys a 32-bit mix of the block's and the element's number."""
    z = ((ordinal + (step << 20) + 1) * _i64(GAMMA)) + seed
    z = (z ^ _shr(z, 30)) * _i64(0xBF58476D1CE4E5B9)
    z = (z ^ _shr(z, 27)) * _i64(0x94D049BB133111EB)
    z = z ^ _shr(z, 31)
    b = _lowbias(_lowbias((block & M32) ^ (z & M32)) ^ (block >> 32) ^ _shr(z, 32))
    x = _lowbias((b[:, None] + torch.arange(BLOCK, device=b.device) * 0x9E3779B9) & M32)
    return x & 0xFFFF, x >> 16


def _encode(x, r):
    """8-bit codes [blocks, BLOCK] and scale bytes [blocks] of fp32 x: the scale 2^(byte - 127) puts the block's largest
    finite magnitude into [2^7, 2^8); each scaled value is rounded up or down to a neighbouring e4m3 value, up when the
    16-bit number r is at least 2^16 times what is missing to it; values that are not finite become NaN."""
    a = x.abs()
    fine = torch.isfinite(a)
    top = torch.where(fine, a, torch.zeros_like(a)).amax(1)
    byte = ((top.view(torch.int32) >> 23) - 7).clamp_(1, 247)
    inv = ((254 - byte) << 23).view(torch.float32)
    t = a * inv[:, None]
    sub = t < 2.0 ** -6
    t = torch.where(sub, t + 2.0 ** -6, t)
    c = ((t.view(torch.int32).to(torch.int64) + (r << 4)) >> 20) - torch.where(sub, 968, 960)
    c = torch.where(fine, c, torch.full_like(c, 0x7F)) | (x.view(torch.int32) < 0).to(torch.int64) << 7
    return c.to(torch.uint8), byte.to(torch.uint8)


def _decode(code, byte):
    return code.view(torch.float8_e4m3fn).float() * (byte.to(torch.int32) << 23).view(torch.float32)[:, None]


def _update(p, grad, m, v, case, wd):
    """m, v, p after one step, in fp32, from fp32 gradients already scaled."""
    b1, b2, t = HYPER["beta1"], HYPER["beta2"], case["step"]
    m = m * b1 + grad * (1 - b1)
    v = v * b2 + grad * grad * (1 - b2)
    u = m / (v.sqrt() / math.sqrt(1 - b2 ** t) + HYPER["eps"])
    return m, v, p * (1 - HYPER["lr"] * wd) - u * (HYPER["lr"] / (1 - b1 ** t))


def _plain_group(q, s):
    case, n = s["case"], q["decayed"]
    g = q["grad"].float() * s["grad_scale"]
    wide = q["param"].float() if q["master"] is None else q["master"]
    if case["bits"] == 32:
        m, v = q["m"], q["v"]
    else:
        m = _decode(q["m"], q["m_scale"]).view(-1)
        v = _decode(q["v"], q["v_scale"]).view(-1).square()
    wd = torch.zeros_like(wide)
    wd[:n] = DECAY
    m, v, p = _update(wide, g, m, v, case, wd)
    if case["bits"] == 32:
        q["m"].copy_(m)
        q["v"].copy_(v)
    else:
        lo, hi = _random(s["seed"], case["step"], q["ordinal"], q["block"])
        for k, x, r in (("m", m, lo), ("v", v.sqrt(), hi)):
            c, b = _encode(x.view(-1, BLOCK), r)
            q[k].copy_(c)
            q[k + "_scale"].copy_(b)
    if q["master"] is not None:
        q["master"].copy_(p)
    q["param"].copy_(p)
    if q["copy"] is not None:
        q["copy"].copy_(q["param"][:n].float().clamp(-65504, 65504))


def _plain_rows(s):
    case = s["case"]
    U, d = case["touched"], case["d"]
    nb = -(-d // BLOCK)
    r = s["row_ids"][:U]
    g = s["grad"][:U].float() * s["grad_scale"]
    wide = (s["param"] if s["master"] is None else s["master"])[r].float()
    if case["bits"] == 32:
        m, v = s["m"][r], s["v"][r]
    else:
        at = (r[:, None] * nb + torch.arange(nb, device="cuda")).view(-1)
        full = lambda x: torch.nn.functional.pad(x, (0, nb * BLOCK - d)).view(-1, BLOCK)  # noqa: E731
        m = _decode(full(s["m"][r]), s["m_scale"][at]).view(U, -1)[:, :d]
        v = _decode(full(s["v"][r]), s["v_scale"][at]).view(U, -1)[:, :d].square()
    m, v, p = _update(wide, g, m, v, case, DECAY)
    if case["bits"] == 32:
        s["m"][r], s["v"][r] = m, v
    else:
        lo, hi = _random(s["seed"], case["step"], torch.zeros_like(at), at)
        for k, x, n in (("m", m, lo), ("v", v.sqrt(), hi)):
            c, b = _encode(full(x).contiguous(), n)
            s[k][r], s[k + "_scale"][at] = c.view(U, -1)[:, :d], b
    if s["master"] is not None:
        s["master"][r] = p
    s["param"][r] = p.to(s["param"].dtype)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "lookup":
        y = s["table"][s["ids"]].float() * case["scale"]
        if case["pad"]:
            y = y * (s["ids"] != 0)[:, None]
        s["out"].copy_(y)
    elif op == "gradient":
        R = case["rows"] + case["actions"]
        dY = s["dY"].float() * case["scale"]
        key = torch.where(s["ids"] == 0, R, s["ids"]) if case["pad"] else s["ids"]
        if case["compact"]:
            key, order = key.sort(stable=True)
            head = torch.ones_like(key)
            head[1:] = key[1:] != key[:-1]
            seg = head.cumsum(0) - 1
            live = key < R
            rows = torch.zeros(case["tokens"], case["d"], device="cuda").index_add_(0, seg, dY[order] * live[:, None])
            cap = s["row_ids"].numel()
            n = (head * live).sum().view(1)
            at = torch.arange(cap, device="cuda")
            s["count"].copy_(n)
            first = torch.full((case["tokens"] + 1,), R, device="cuda").scatter_(0, seg, key)[:cap]
            s["row_ids"].copy_(torch.where(at < n, first, s["row_ids"]))
            s["grad"].copy_(torch.where((at < n)[:, None], rows[:cap], s["grad"].float()))
        else:
            acc = torch.zeros(R + 1, case["d"], device="cuda").index_add_(0, key, dY)[:R]
            s["grad"].copy_(s["grad"].float() + acc if case["accumulate"] else acc)
    elif op == "norm":
        n = s["grad"].double().square().sum()
        if case["rows"]:
            n = n + s["rows"].double().square().sum()
        n = n.sqrt()
        s["out"].copy_(torch.stack([n, (MAX_NORM / n).clamp(max=1.0)]))
    elif op == "adamw":
        _plain_group(s["groups"][0], s)
        _plain_group(s["groups"][1], s)
    elif case["touched"]:
        _plain_rows(s)


def _state_out(q):
    """The state's buffers as the values that their bytes stand for."""
    r = {k: q[k] for k in ("param", "master", "copy") if q.get(k) is not None}
    for k in ("m", "v"):
        if k + "_scale" in q:
            r[k] = q[k].view(torch.float8_e4m3fn)
            r[k + "_scale"] = q[k + "_scale"].view(torch.float8_e8m0fnu)
        else:
            r[k] = q[k]
    return r


def run(state):
    if own:
        _own(state)
    else:
        _plain(state)
    op = state["case"]["op"]
    if op in ("lookup", "norm"):
        return state["out"]
    if op == "gradient":
        return {k: state[k] for k in ("row_ids", "grad", "count") if k in state}
    if op == "adamw":
        return [_state_out(q) for q in state["groups"]]
    return _state_out(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _unique(case):
    """Expected number of different ids of _ids()."""
    T, R = case["tokens"], case["rows"]
    p = np.arange(1, R + 1, dtype=np.float64) ** -1.1
    n = T - T // 2 if case["actions"] else T
    u = float((1 - np.exp(n * np.log1p(-p / p.sum() + 1e-300))).sum())
    return min(u + min(case["actions"], T // 2), T)


def work(case):
    op = case["op"]
    if op == "lookup":
        T, d = case["tokens"], case["d"]
        return dict(bytes=8 * T + _unique(case) * d * SIZE[case["table"]] + T * d * SIZE[case["out"]], flops=T * d)
    if op == "gradient":
        T, d, R, e = case["tokens"], case["d"], case["rows"] + case["actions"], SIZE[case["out"]]
        u = _unique(case)
        out = u * (8 + d * e) if case["compact"] else 2 * u * d * e if case["accumulate"] else R * d * e
        return dict(bytes=8 * T + T * d * SIZE[case["dy"]] + out, flops=2 * T * d)
    if op == "norm":
        a, b = _tensors(case)
        n = sum(k for k, _ in a + b)
        r = case["rows"] * case["d_model"]
        return dict(bytes=n * SIZE[case["grad"]] + r * 4, flops=2 * (n + r))
    state = 16 if case["bits"] == 32 else 4 + 4 / BLOCK
    if op == "adamw":
        a, b = _tensors(case)
        n, nb = sum(k for k, _ in a), sum(k for k, _ in b)
        nc = sum(k for k, w in a if w)
        p = SIZE[case["param"]]
        p = (8 + p) if case["master"] and case["param"] != "f32" else 2 * p
        by = n * (p + SIZE[case["grad"]] + state) + nb * (8 + SIZE[case["grad"]] + state) + 2 * nc * case["copy"]
        return dict(bytes=by, flops=16 * (n + nb))
    n = case["touched"] * case["d"]
    p = SIZE[case["param"]]
    p = (8 + p) if case["master"] and case["param"] != "f32" else 2 * p
    return dict(bytes=n * (p + SIZE[case["grad"]] + state) + 8 * case["touched"] + 8, flops=16 * n + 1)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _quantised(x, r):
    """Values of the 8-bit codes and of the scales of x [blocks, BLOCK] in fp64, by real arithmetic: k puts the largest
    magnitude into [2^7, 2^8); y = x / 2^k is rounded on the grid of step 2^(max(floor(log2 |y|), -6) - 3)."""
    top = x.abs().amax(1)
    k = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 7, torch.full_like(top, -126)).clamp(-126, 120)
    y = x.abs() / torch.exp2(k)[:, None]
    e = torch.floor(torch.log2(y.clamp(min=2.0 ** -6)))
    grid = torch.exp2(e - 3)
    q = torch.floor(y / grid + r.double() / 65536) * grid
    return torch.copysign(q, x), torch.exp2(k)


def _adamw64(p, g, m, v, step, wd):
    m = HYPER["beta1"] * m + (1 - HYPER["beta1"]) * g
    v = HYPER["beta2"] * v + (1 - HYPER["beta2"]) * g ** 2
    mh, vh = m / (1 - HYPER["beta1"] ** step), v / (1 - HYPER["beta2"] ** step)
    return p - HYPER["lr"] * (mh / (torch.sqrt(vh) + HYPER["eps"]) + wd * p), m, v


def _old(x, scale, shape):
    """A state buffer's values in fp64 (`scale`: one byte per block of x, or None)."""
    if scale is None:
        return x.double()
    return (x.view(torch.float8_e4m3fn).double().view(shape) * torch.exp2(scale.double() - 127).view(shape[0], 1))


def _exact_group(q, s):
    case, B = s["case"], (q["block"].numel(), BLOCK)
    wd = torch.zeros(q["param"].numel(), dtype=torch.float64, device="cuda")
    wd[:q["decayed"]] = DECAY
    p = (q["param"] if q["master"] is None else q["master"]).double()
    m, v = _old(q["m"], q.get("m_scale"), B).view(-1), _old(q["v"], q.get("v_scale"), B).view(-1)
    p, m, v = _adamw64(p, q["grad"].double() * s["grad_scale"].double(), m, v if case["bits"] == 32 else v ** 2,
                       case["step"], wd)
    out = dict(param=p)
    if q["master"] is not None:
        out["master"] = p
    if q["copy"] is not None:
        out["copy"] = p[:q["decayed"]].to(q["param"].dtype).double()
    if case["bits"] == 32:
        return dict(out, m=m, v=v)
    lo, hi = _random(s["seed"], case["step"], q["ordinal"], q["block"])
    out["m"], out["m_scale"] = _quantised(m.view(B), lo)
    out["v"], out["v_scale"] = _quantised(v.sqrt().view(B), hi)
    return out


def _exact_rows(s):
    case, out = s["case"], {}
    U, d, R = case["touched"], case["d"], case["rows"]
    nb = -(-d // BLOCK)
    r = s["row_ids"][:U]
    at = (r[:, None] * nb + torch.arange(nb, device="cuda")).view(-1)
    wide = lambda x: torch.nn.functional.pad(x, (0, nb * BLOCK - d))  # noqa: E731
    if case["bits"] == 8:
        m, v = (_old(wide(s[k][r]).contiguous(), s[k + "_scale"][at], (U * nb, BLOCK)).view(U, -1)[:, :d] for k in "mv")
        v = v ** 2
    else:
        m, v = s["m"][r].double(), s["v"][r].double()
    p = (s["param"] if s["master"] is None else s["master"])[r].double()
    p, m, v = _adamw64(p, s["grad"][:U].double() * s["grad_scale"].double(), m, v, case["step"], DECAY)
    out["param"] = s["param"].double()
    out["param"][r] = p
    if s["master"] is not None:
        out["master"] = s["master"].double()
        out["master"][r] = p
    if case["bits"] == 32:
        for k, x in (("m", m), ("v", v)):
            out[k] = s[k].double()
            out[k][r] = x
        return out
    lo, hi = _random(s["seed"], case["step"], torch.zeros_like(at), at)
    for k, x, n in (("m", m, lo), ("v", v.sqrt(), hi)):
        c, b = _quantised(wide(x).reshape(-1, BLOCK), n)
        out[k] = s[k].view(torch.float8_e4m3fn).double()
        out[k][r] = c.view(U, -1)[:, :d]
        out[k + "_scale"] = torch.exp2(s[k + "_scale"].double() - 127)
        out[k + "_scale"][at] = b
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        y = case["scale"] * s["table"].index_select(0, s["ids"]).double()
        if case["pad"]:
            y[s["ids"] == 0] = 0
        return y
    if op == "gradient":
        R = case["rows"] + case["actions"]
        w = s["dY"].double() * case["scale"]
        if case["pad"]:
            w[s["ids"] == 0] = 0
        if not case["compact"]:
            return dict(grad=s["grad"].double().index_add_(0, s["ids"], w), row_ids=None, count=None)
        rows, slot = s["ids"].unique(return_inverse=True)
        if case["pad"] and bool((rows == 0).any()):
            rows, slot = rows[1:], slot - 1        # the pad id sorts first
        g = torch.zeros(s["grad"].shape, dtype=torch.float64, device="cuda")
        g.index_add_(0, slot.clamp(min=0), w)
        return dict(grad=g, row_ids=None, count=None)
    if op == "norm":
        n = math.sqrt(sum(float((x.double() ** 2).sum()) for x in (s["grad"], s.get("rows")) if x is not None))
        return torch.tensor([n, min(1.0, MAX_NORM / n)], dtype=torch.float64)
    if op == "adamw":
        return [_exact_group(q, s) for q in s["groups"]]
    return _exact_rows(s)
