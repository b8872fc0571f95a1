"""Plain float64 forms of the training-side operators: embedding lookup with
scaling and its gradient, the global gradient norm, AdamW, and the 8-bit
states' codes (there also a float32 form with one rounding per operation,
which the stored bytes must equal).  numpy only, no code of the library."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 256


# ---------------------------------------------------------------- embedding
def _keep(ids, n_rows, pad):
    ids = np.asarray(ids, np.int64)
    return (ids != pad) & (ids >= 0) & (ids < n_rows)


def embed_fwd(ids, table, scale, pad=-1):
    table = np.asarray(table, np.float64)
    keep = _keep(ids, len(table), pad)
    out = np.zeros((len(ids), table.shape[1]))
    out[keep] = scale * table[np.asarray(ids)[keep]]
    return out


def embed_bwd(ids, dY, n_rows, scale, pad=-1):
    """(dense gradient, sum of |scale dY| per element, tokens per row)."""
    dY = np.asarray(dY, np.float64)
    g, a = np.zeros((n_rows, dY.shape[1])), np.zeros((n_rows, dY.shape[1]))
    n = np.zeros(n_rows, np.int64)
    keep = _keep(ids, n_rows, pad)
    for t in np.flatnonzero(keep):
        r = int(ids[t])
        g[r] += scale * dY[t]
        a[r] += abs(scale) * np.abs(dY[t])
        n[r] += 1
    return g, a, n


# ---------------------------------------------------------------- optimizer
def grad_norm(grads, max_norm):
    """(norm, clip factor) of a list of arrays; (norm, NaN) if not finite."""
    with np.errstate(over="ignore", invalid="ignore"):
        n = math.sqrt(math.fsum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads)) \
            if all(np.isfinite(g).all() for g in grads) else math.nan
    if not n <= float(np.finfo(np.float32).max):
        return n, math.nan
    return n, min(1.0, max_norm / n) if n > 0 else 1.0


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after one step, float64."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * weight_decay * p - lr * mh / (np.sqrt(vh) + eps), m, v


# ---------------------------------------------------------------- 8-bit states
def _mix32(x):
    x = np.asarray(x, np.uint32).copy()
    x ^= x >> np.uint32(16)
    x *= np.uint32(0x7FEB352D)
    x ^= x >> np.uint32(15)
    x *= np.uint32(0x846CA68B)
    return x ^ (x >> np.uint32(16))


def random16(seed, step, ordinal, blocks):
    """The two 16-bit numbers of each element of the given block numbers:
    uint32 arrays [len(blocks), BLOCK] for m and for r = sqrt(v)."""
    mask = (1 << 64) - 1
    z = (seed + ((step << 20) + ordinal + 1) * 0x9E3779B97F4A7C15) & mask
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
    z ^= z >> 31
    b = np.asarray(blocks, np.uint64)
    lo, hi = (b & np.uint64(0xFFFFFFFF)).astype(np.uint32), (b >> np.uint64(32)).astype(np.uint32)
    with np.errstate(over="ignore"):
        base = _mix32(_mix32(lo ^ np.uint32(z & 0xFFFFFFFF)) ^ hi ^ np.uint32(z >> 32))
        e = np.arange(BLOCK, dtype=np.uint32) * np.uint32(0x9E3779B9)
        x = _mix32(base[:, None] + e[None, :])
    return x & np.uint32(0xFFFF), x >> np.uint32(16)


_E4M3 = np.array([(-1.0 if c & 128 else 1.0) *
                  ((c & 7) / 8 * 2.0 ** -6 if (c >> 3) & 15 == 0 else
                   (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7))
                  for c in range(256)])
_E4M3[[0x7F, 0xFF]] = np.nan


def decode(codes, scales):
    """float64 values of codes [blocks, n] with one scale byte per block."""
    s = np.where(scales == 0, 0.0, np.exp2(scales.astype(np.float64) - 127))
    return _E4M3[codes] * s[:, None]


def round_states(x, r16):
    """(values of the codes, scale exponents k) of x [blocks, n] by the
    definition in real arithmetic: 2^k puts the largest finite magnitude into
    [2^7, 2^8); |x| / 2^k is rounded on the grid of step 2^(max(floor(log2),
    -6) - 3), up when r16 / 2^16 reaches the missing part."""
    x = np.asarray(x, np.float64)
    top = np.where(np.isfinite(x), np.abs(x), 0).max(axis=1)
    k = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1))) - 7, -126)
    k = np.clip(k, -126, 120)
    y = np.abs(x) / np.exp2(k)[:, None]
    grid = np.exp2(np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    return np.copysign(np.floor(y / grid + r16 / 65536.0) * grid, x), k


def encode_f32(x, r16):
    """Codes and scale bytes of float32 x [blocks, n], operation by operation
    in float32."""
    x = np.asarray(x, np.float32)
    a = np.abs(x)
    fine = np.isfinite(a)
    top = np.where(fine, a, np.float32(0)).max(axis=1).astype(np.float32)
    byte = np.maximum(1, (top.view(np.uint32) >> 23).astype(np.int64) - 7)
    inv = ((254 - byte).astype(np.uint32) << np.uint32(23)).view(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        t = (a * inv[:, None]).astype(np.float32)
        sub = t < np.float32(2.0 ** -6)
        t = np.where(sub, t + np.float32(2.0 ** -6), t).astype(np.float32)
    c = ((t.view(np.uint32).astype(np.int64) + (r16.astype(np.int64) << 4)) >> 20) - \
        np.where(sub, 968, 960)
    c = np.where(fine, c, 0x7F) | ((x.view(np.uint32) >> np.uint32(31)).astype(np.int64) << 7)
    return c.astype(np.uint8), byte.astype(np.uint8)


def moments_f32(g, m, v, beta1, beta2, grad_scale=1.0):
    """m and v after one step in float32, one rounding per operation."""
    f = np.float32
    with np.errstate(over="ignore", invalid="ignore"):
        gg = f(grad_scale) * np.asarray(g, f)
        m = np.asarray(m, f) * f(beta1) + gg * f(1 - beta1)
        v = np.asarray(v, f) * f(beta2) + (gg * gg) * f(1 - beta2)
    return m, v


def adamw_step_8bit(codes_m, scale_m, codes_r, scale_r, g, seed, step, ordinal, blocks, beta1,
                    beta2, grad_scale=1.0):
    """The bytes that one step stores for blocks [blocks, n] (n <= BLOCK; the
    last block of a tensor may be shorter): (m codes, m scales, r codes, r
    scales), in float32."""
    n = codes_m.shape[1]
    old_r = decode(codes_r, scale_r).astype(np.float32)
    m, v = moments_f32(g, decode(codes_m, scale_m).astype(np.float32), old_r * old_r, beta1,
                       beta2, grad_scale)
    lo, hi = random16(seed, step, ordinal, blocks)
    with np.errstate(invalid="ignore"):
        r = np.sqrt(v)
    cm, sm = encode_f32(m, lo[:, :n])
    cr, sr = encode_f32(r, hi[:, :n])
    return cm, sm, cr, sr
