"""Plain 64-bit implementations of dropout and of the low-rank adapters (torch float64, no code of the library), with
element-wise error bounds for the kernels' arithmetic.

Bounds.  u is half a step of the output type relative to the value (bf16 2^-8, fp16 2^-11, fp32 2^-24).  Products of
16-bit operands are exact in fp32; a sum of n of them in fp32 is off by at most n steps of 2^-23 of the sum of the
absolute values, whatever the order and whether additions round or truncate (SUM below, with a few spare steps for
the scale factors and the sums of partial sums).  t and dt enter their second product as 16-bit parts: bf16 hi + lo is
within 2^-16, bf16 three parts within 2^-23; fp16 parts within 2^-21 of the value and 2^-38 of the largest value that
shares their power of two (SPLIT)."""
from __future__ import annotations

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half a subnormal step


def SUM(n):
    return (n + 16) * 2.0 ** -23


def philox_fields(rows, cols, seed, offset):
    """The 16-bit fields, [rows, cols], of Philox 4x32-10 with key seed and counter (col / 8, row, offset)."""
    u = np.uint64
    low, sh = u(0xFFFFFFFF), u(32)
    blocks = (cols + 7) // 8
    c = [np.broadcast_to(np.arange(blocks, dtype=u)[None, :], (rows, blocks)).copy(),
         np.broadcast_to(np.arange(rows, dtype=u)[:, None], (rows, blocks)).copy(),
         np.full((rows, blocks), offset & 0xFFFFFFFF, dtype=u), np.full((rows, blocks), (offset >> 32) & 0xFFFFFFFF, dtype=u)]
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        p0, p1 = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(p1 >> sh) ^ c[1] ^ u(k0), p1 & low, (p0 >> sh) ^ c[3] ^ u(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    out = np.empty((rows, blocks, 8), dtype=np.int64)
    for i in range(4):
        out[:, :, 2 * i] = (c[i] & u(0xFFFF)).astype(np.int64)
        out[:, :, 2 * i + 1] = (c[i] >> u(16)).astype(np.int64)
    return out.reshape(rows, blocks * 8)[:, :cols]


def keep_factor(rows, cols, p, rng):
    """0 for a dropped element, 1 / (1 - p) for a kept one, float64 on rng's device; all ones where p rounds to 0."""
    thr = int(np.floor(p * 65536 + 0.5))
    if thr == 0:
        return None
    seed, offset = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    keep = philox_fields(rows, cols, seed, offset) >= thr
    return torch.from_numpy(keep).to(rng.device).double() * (65536.0 / (65536 - thr))


def drop(x, f):
    """x times the factors, 0 where the factor is 0 whatever x holds."""
    return x if f is None else torch.where(f > 0, x * f, torch.zeros_like(x))


def segments(seg_off, seg_adapter):
    off = seg_off.tolist()
    return [(off[i], off[i + 1], a) for i, a in enumerate(seg_adapter.tolist())]


def t_split(t, dtype):
    """Bound on what the 16-bit parts of t (hi + lo, a row shares its power of two) lose."""
    if dtype == torch.bfloat16:
        return t.abs() * 2.0 ** -16
    return t.abs() * 2.0 ** -21 + t.abs().amax(dim=1, keepdim=True) * 2.0 ** -38


def lora(x, A, B, ranks, scales, seg_off, seg_adapter, base=None, p=0.0, rng=None):
    """(y, bound, t, t bound) in float64; rows behind the last segment and without an adapter: base and zero."""
    M, K = x.shape
    L, N, R = B.shape
    f = keep_factor(M, K, p, rng)
    t = torch.zeros((M, R), dtype=torch.float64, device=x.device)
    et = torch.zeros_like(t)
    y = torch.zeros((M, N), dtype=torch.float64, device=x.device) if base is None else base.double().clone()
    ey = torch.zeros((M, N), dtype=torch.float64, device=x.device)
    for m0, m1, a in segments(seg_off, seg_adapter):
        r = int(ranks[a]) if a >= 0 else 0
        if m1 <= m0 or r == 0:
            continue
        s = float(scales[a].double())
        xd, Aa, Ba = drop(x[m0:m1].double(), None if f is None else f[m0:m1]), A[a, :r].double(), B[a, :, :r].double()
        tt = xd @ Aa.t()
        e = SUM(K) * (xd.abs() @ Aa.abs().t())
        t[m0:m1, :r], et[m0:m1, :r] = tt, e
        y[m0:m1] += s * (tt @ Ba.t())
        ey[m0:m1] = abs(s) * ((e + t_split(tt, x.dtype) + tt.abs() * SUM(R)) @ Ba.abs().t())
    u = HALF_STEP[x.dtype]
    bound = u * y.abs() + (1 + u) * (ey + 2.0 ** -23 * (y.abs() + ey)) + TINY[x.dtype]
    return y, bound, t, et + 2.0 ** -23 * t.abs()


def lora_grad(dy, x, t, A, B, ranks, scales, seg_off, seg_adapter, base=None, p=0.0, rng=None):
    """(dx, bound, dA, bound, dB, bound) in float64 for the t given (fp32)."""
    M, K = x.shape
    L, N, R = B.shape
    f = keep_factor(M, K, p, rng)
    dev = x.device
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)  # noqa: E731
    dx = z(M, K) if base is None else base.double().clone()
    ex, dA, eA, dB, eB = z(M, K), z(L, R, K), z(L, R, K), z(L, N, R), z(L, N, R)
    rows, largest_t, largest_dt = [0] * L, [0.0] * L, [0.0] * L
    part = 2.0 ** -23 if x.dtype == torch.bfloat16 else 2.0 ** -21
    for m0, m1, a in segments(seg_off, seg_adapter):
        r = int(ranks[a]) if a >= 0 else 0
        if m1 <= m0 or r == 0:
            continue
        s = float(scales[a].double())
        g, Aa, Ba = dy[m0:m1].double(), A[a, :r].double(), B[a, :, :r].double()
        fm = None if f is None else f[m0:m1]
        xd, tt = drop(x[m0:m1].double(), fm), t[m0:m1, :r].double()
        dt = s * (g @ Ba)
        e = abs(s) * SUM(N) * (g.abs() @ Ba.abs()) + 2.0 ** -23 * dt.abs()
        delta, ed = dt @ Aa, (e + t_split(dt, x.dtype) + dt.abs() * SUM(R)) @ Aa.abs()
        dx[m0:m1] += drop(delta, fm)
        ex[m0:m1] = drop(ed, fm)
        dA[a, :r] += dt.t() @ xd
        eA[a, :r] += (e + dt.abs() * part).t() @ xd.abs()
        dB[a, :, :r] += s * (g.t() @ tt)
        eB[a, :, :r] += abs(s) * part * (g.abs().t() @ tt.abs())
        rows[a] += m1 - m0
        largest_t[a], largest_dt[a] = max(largest_t[a], float(tt.abs().max())), max(largest_dt[a], float(dt.abs().max()))
    # fp32 sums over the adapter's rows, and fp16 parts share a power of two with the largest value
    for m0, m1, a in segments(seg_off, seg_adapter):
        r = int(ranks[a]) if a >= 0 else 0
        if m1 <= m0 or r == 0:
            continue
        s = float(scales[a].double())
        g, fm = dy[m0:m1].double(), None if f is None else f[m0:m1]
        xd, tt = drop(x[m0:m1].double(), fm), t[m0:m1, :r].double()
        dt = s * (g @ B[a, :, :r].double())
        floor = 0.0 if x.dtype == torch.bfloat16 else 2.0 ** -38
        eA[a, :r] += SUM(rows[a]) * (dt.abs().t() @ xd.abs()) + floor * largest_dt[a] * xd.abs().sum(0)
        eB[a, :, :r] += abs(s) * (SUM(rows[a]) * (g.abs().t() @ tt.abs()) + floor * largest_t[a] * g.abs().sum(0)[:, None])
    u = HALF_STEP[x.dtype]
    bx = u * dx.abs() + (1 + u) * (ex + 2.0 ** -23 * (dx.abs() + ex)) + TINY[x.dtype]
    return dx, bx, dA, eA + 2.0 ** -22 * dA.abs() + 1e-300, dB, eB + 2.0 ** -22 * dB.abs() + 1e-300


def assert_within(name, got, want, bound):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} elements outside their bound; first at {i}: "
                             f"{float(got.reshape(-1)[i])} against {float(want.reshape(-1)[i])} +- "
                             f"{float(bound.reshape(-1)[i])}")
