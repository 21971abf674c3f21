"""Cases for measuring the low-rank adapter operators that run beside the weight-only linear layer, and dropout.

Three operators, each in two forms.  With ``own`` false, ``run`` computes the plain form: elementary torch operations
in 32 bits, rounded once.  With ``own`` true it makes the calls that a user makes of the library's kernels.

``lora``     y = base + scale[a] (drop(x) A[a]^T) B[a]^T for rows grouped into segments, each with an adapter a of a pool
             (or none); with ``save`` it also returns t = drop(x) A[a]^T, which the backward pass reads
``lora_grad`` dx = base + drop'(scale[a] (dy B[a]) A[a]), dA[a], dB[a]
``dropout``  y = x mask / (1 - p), the mask drawn from a counter-based generator (Philox 4x32-10) and never stored

A row behind the last segment is left as it was.  The mask of element (i, j) is a 16-bit field of one generator block:
key (seed), counter (j / 8, i, offset), field j % 8; it is kept where the field is at least round(p 65536).
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
WIDTHS = {"bf16": 2, "f16": 2, "f32": 4}


def _lora(name, op, tokens, k, n, r, adapters, segments, dtype="bf16", ranks="same", p=0.0, save=False, idle=False,
          tail=0, strided=False):
    return {"name": name, "op": op, "tokens": tokens, "k": k, "n": n, "r": r, "adapters": adapters,
            "segments": segments, "dtype": dtype, "ranks": ranks, "p": p, "save": save, "idle": idle, "tail": tail,
            "strided": strided}


def _drop(name, rows, cols, dtype, p, strided=False):
    return {"name": name, "op": "dropout", "rows": rows, "cols": cols, "dtype": dtype, "p": p, "strided": strided}


def listed():
    return [
        # one request, one new token, the output projection of a layer: launch latency
        _lora("lora_1_token", "lora", 1, 4096, 4096, 16, 8, 1),
        # 16 requests, each with its own adapter of a pool with mixed ranks, one new token each, the down projection
        _lora("lora_16_requests", "lora", 16, 14336, 4096, 64, 32, 16, ranks="mixed"),
        # a decode batch: adapters shared by neighbours, requests without one, padding rows behind the last, the query
        # slice of a fused output, odd sizes and fp16
        _lora("lora_61_ragged", "lora", 61, 1032, 1000, 24, 5, 9, "f16", "mixed", idle=True, tail=4, strided=True),
        # prompts of five requests in one batch, the gate-and-up projection: writing y bounds it
        _lora("lora_prompt_2048", "lora", 2048, 4096, 28672, 16, 4, 5, ranks="mixed", idle=True),
        # the largest prompt batch, the down projection: reading x bounds it
        _lora("lora_prompt_8192", "lora", 8192, 14336, 4096, 64, 8, 13),
        # training forward of one adapter with dropout, t kept for the backward pass
        _lora("lora_train_4096", "lora", 4096, 4096, 4096, 64, 1, 1, p=0.05, save=True),
        # backward of a short ragged batch over three adapters, fp16, odd sizes, one adapter twice
        _lora("grad_37_ragged", "lora_grad", 37, 520, 264, 8, 3, 5, "f16", "mixed", p=0.1, idle=True, tail=3),
        # backward of one adapter with dropout at an ordinary training length
        _lora("grad_4096", "lora_grad", 4096, 4096, 4096, 16, 1, 1, p=0.05),
        # backward of four adapters trained at once, the gate projection: the largest backward
        _lora("grad_8192_4_adapters", "lora_grad", 8192, 4096, 14336, 64, 4, 8),
        # the input of one token: launch latency
        _drop("dropout_1_row", 1, 4096, "bf16", 0.1),
        # odd rows and columns, fp32, rows with a stride
        _drop("dropout_odd_f32", 1001, 1033, "f32", 0.3, True),
        # the activations of a long training batch
        _drop("dropout_8192x14336", 8192, 14336, "bf16", 0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("lora", "lora", "lora_grad", "dropout"))
    if op == "dropout":
        cols = _log(rng, 5, 14336)
        return {"op": op, "rows": min(_log(rng, 1, 16384), (8192 * 14336) // cols // 2), "cols": cols,
                "dtype": rng.choice(("bf16", "f16", "f32")), "p": round(rng.uniform(0.0, 0.6), 3),
                "strided": rng.random() < 0.3}
    tokens = _log(rng, 1, 8192)
    r = 8 * _log(rng, 1, 16)
    adapters = _log(rng, 1, max(1, 512 // r))
    tail = rng.choice((0, 0, rng.randrange(0, 9)))
    case = {"op": op, "tokens": tokens, "k": 8 * _log(rng, 8, 1792), "n": 8 * _log(rng, 8, 1792), "r": r,
            "adapters": adapters, "segments": _log(rng, 1, min(64, tokens)), "dtype": rng.choice(("bf16", "bf16", "f16")),
            "ranks": rng.choice(("same", "mixed")), "p": rng.choice((0.0, 0.0, 0.05, 0.15)),
            "save": op == "lora" and rng.random() < 0.4, "idle": rng.random() < 0.4,
            "tail": min(tail, tokens - 1), "strided": rng.random() < 0.3}
    # no more than the largest listed cases
    while (case["tokens"] * (case["k"] + case["n"]) * case["r"] > 8192 * (14336 + 4096) * 64
           or case["tokens"] * (case["k"] + 2 * case["n"] + (2 * case["k"] if op == "lora_grad" else 0)) > 150_000_000):
        case["tokens"] = max(1, case["tokens"] * 2 // 3)
        case["segments"] = min(case["segments"], case["tokens"])
        case["tail"] = min(case["tail"], case["tokens"] - 1)
    return case


def _plan(case):
    """Segment offsets, the segments' adapters and the adapters' ranks: fixed by the case alone."""
    rows, S, L, R = case["tokens"] - case["tail"], case["segments"], case["adapters"], case["r"]
    rng = random.Random("%d %d %d %d" % (rows, S, L, R))
    if S >= rows:
        cuts = list(range(rows)) + [rows] * (S - rows)
        cuts = sorted(cuts)[:S]
        off = [0] + cuts[1:] + [rows]
    else:
        off = [0] + sorted(rng.sample(range(1, rows), S - 1)) + [rows]
    adapter = [-1 if case["idle"] and i % 4 == 3 else (i * 7) % L for i in range(S)]
    if case["ranks"] == "same":
        ranks = [R] * L
    else:
        ranks = [(R, max(1, R // 2), max(1, R // 4 + 1), max(1, R - 3))[i % 4] for i in range(L)]
    return off, adapter, ranks


def _wide(shape, dtype, std, gen, strided):
    """[rows, cols] of N(0, std): contiguous, or 24 columns inside a wider matrix, as a slice of a fused projection is."""
    rows, cols = shape
    pad = 24 if strided else 0
    t = (torch.randn((rows, cols + 2 * pad), generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)
    return t[:, pad:pad + cols]


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]
    rng = torch.tensor([(int(seed) * 2654435761 + 12345) % (1 << 62), int(seed) % 1000], dtype=torch.int64, device="cuda")
    if case["op"] == "dropout":
        shape = (case["rows"], case["cols"])
        return {"x": _wide(shape, dtype, 1.0, gen, case["strided"]), "rng": rng, "p": case["p"]}
    off, adapter, ranks = _plan(case)
    M, K, N, R, L = case["tokens"], case["k"], case["n"], case["r"], case["adapters"]
    s = {"x": _wide((M, K), dtype, 1.0, gen, case["strided"]),
         "A": (torch.randn((L, R, K), generator=gen, device="cuda") / math.sqrt(K)).to(dtype),
         "B": (torch.randn((L, N, R), generator=gen, device="cuda") * 0.05).to(dtype),
         "ranks": torch.tensor(ranks, dtype=torch.int32, device="cuda"),
         "scales": torch.tensor([2.0 / (1 + i % 3) for i in range(L)], dtype=torch.float32, device="cuda"),
         "seg_off": torch.tensor(off, dtype=torch.int32, device="cuda"),
         "seg_adapter": torch.tensor(adapter, dtype=torch.int32, device="cuda"),
         "rng": rng, "p": case["p"]}
    if case["op"] == "lora":
        s["base"] = _wide((M, N), dtype, 1.0, gen, case["strided"])
    else:
        s["dy"] = _wide((M, N), dtype, 0.02, gen, case["strided"])
        s["base"] = _wide((M, K), dtype, 0.02, gen, case["strided"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"] = case["op"]
    if case["op"] == "dropout":
        s["out"] = torch.zeros_like(s["x"])
        return s
    # the buffers that a program keeps: outputs, and t as the forward pass left it
    s["out"] = torch.zeros((case["tokens"], s["base"].shape[1]), dtype=s["base"].dtype, device="cuda")
    if case["op"] == "lora":
        s["t"] = torch.zeros((case["tokens"], case["r"]), device="cuda") if case["save"] else None
    else:
        s["t"] = _plain_t(s, *_rows(s))
        s["dA"] = torch.zeros(s["A"].shape, device="cuda")
        s["dB"] = torch.zeros(s["B"].shape, device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

_M32 = 0xFFFFFFFF


def _mul32(a, m):
    """High and low 32 bits of a * m, a in [0, 2^32) held in 64 bits (the low 64 bits of the product are exact)."""
    q = a * m
    return (q >> 32) & _M32, q & _M32


def _fields(rows, cols, rng):
    """The 16-bit fields of the elements of a rows x cols matrix."""
    blocks = (cols + 7) // 8
    c = [torch.arange(blocks, device=rng.device).expand(rows, blocks),
         torch.arange(rows, device=rng.device)[:, None].expand(rows, blocks),
         (rng[1] & _M32).expand(rows, blocks), ((rng[1] >> 32) & _M32).expand(rows, blocks)]
    k = [rng[0] & _M32, (rng[0] >> 32) & _M32]
    for _ in range(10):
        h0, l0 = _mul32(c[0], 0xD2511F53)
        h1, l1 = _mul32(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k[0], l1, h0 ^ c[3] ^ k[1], l0]
        k = [(k[0] + 0x9E3779B9) & _M32, (k[1] + 0xBB67AE85) & _M32]
    words = torch.stack(c, dim=-1)
    return torch.stack([words & 0xFFFF, words >> 16], dim=-1).reshape(rows, blocks * 8)[:, :cols]


def _threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def _plain_drop(x, p, rng):
    """x mask / (1 - p) in 32 bits."""
    thr = _threshold(p)
    x = x.float()
    if thr == 0:
        return x
    keep = _fields(x.shape[0], x.shape[1], rng) >= thr
    return torch.where(keep, x * (65536.0 / (65536 - thr)), torch.zeros((), device=x.device))


def _rows(s):
    """Each row's adapter (0 where it has none), whether it has one, and whether it is in a segment."""
    M = s["x"].shape[0]
    row = torch.arange(M, device=s["x"].device)
    seg = torch.searchsorted(s["seg_off"][1:].contiguous(), row.to(torch.int32), right=True)
    inside = seg < s["seg_adapter"].shape[0]
    a = s["seg_adapter"][seg.clamp(max=s["seg_adapter"].shape[0] - 1)].long()
    has = inside & (a >= 0)
    return torch.where(has, a, torch.zeros_like(a)), has, inside


def _weights(s):
    """The adapters in 32 bits, zero behind their ranks."""
    live = torch.arange(s["A"].shape[1], device=s["A"].device)[None, :] < s["ranks"][:, None]
    zero = torch.zeros((), device=s["A"].device)
    return torch.where(live[:, :, None], s["A"].float(), zero), torch.where(live[:, None, :], s["B"].float(), zero)


def _down(v, w, a, has):
    """v[m] . w[a[m]]^T, w [L, R, C]; zero for rows without an adapter."""
    L, R, C = w.shape
    if v.shape[0] < L:
        t = torch.bmm(w[a], v[:, :, None])[:, :, 0]
    else:
        t = (v @ w.reshape(L * R, C).t()).view(-1, L, R).gather(1, a[:, None, None].expand(-1, 1, R))[:, 0]
    return torch.where(has[:, None], t, torch.zeros((), device=v.device))


def _spread(t, a, L):
    """t [M, R] at its adapter's place in [M, L * R], zero elsewhere."""
    M, R = t.shape
    return torch.zeros((M, L, R), device=t.device).scatter_(1, a[:, None, None].expand(-1, 1, R), t[:, None]).view(M, L * R)


def _up(t, w, a):
    """t[m] . w[a[m]], w [L, R, C]."""
    L, R, C = w.shape
    if t.shape[0] < L:
        return torch.bmm(t[:, None], w[a])[:, 0]
    return _spread(t, a, L) @ w.reshape(L * R, C)


def _plain_t(s, a, has, inside):
    return _down(_plain_drop(s["x"], s["p"], s["rng"]), _weights(s)[0], a, has)


def _plain_lora(s):
    a, has, inside = _rows(s)
    A, B = _weights(s)
    t = _down(_plain_drop(s["x"], s["p"], s["rng"]), A, a, has)
    y = s["base"].float() + _up(t * s["scales"][a][:, None], B.transpose(1, 2), a)
    s["out"].copy_(torch.where(inside[:, None], y, s["out"].float()))
    if s["t"] is None:
        return {"y": s["out"]}
    s["t"].copy_(torch.where(inside[:, None], t, s["t"]))
    return {"y": s["out"], "t": s["t"]}


def _plain_grad(s):
    a, has, inside = _rows(s)
    A, B = _weights(s)
    L = A.shape[0]
    dy, xd, scale = s["dy"].float(), _plain_drop(s["x"], s["p"], s["rng"]), s["scales"][a][:, None]
    dt = _down(dy, B.transpose(1, 2), a, has) * scale
    delta = _plain_drop(_up(dt, A, a), s["p"], s["rng"])
    s["out"].copy_(torch.where(inside[:, None], s["base"].float() + delta, s["out"].float()))
    zero = torch.zeros((), device=dy.device)
    dyz, xz = torch.where(has[:, None], dy, zero), torch.where(has[:, None], xd, zero)
    s["dA"].copy_((_spread(dt, a, L).t() @ xz).view(s["dA"].shape))
    s["dB"].copy_((_spread(torch.where(has[:, None], s["t"], zero) * scale, a, L).t() @ dyz).view(L, -1, dy.shape[1]).transpose(1, 2))
    return {"dx": s["out"], "dA": s["dA"], "dB": s["dB"]}


def run(state):
    if own:
        from quantized_gemm_group_b200 import bq
        s = state
        if s["op"] == "dropout":
            return {"y": bq.bq_dropout(s["x"], s["p"], s["rng"], out=s["out"])}
        if s["op"] == "lora":
            y = bq.bq_lora(s["x"], s["A"], s["B"], s["ranks"], s["scales"], s["seg_off"], s["seg_adapter"],
                           base=s["base"], out=s["out"], p=s["p"], rng=s["rng"], t=s["t"])
            return {"y": y} if s["t"] is None else {"y": y, "t": s["t"]}
        dx, dA, dB = bq.bq_lora_grad(s["dy"], s["x"], s["t"], s["A"], s["B"], s["ranks"], s["scales"], s["seg_off"],
                                     s["seg_adapter"], base=s["base"], out=s["out"], p=s["p"], rng=s["rng"],
                                     dA=s["dA"], dB=s["dB"])
        return {"dx": dx, "dA": dA, "dB": dB}
    if state["op"] == "dropout":
        state["out"].copy_(_plain_drop(state["x"], state["p"], state["rng"]))
        return {"y": state["out"]}
    return _plain_lora(state) if state["op"] == "lora" else _plain_grad(state)


def work(case):
    """Each input read once, each output written once; adapters in use only, up to their ranks."""
    w = WIDTHS[case["dtype"]]
    if case["op"] == "dropout":
        e = case["rows"] * case["cols"]
        return {"bytes": 2 * w * e, "flops": e}
    off, adapter, ranks = _plan(case)
    K, N, R = case["k"], case["n"], case["r"]
    rows = [off[i + 1] - off[i] for i in range(len(adapter))]
    busy = [(m, ranks[l]) for m, l in zip(rows, adapter) if l >= 0 and m > 0]
    used = sum(ranks[l] for l in {l for m, l in zip(rows, adapter) if l >= 0 and m > 0})
    m_all, m_busy, mr = sum(rows), sum(m for m, _ in busy), sum(m * r for m, r in busy)
    weights = used * (K + N) * w
    if case["op"] == "lora":
        saved = 4 * m_all * R if case["save"] else 0
        return {"bytes": m_busy * K * w + 2 * m_all * N * w + weights + saved, "flops": 2 * mr * (K + N)}
    grads = 4 * case["adapters"] * R * (K + N)
    return {"bytes": m_busy * (N + K) * w + 4 * mr + 2 * m_all * K * w + weights + grads, "flops": 4 * mr * (K + N)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_keep(rows, cols, seed, offset, thr):
    """Kept elements, with the generator in unsigned 64-bit host integers."""
    u = np.uint64
    blocks = (cols + 7) // 8
    low, shift = u(0xFFFFFFFF), u(32)
    c0, c1 = np.meshgrid(np.arange(blocks, dtype=u), np.arange(rows, dtype=u))
    c2, c3 = np.full_like(c0, offset & 0xFFFFFFFF), np.full_like(c0, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for i in range(10):
        a, b = c0 * u(0xD2511F53), c2 * u(0xCD9E8D57)
        c0, c1, c2, c3 = (b >> shift) ^ c1 ^ u(k0), b & low, (a >> shift) ^ c3 ^ u(k1), a & low
        k0, k1 = (k0 + 0x9E3779B9) % (1 << 32), (k1 + 0xBB67AE85) % (1 << 32)
    keep = np.empty((rows, blocks, 8), dtype=bool)
    for i, c in enumerate((c0, c1, c2, c3)):
        keep[:, :, 2 * i] = (c & u(0xFFFF)) >= thr
        keep[:, :, 2 * i + 1] = (c >> u(16)) >= thr
    return torch.from_numpy(keep.reshape(rows, blocks * 8)[:, :cols])


def exact(case, seed):
    s = _inputs(case, seed)
    thr = _threshold(case["p"])
    factor = 65536.0 / (65536 - thr)
    first = s["x"]
    keep = None
    if thr:
        at = s["rng"].tolist()
        keep = _exact_keep(first.shape[0], first.shape[1], at[0], at[1], thr).to(first.device)

    def dropped(v):
        return v if keep is None else torch.where(keep, v * factor, torch.zeros_like(v))

    if case["op"] == "dropout":
        return {"y": dropped(s["x"].double())}
    off, adapter, ranks = _plan(case)
    scales = s["scales"].double().tolist()
    x = dropped(s["x"].double())
    M, R = case["tokens"], case["r"]
    t = torch.zeros((M, R), dtype=torch.float64, device=x.device)
    out = torch.zeros((M, s["base"].shape[1]), dtype=torch.float64, device=x.device)
    out[:off[-1]] = s["base"][:off[-1]].double()
    if case["op"] == "lora":
        for i, l in enumerate(adapter):
            if l >= 0 and off[i + 1] > off[i]:
                m, r = slice(off[i], off[i + 1]), ranks[l]
                t[m, :r] = x[m] @ s["A"][l, :r].double().t()
                out[m] += scales[l] * (t[m, :r] @ s["B"][l, :, :r].double().t())
        return {"y": out, "t": t} if case["save"] else {"y": out}
    dA = torch.zeros(s["A"].shape, dtype=torch.float64, device=x.device)
    dB = torch.zeros(s["B"].shape, dtype=torch.float64, device=x.device)
    delta = torch.zeros_like(out)
    for i, l in enumerate(adapter):
        if l >= 0 and off[i + 1] > off[i]:
            m, r = slice(off[i], off[i + 1]), ranks[l]
            dy, A, B = s["dy"][m].double(), s["A"][l, :r].double(), s["B"][l, :, :r].double()
            dt = scales[l] * (dy @ B)
            delta[m] = dt @ A
            dA[l, :r] += dt.t() @ x[m]
            dB[l, :, :r] += scales[l] * (dy.t() @ (x[m] @ A.t()))
    return {"dx": out + dropped(delta), "dA": dA, "dB": dB}
