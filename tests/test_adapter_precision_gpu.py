"""How exact the fp32 results of the adapters are over long contractions: t, dt, dA and dB against 64 bits, in the norm.

The element-wise bounds of adapter_ref grow with the length of a sum; these do not hide a sum that is kept in a tensor
core's accumulator for too long.  Such an accumulator loses up to one step of 2^-23 of the running sum at each
instruction (it cuts, so the losses do not cancel).  The kernels let at most 16 instructions of 16 products add up
there before fp32 additions that round to nearest take over.  For terms of random signs the running sum's norm grows
with the square root of the terms, so 16 instructions lose at most 16 * 2/3 * 2^-23 of it, and n rounded additions, whose
errors are independent, sqrt(n) * 2^-24; n is 64 for 16384 terms.  The kernel of short segments adds
the sums of two instructions, each possibly cutting twice, where a warp has more than 32 of them, up to 64 such sums."""
from __future__ import annotations

import pytest
import torch

from quantized_gemm_group_b200 import bq

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
LONG = 16 * 2 / 3 * 2.0 ** -23 + 8 * 2.0 ** -24     # 1.75e-6
SHORT = 4 * 2 / 3 * 2.0 ** -23 + 8 * 2.0 ** -24     # 0.80e-6


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def inputs(M, K, N, R, L, adapter, dtype, lens, seed=3):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=g, device=DEV) * std).to(dtype)  # noqa: E731
    x, dy, A, B = rnd(M, K), rnd(M, N, std=0.02), rnd(L, R, K, std=K ** -0.5), rnd(L, N, R, std=0.05)
    offs = [0]
    for n in lens:
        offs.append(offs[-1] + n)
    assert offs[-1] == M
    i32 = dict(dtype=torch.int32, device=DEV)
    tail = (torch.full((L,), R, **i32), torch.full((L,), 0.5, device=DEV), torch.tensor(offs, **i32),
            torch.full((len(lens),), adapter, **i32))
    return x, dy, A, B, tail


# rows and rank choose the kernel's clusters: two CTAs and one CTA each with one CTA an SM, one CTA with two an SM
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,R", [(9000, 64), (19000, 64), (9600, 128)])
def test_long_segments_down(M, R, dt):
    C = 14336
    x, dy, A, B, tail = inputs(M, C, 64, R, 2, 1, DT[dt], [M])
    t = torch.empty((M, R), device=DEV)
    bq.bq_lora(x, A, B, *tail, t=t)
    assert off(t, x.double() @ A[1].double().t()) <= LONG
    del x
    x, dy, A, B, tail = inputs(M, 64, C, R, 2, 1, DT[dt], [M])
    ws = torch.empty((M, R), device=DEV)
    bq.bq_lora_grad(dy, None, None, A, B, *tail, workspace=ws, need_weights=False)
    assert off(ws, 0.5 * (dy.double() @ B[1].double())) <= LONG


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("R", [16, 64, 128])
def test_short_segments_down(R, dt):
    """Enough segments that one CTA takes a tile's whole contraction."""
    C, lens = 14336, [20] * 160
    M = sum(lens)
    x, dy, A, B, tail = inputs(M, C, 64, R, 2, 1, DT[dt], lens)
    t = torch.empty((M, R), device=DEV)
    bq.bq_lora(x, A, B, *tail, t=t)
    assert off(t, x.double() @ A[1].double().t()) <= SHORT
    x, dy, A, B, tail = inputs(M, 64, C, R, 2, 1, DT[dt], lens)
    ws = torch.empty((M, R), device=DEV)
    bq.bq_lora_grad(dy, None, None, A, B, *tail, workspace=ws, need_weights=False)
    assert off(ws, 0.5 * (dy.double() @ B[1].double())) <= SHORT


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("K,N,R", [(4096, 16384, 64), (2048, 8192, 128)])
@pytest.mark.parametrize("lens", [[8229], [5000, 3001]])
def test_weight_gradients(K, N, R, lens, dt):
    """So many columns that one CTA takes all rows of a tile; dA against the dt that the call left in its workspace."""
    M = sum(lens)
    x, dy, A, B, tail = inputs(M, K, N, R, 2, 1, DT[dt], lens)
    t = x.float() @ A[1].float().t()
    ws = torch.empty((M, R), device=DEV)
    _, dA, dB = bq.bq_lora_grad(dy, x, t, A, B, *tail, workspace=ws, need_dx=False)
    assert off(dA[1], ws.double().t() @ x.double()) <= LONG
    assert off(dB[1], 0.5 * (dy.double().t() @ t.double())) <= LONG
    assert bool((dA[0] == 0).all()) and bool((dB[0] == 0).all())


# t enters its second product as two 16-bit parts of one sign.  The first is cut: bf16 keeps 8 bits and leaves less than
# 2^-7 of t, of which the second part's 8 bits lose half a step, 2^-9: 2^-16.  fp16 with 11 bits each: 2^-10 * 2^-11 (2^-12
# of a rest in [2^-11, 2^-10), so 2^-21 is safe).  A rest of 0 counts as 2^-24.  One product each, two cutting additions
# and the fp32 addition of the base: 3 * 2^-23.
PARTS = {torch.bfloat16: 2.0 ** -16 + 4 * 2.0 ** -23, torch.float16: 2.0 ** -21 + 4 * 2.0 ** -23}
STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("R", [8, 64, 128])
@pytest.mark.parametrize("M", [16, 200])
def test_second_product(M, R, dt):
    """Rank 1 and a single element of x (of dy) in each row, so that t (dt) is one exact product; the base is the negative
    result rounded to 16 bits, so that what is left shows the error of the product itself."""
    d = DT[dt]
    g = torch.Generator(device=DEV)
    g.manual_seed(M + R)
    rnd = lambda *s: (torch.rand(s, generator=g, device=DEV) + 1).to(d)  # noqa: E731
    one = dict(dtype=torch.int32, device=DEV)
    tail = (torch.ones(1, **one), torch.ones(1, device=DEV), torch.tensor([0, M], **one), torch.zeros(1, **one))
    N = 256
    v, first, up = rnd(M), rnd(1), rnd(N)
    x = torch.zeros((M, 8), dtype=d, device=DEV)
    x[:, 3] = v
    A, B = torch.zeros((1, R, 8), dtype=d, device=DEV), torch.zeros((1, N, R), dtype=d, device=DEV)
    A[0, 0, 3], B[0, :, 0] = first[0], up
    whole = (v.double() * first.double())[:, None] * up.double()[None]
    base = (-whole).to(d)
    want = whole + base.double()
    bound = whole * PARTS[d] + STEP[d] * want.abs() + 2.0 ** -25
    y = bq.bq_lora(x, A, B, *tail, base=base)
    assert bool(((y.double() - want).abs() <= bound).all())
    # the gradient: dy takes x's place, A and B each other's
    A, B = torch.zeros((1, R, N), dtype=d, device=DEV), torch.zeros((1, 8, R), dtype=d, device=DEV)
    B[0, 3, 0], A[0, 0] = first[0], up
    dx, _, _ = bq.bq_lora_grad(x, None, None, A, B, *tail, base=base, need_weights=False)
    assert bool(((dx.double() - want).abs() <= bound).all())
