"""Infinite elements of the adapters' operands: every result is what the formula gives in 64 bits, an infinity of its
sign or NaN, and results that the element has no part in keep their bits."""
from __future__ import annotations

import pytest
import torch

from quantized_gemm_group_b200 import bq

from .test_lora_gpu import DT, Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


def same_kind(name, got, want, before):
    """NaN and infinities where the formula has them, elsewhere the bits from before the infinity came in."""
    got, want = got.double(), want.double()
    fine = torch.isfinite(want)
    assert bool((~fine).any()), name
    assert torch.equal(torch.isnan(got), torch.isnan(want)), name
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)]), name
    assert torch.equal(got[fine], before.double()[fine]), name


def case(lens, R, dt, p=0.0):
    return Case(264, 200, R, [R, R - 3], lens, [0, 1], dtype=DT[dt], p=p)


def segments(c):
    return [(a, slice(m0, m1), int(c.ranks[a])) for m0, m1, a in
            zip(c.seg_off.tolist(), c.seg_off.tolist()[1:], c.seg_adapter.tolist())]


def formula_y(c):
    y = c.base.double().clone()
    for a, m, r in segments(c):
        y[m] += float(c.scales[a]) * (c.x[m].double() @ c.A[a, :r].double().t()) @ c.B[a, :, :r].double().t()
    return y


def formula_grad(c, t):
    dx, dA, dB = c.dbase.double().clone(), torch.zeros_like(c.A.double()), torch.zeros_like(c.B.double())
    for a, m, r in segments(c):
        s, g = float(c.scales[a]), c.dy[m].double()
        d = s * (g @ c.B[a, :, :r].double())
        dx[m] += d @ c.A[a, :r].double()
        dA[a, :r] += d.t() @ c.x[m].double()
        dB[a, :, :r] += s * (g.t() @ t[m, :r].double())
    return dx, dA, dB


LENS = [[4, 3], [150, 65]]
RANKS = [16, 64, 128]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("R", RANKS)
@pytest.mark.parametrize("lens", LENS)
def test_weight_gradients(lens, R, dt):
    c = case(lens, R, dt)
    t = torch.zeros((c.M, R), device=DEV)
    c.forward(t=t)
    _, dA, dB = c.grad(t)
    x, dy = c.x.clone(), c.dy.clone()
    c.x[1, 9], c.x[lens[0] + 1, 200] = INF, -INF
    _, gA, gB = c.grad(t)
    same_kind("dA", gA, formula_grad(c, t)[1], dA)
    assert torch.equal(gB, dB)
    c.x = x
    c.dy[2, 6], c.dy[lens[0], 3] = -INF, INF
    _, gA, gB = c.grad(t)
    same_kind("dB", gB, formula_grad(c, t)[2], dB)
    same_kind("dA", gA, formula_grad(c, t)[1], dA)
    c.dy = dy
    t[1, 2], t[0, 0] = INF, -INF
    _, _, gB = c.grad(t)
    same_kind("dB", gB, formula_grad(c, t)[2], dB)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("R", RANKS)
@pytest.mark.parametrize("lens", LENS)
def test_outputs(lens, R, dt):
    """B in the forward pass and A in the gradient, one infinity in a column and two of either sign in another; x and dy."""
    c = case(lens, R, dt)
    y0 = c.forward()
    t = torch.zeros((c.M, R), device=DEV)
    c.forward(t=t)
    dx0 = c.grad(t, need_weights=False)[0]
    A, B, x, dy = (v.clone() for v in (c.A, c.B, c.x, c.dy))
    c.B[0, 5, 3] = c.B[1, 199, 0] = INF
    c.B[1, 64, 2], c.B[1, 64, 4] = -INF, INF
    same_kind("y", c.forward(), formula_y(c), y0)
    c.B.copy_(B)
    c.A[0, 3, 11] = c.A[1, 0, 263] = -INF
    c.A[1, 2, 70], c.A[1, 4, 70] = -INF, INF
    same_kind("dx", c.grad(t, need_weights=False)[0], formula_grad(c, t)[0], dx0)
    c.A.copy_(A)
    c.x[1, 7] = INF
    same_kind("y", c.forward(), formula_y(c), y0)
    c.x = x
    c.dy[2, 6] = -INF
    same_kind("dx", c.grad(t, need_weights=False)[0], formula_grad(c, t)[0], dx0)
    assert bq.bq_device_status() == bq.BQ_OK
