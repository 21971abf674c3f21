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
