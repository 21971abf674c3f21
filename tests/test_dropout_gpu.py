"""bq_dropout against a plain implementation in 64 bits: the mask of the same counter-based generator bit for bit, the
kept values within the one rounding of the output type."""
from __future__ import annotations

import pytest
import torch

from quantized_gemm_group_b200 import bq

from . import adapter_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def rng_of(seed=0x1234567890ABCDEF, offset=77):
    return torch.tensor([seed, offset], dtype=torch.int64, device=DEV)


def want_of(x, p, rng):
    f = ref.keep_factor(x.shape[0], x.shape[1], p, rng)
    return ref.drop(x.double(), f), f


def check(x, p, rng, y):
    w, f = want_of(x, p, rng)
    u = ref.HALF_STEP[x.dtype]
    if x.dtype == torch.float32:
        u += 2.0 ** -24              # 65536 / (65536 - thr) is itself rounded to fp32
    else:
        u += 2.0 ** -22              # and the fp32 product, before the rounding to 16 bits
    ref.assert_within("y", y, w, u * w.abs() + ref.TINY[x.dtype])
    if f is not None:
        assert bool(((y == 0) | (f > 0)).all()) and bool(((y != 0) | (f == 0) | (x == 0)).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (2, 9), (5, 64), (17, 1033), (64, 4096), (300, 264)])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_against_plain(dtype, rows, cols, p):
    x = torch.randn((rows, cols), device=DEV).to(dtype)
    rng = rng_of(offset=rows)
    check(x, p, rng, bq.bq_dropout(x, p, rng))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,first", [(8, 8), (8, 4), (5, 1), (3, 0)])
def test_strided_rows_and_odd_alignment(dtype, pad, first):
    wide = torch.randn((33, 200 + pad), device=DEV).to(dtype)
    x = wide[:, first:first + 200]
    out_wide = torch.full((33, 211), 7.0, device=DEV).to(dtype)
    out = out_wide[:, 3:203]
    rng = rng_of()
    assert bq.bq_dropout(x, 0.25, rng, out=out).data_ptr() == out.data_ptr()
    check(x, 0.25, rng, out)
    assert bool((out_wide[:, :3] == 7).all()) and bool((out_wide[:, 203:] == 7).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_dropped_places_are_zero_whatever_they_hold(dtype):
    x = torch.randn((16, 512), device=DEV).to(dtype)
    rng = rng_of()
    f = ref.keep_factor(16, 512, 0.4, rng)
    x[f == 0] = float("nan")
    x[0][f[0] == 0] = float("inf")
    y = bq.bq_dropout(x, 0.4, rng)
    assert bool(torch.isfinite(y).all()) and bool((y[f == 0] == 0).all())


def test_p_zero_copies_bits_and_needs_no_generator():
    x = torch.randn((9, 100), device=DEV).to(torch.bfloat16)
    x[0, 0], x[1, 1], x[2, 2] = float("nan"), float("inf"), -0.0
    for p in (0.0, 2.0 ** -18):
        y = bq.bq_dropout(x, p)
        assert torch.equal(y.view(torch.int16), x.view(torch.int16))


def test_in_place_and_gradient_is_the_same_map():
    x = torch.randn((40, 1000), device=DEV)
    dy = torch.randn((40, 1000), device=DEV)
    rng = rng_of()
    y, dx = bq.bq_dropout(x, 0.3, rng), bq.bq_dropout(dy, 0.3, rng)
    # y is linear in x: the inner products with dy and with its gradient agree up to fp32 rounding of each element
    f = ref.keep_factor(40, 1000, 0.3, rng)
    assert torch.equal(dx == 0, f == 0)
    lhs, rhs = (y.double() * dy.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(float(lhs - rhs)) <= 2.0 ** -22 * float((y.double() * dy.double()).abs().sum())
    # against differences: the map is linear, so a difference quotient is exact up to rounding
    d = torch.randn_like(x)
    quotient = (bq.bq_dropout(x + d, 0.3, rng).double() - bq.bq_dropout(x - d, 0.3, rng).double()) / 2
    ref.assert_within("quotient", quotient, d.double() * f, 2.0 ** -21 * (x.abs() + d.abs()).double() * f + 1e-30)
    z = x.clone()
    assert bq.bq_dropout(z, 0.3, rng, out=z) is z and torch.equal(z, y)


@pytest.mark.parametrize("p", [2.0 ** -16, 0.05, 0.9, 1 - 2.0 ** -16])
def test_share_of_kept_elements(p):
    """The number kept is binomial: within 6 standard deviations of its mean."""
    n = 1 << 22
    y = bq.bq_dropout(torch.ones((1024, n // 1024), device=DEV), p, rng_of(5, 9))
    kept, mean = int((y != 0).sum()), n * (1 - p)
    assert abs(kept - mean) <= 6 * (n * p * (1 - p)) ** 0.5 + 1


def test_seed_and_offset_give_other_masks():
    x = torch.ones((64, 1024), device=DEV)
    masks = [bq.bq_dropout(x, 0.5, rng_of(s, o)) != 0 for s, o in ((1, 1), (2, 1), (1, 2), (1 + (1 << 32), 1), (1, 1 + (1 << 32)))]
    for i in range(len(masks)):
        for j in range(i):
            same = float((masks[i] == masks[j]).double().mean())
            assert abs(same - 0.5) < 6 * 0.5 / 65536 ** 0.5


def test_graph_replay_reads_the_generator_again():
    x = torch.randn((32, 512), device=DEV)
    rng = rng_of(3, 0)
    out = torch.empty_like(x)
    bq.bq_dropout(x, 0.2, rng, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bq.bq_dropout(x, 0.2, rng, out=out)
    for step in range(3):
        rng[1] = step
        g.replay()
        check(x, 0.2, rng, out)


def test_other_stream():
    x = torch.randn((256, 4096), device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(x)
    bq.bq_dropout(x, 0.1, rng_of(), out=out, stream=s)
    s.synchronize()
    check(x, 0.1, rng_of(), out)


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart."""
    stride = (1 << 30) + 64
    flat = torch.zeros(3 * stride, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(flat, (4, 48), (stride - 8192, 1))
    x.copy_(torch.randn((4, 48), device=DEV))
    rng = rng_of()
    check(x, 0.5, rng, bq.bq_dropout(x, 0.5, rng))
    out = torch.as_strided(flat, (4, 48), (stride - 8192, 1), 64)
    bq.bq_dropout(x, 0.5, rng, out=out)
    check(x, 0.5, rng, out)


def test_empty():
    for shape in ((0, 8), (8, 0)):
        assert bq.bq_dropout(torch.empty(shape, device=DEV), 0.5, rng_of()).shape == shape
