"""bq_lora_grad through the C entry with single gradients wanted, which the binding does not ask for."""
from __future__ import annotations

import pytest
import torch

from quantized_gemm_group_b200 import bq

from . import adapter_ref as ref
from .test_lora_gpu import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def grad(c, t, dA=None, dB=None, dt=None, **kw):
    """The status of a call for dA or dB alone; kw: other values of the named fields."""
    f = dict(dy=c.dy, x=c.x if dA is not None else None, t=t if dB is not None else None, A=c.A, B=c.B, ranks=c.ranks,
             scales=c.scales, seg_off=c.seg_off, seg_adapter=c.seg_adapter, rng=c.rng, base=None, dx=None, dt=dt, dA=dA, dB=dB)
    f.update(kw)
    ptrs = [0 if v is None else v.data_ptr() for v in f.values()]
    args = bq._LORA_GRAD_ARGS.pack(*ptrs, c.M, c.K, c.N, c.N, c.K, 0, 0, c.p, c.R, c.L, c.seg_adapter.shape[0],
                                   bq.DTYPE_CODE[c.dtype])
    return bq.lib().bq_lora_grad(args, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("lens", [[5, 9], [130, 77]])
def test_one_gradient_alone(lens):
    c = Case(264, 520, 40, [40, 12], lens, [0, 1], p=0.1)
    t = torch.zeros((c.M, c.R), device=DEV)
    c.forward(t=t)
    _, wA, wB = c.grad(t)
    dA, dB, dt = torch.full_like(wA, 3.0), torch.full_like(wB, 3.0), torch.zeros((c.M, c.R), device=DEV)
    assert grad(c, t, dB=dB) == bq.BQ_OK and torch.equal(dB, wB)
    assert grad(c, t, dA=dA, dt=dt) == bq.BQ_OK and torch.equal(dA, wA)
    assert bq.bq_device_status() == bq.BQ_OK


@pytest.mark.parametrize("lens", [[4, 6, 5], [150, 60, 90]])
def test_bad_segments_are_recorded_for_db_alone(lens):
    c = Case(136, 200, 16, [16, 8], lens, [0, 1, 0])
    t = torch.zeros((c.M, c.R), device=DEV)
    c.forward(t=t)
    dB = torch.zeros(c.B.shape, device=DEV)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    off = c.seg_off.tolist()
    for kw in (dict(seg_adapter=i32([0, 2, 0])), dict(seg_adapter=i32([0, -2, 0])), dict(ranks=i32([16, 17])),
               dict(seg_off=i32([0, off[1], off[2], c.M + 1])), dict(seg_off=i32([off[1], 0, off[2], off[3]]))):
        assert grad(c, t, dB=dB, **kw) == bq.BQ_OK
        assert bq.bq_device_status() == bq.BQ_ERR_UNSUPPORTED, kw
    assert grad(c, t, dB=dB) == bq.BQ_OK and bq.bq_device_status() == bq.BQ_OK
    # what a bad segment would add is left out: the others' sums
    assert grad(c, t, dB=dB, seg_adapter=i32([0, 2, 0])) == bq.BQ_OK
    keep = i32([0, -1, 0])
    w = ref.lora_grad(c.dy, c.x, t, c.A, c.B, c.ranks, c.scales, c.seg_off, keep)
    ref.assert_within("dB", dB, w[4], w[5])
    assert bq.bq_device_status() == bq.BQ_ERR_UNSUPPORTED
