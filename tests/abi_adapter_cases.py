"""Argument-validation cases of the adapter and dropout entry points, with fake device pointers.

Never collected directly: tests/test_adapters_host.py runs this file in a child process with CUDA_VISIBLE_DEVICES set
to empty, so even a validation bug can only return an error code.  The only BQ_OK cases are calls that have nothing to
do."""
from __future__ import annotations

import os

import pytest

from quantized_gemm_group_b200 import bq

assert os.environ.get("CUDA_VISIBLE_DEVICES") == "", "run only through tests/test_adapters_host.py"

FAKE, MIS16, MIS4 = 0x7F0000001000, 0x7F0000001008, 0x7F0000001002


@pytest.fixture(scope="module")
def L():
    return bq.lib()


def dropout(L, x=FAKE, dtype=bq.BQ_BF16, rows=4, cols=16, ldx=16, p=0.1, rng=FAKE, out=FAKE, ldo=16):
    return L.bq_dropout(x, dtype, rows, cols, ldx, p, rng, out, ldo, None)


def test_dropout(L):
    assert dropout(L, rows=-1) == bq.BQ_ERR_SHAPE
    assert dropout(L, cols=-1) == bq.BQ_ERR_SHAPE
    assert dropout(L, ldx=8) == bq.BQ_ERR_SHAPE
    assert dropout(L, ldo=15) == bq.BQ_ERR_SHAPE
    assert dropout(L, dtype=7) == bq.BQ_ERR_UNSUPPORTED
    for p in (-0.1, 1.0, 1.5, float("nan"), float("inf"), 1 - 2.0 ** -18):
        assert dropout(L, p=p) == bq.BQ_ERR_UNSUPPORTED, p
    assert dropout(L, x=None) == bq.BQ_ERR_NULL
    assert dropout(L, out=None) == bq.BQ_ERR_NULL
    assert dropout(L, rng=None) == bq.BQ_ERR_NULL
    assert dropout(L, x=FAKE + 1) == bq.BQ_ERR_ALIGN
    assert dropout(L, dtype=bq.BQ_F32, out=MIS4) == bq.BQ_ERR_ALIGN
    assert dropout(L, rng=FAKE + 4) == bq.BQ_ERR_ALIGN
    assert dropout(L, rows=0, x=None, out=None) == bq.BQ_OK
    assert dropout(L, cols=0, x=None, out=None) == bq.BQ_OK


FORWARD = dict(x=FAKE, A=FAKE, B=FAKE, ranks=FAKE, scales=FAKE, seg_off=FAKE, seg_adapter=FAKE, rng=FAKE, base=FAKE, y=FAKE,
               t=FAKE, M=4, K=64, N=72, ldx=64, ldbase=72, ldy=72, p=0.1, R=16, L=2, S=1, dtype=bq.BQ_BF16)
GRAD = dict(dy=FAKE, x=FAKE, t=FAKE, A=FAKE, B=FAKE, ranks=FAKE, scales=FAKE, seg_off=FAKE, seg_adapter=FAKE, rng=FAKE,
            base=FAKE, dx=FAKE, dt=FAKE, dA=FAKE, dB=FAKE, M=4, K=64, N=72, lddy=72, ldx=64, ldbase=64, lddx=64, p=0.1, R=16,
            L=2, S=1, dtype=bq.BQ_BF16)


def forward(lib, **kw):
    assert set(kw) <= set(FORWARD)
    return lib.bq_lora(bq._LORA_ARGS.pack(*{**FORWARD, **kw}.values()), None)


def grad(lib, **kw):
    assert set(kw) <= set(GRAD)
    return lib.bq_lora_grad(bq._LORA_GRAD_ARGS.pack(*{**GRAD, **kw}.values()), None)


@pytest.mark.parametrize("f", [forward, grad])
def test_common(L, f):
    for kw in (dict(M=-1), dict(K=-8), dict(N=-8), dict(S=-1), dict(L=-1), dict(R=-8), dict(K=60), dict(N=76), dict(R=12),
               dict(M=(1 << 30) + 1), dict(K=(1 << 28) + 8), dict(N=(1 << 28) + 8), dict(ldx=60), dict(ldx=68),
               dict(ldbase=100)):
        assert f(L, **kw) == bq.BQ_ERR_SHAPE, kw
    for kw in (dict(R=0), dict(R=136), dict(dtype=bq.BQ_F32), dict(dtype=9), dict(p=1.0), dict(p=-1.0), dict(p=float("nan"))):
        assert f(L, **kw) == bq.BQ_ERR_UNSUPPORTED, kw
    for name in ("x", "A", "B", "ranks", "scales", "seg_off", "seg_adapter", "rng"):
        assert f(L, **{name: 0}) == bq.BQ_ERR_NULL, name
    for kw in (dict(x=MIS16), dict(A=MIS16), dict(B=MIS16), dict(base=MIS16), dict(t=MIS16), dict(ranks=MIS4),
               dict(scales=MIS4), dict(seg_off=MIS4), dict(seg_adapter=MIS4), dict(rng=FAKE + 4)):
        assert f(L, **kw) == bq.BQ_ERR_ALIGN, kw
    assert (L.bq_lora if f is forward else L.bq_lora_grad)(None, None) == bq.BQ_ERR_NULL


def test_forward(L):
    assert forward(L, y=0) == bq.BQ_ERR_NULL
    assert forward(L, y=MIS16) == bq.BQ_ERR_ALIGN
    assert forward(L, ldy=64) == bq.BQ_ERR_SHAPE
    assert forward(L, M=0, x=0, y=0) == bq.BQ_OK
    assert forward(L, S=0, x=0, y=0) == bq.BQ_OK


def test_grad(L):
    assert grad(L, dy=0) == bq.BQ_ERR_NULL
    assert grad(L, t=0) == bq.BQ_ERR_NULL
    assert grad(L, dt=0) == bq.BQ_ERR_NULL
    assert grad(L, dy=MIS16) == bq.BQ_ERR_ALIGN
    assert grad(L, dx=MIS16) == bq.BQ_ERR_ALIGN
    assert grad(L, dt=MIS16) == bq.BQ_ERR_ALIGN
    assert grad(L, dA=MIS16) == bq.BQ_ERR_ALIGN
    assert grad(L, dB=MIS16) == bq.BQ_ERR_ALIGN
    assert grad(L, lddx=60) == bq.BQ_ERR_SHAPE
    assert grad(L, lddy=76) == bq.BQ_ERR_SHAPE
    assert grad(L, M=0, dA=0, dB=0) == bq.BQ_OK               # no rows and no gradients of weights wanted
    assert grad(L, L=0, M=0) == bq.BQ_OK                      # no adapters: empty gradients


def test_in_place_means_the_same_rows(L):
    assert forward(L, ldbase=80) == bq.BQ_ERR_SHAPE
    assert grad(L, ldbase=80) == bq.BQ_ERR_SHAPE


def test_a_generator_is_wanted_without_rows_too(L):
    """dA and dB of an empty batch are still written by a kernel."""
    for kw in (dict(M=0), dict(S=0)):
        assert grad(L, rng=0, **kw) == bq.BQ_ERR_NULL
    assert grad(L, rng=0, M=0, p=0.0, dA=0, dB=0) == bq.BQ_OK


def test_dropout_in_place_means_the_same_rows(L):
    for kw in (dict(ldo=24), dict(ldx=24), dict(ldx=24, dtype=bq.BQ_F32)):
        assert dropout(L, **kw) == bq.BQ_ERR_SHAPE, kw
