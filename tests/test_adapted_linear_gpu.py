"""AdaptedLinear: the frozen low-bit layer and its adapters run together, serving and training, against the frozen
layer's own results plus the 64-bit adapter."""
from __future__ import annotations

import pytest
import torch

from quantized_gemm_group_b200 import adapters, bq, synth

from . import adapter_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def layer(bits, K=1024, N=384, R=16, dtype="bf16"):
    W = synth.normal((N, K), 0.02, seed=bits, dtype="f16", device=DEV)
    pool = synth.adapters(3, R, K, N, seed=5, dtype=dtype, device=DEV, ranks=[R, 7, 0])
    return adapters.AdaptedLinear(W, bits, *pool)


@pytest.mark.parametrize("bits", [4, 2])
@pytest.mark.parametrize("lens", [[1, 1, 1, 1, 1], [40, 3, 100]])
def test_serving(bits, lens):
    ly = layer(bits)
    M = sum(lens) + 2                                    # two padding rows
    x = synth.activations(M, ly.K, seed=9, device=DEV)
    segs = adapters.segments(lens, [i % 4 - 1 for i in range(len(lens))])
    y = ly(x, segs)
    base = bq.bq_linear(x, *ly.weights, ly.N, ly.bits, ly.group)
    w, b, _, _ = ref.lora(x, ly.A, ly.B, ly.ranks, ly.scales, *segs, base=base)
    ref.assert_within("y", y, w, b)
    assert torch.equal(y[sum(lens):], base[sum(lens):])
    out = torch.empty_like(y)
    assert ly(x, segs, out=out) is out and torch.equal(out, y)
    assert bq.bq_device_status() == bq.BQ_OK


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lens", [[5, 9, 2], [40, 3, 100]])
def test_training_step(lens, dtype):
    ly = layer(4, dtype=dtype)
    M, p = sum(lens), 0.1
    x, dy = (synth.activations(M, c, seed=s, dtype=dtype, device=DEV) for c, s in ((ly.K, 9), (ly.N, 10)))
    segs = adapters.segments(lens, [0, 1, 0])
    rng = torch.tensor([3, 4], dtype=torch.int64, device=DEV)
    y, saved = ly.forward(x, segs, p, rng)
    rng[1] += 1                                          # the next step's masks; this step's backward keeps its own
    dx, dA, dB = ly.backward(dy, saved)
    rng[1] -= 1
    pool = (ly.A, ly.B, ly.ranks, ly.scales, *segs)
    base = bq.bq_linear(x, *ly.weights, ly.N, ly.bits, ly.group)
    w, b, _, _ = ref.lora(x, *pool, base=base, p=p, rng=rng)
    ref.assert_within("y", y, w, b)
    dbase = bq.bq_linear_grad_input(dy, *ly.weights, ly.K, ly.bits, ly.group)
    wx, bx, wA, bA, wB, bB = ref.lora_grad(dy, x, saved[1], *pool, base=dbase, p=p, rng=rng)
    ref.assert_within("dx", dx, wx, bx)
    ref.assert_within("dA", dA, wA, bA)
    ref.assert_within("dB", dB, wB, bB)
    assert bq.bq_device_status() == bq.BQ_OK


def test_segments_are_checked():
    with pytest.raises(ValueError):
        adapters.segments([1, 2], [0])
    with pytest.raises(ValueError):
        adapters.segments([1, -2], [0, 1])


def test_rows_with_a_stride():
    """Slices of a fused tensor give what their dense copies give; an output with strides is refused."""
    ly = layer(4)
    lens = [40, 3, 100]
    M = sum(lens)
    wide = lambda cols, seed: synth.activations(M, cols + 48, seed=seed, device=DEV)[:, 24:24 + cols]  # noqa: E731
    x, dy = wide(ly.K, 3), wide(ly.N, 4)
    segs = adapters.segments(lens, [0, 1, 0])
    assert torch.equal(ly(x, segs), ly(x.contiguous(), segs))
    y, saved = ly.forward(x, segs)
    want, kept = ly.forward(x.contiguous(), segs)
    assert torch.equal(y, want)
    for a, b in zip(ly.backward(dy, saved), ly.backward(dy.contiguous(), kept)):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        ly(x, segs, out=wide(ly.N, 5))
    with pytest.raises(ValueError):
        ly(x, segs, out=torch.empty((M + 1, ly.N), dtype=x.dtype, device=DEV))
    W = synth.normal((ly.N, 2 * ly.K), 0.02, seed=4, dtype="f16", device=DEV)[:, ::2]
    pool = (ly.A, ly.B, ly.ranks, ly.scales)
    a, b = adapters.AdaptedLinear(W, 4, *pool), adapters.AdaptedLinear(W.contiguous(), 4, *pool)
    assert all(torch.equal(p, q) for p, q in zip(a.weights, b.weights))
