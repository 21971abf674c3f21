"""A frozen low-bit linear layer with low-rank adapters: the packed weights stay as they are, adapters are served to
many requests at once or trained (QLoRA: a 4-bit frozen base and 16-bit adapters).

Serving: ``y = layer(x, segments)`` with the rows of the batch grouped by request.  Training: ``forward`` keeps what
the backward pass needs, ``backward`` returns the gradients of x and of the adapters.  Host logic only: the products
are bq_linear, bq_lora, bq_linear_grad_input and bq_lora_grad, each adapter added in place to the frozen layer's result.
"""
from __future__ import annotations

import torch

from . import bq


def segments(lengths, adapters, device="cuda"):
    """(seg_off, seg_adapter) int32 device tensors for requests of these row counts and adapters (-1: none)."""
    if len(lengths) != len(adapters):
        raise ValueError("one adapter per segment expected")
    off = [0]
    for n in lengths:
        if n < 0:
            raise ValueError("segment lengths are not negative")
        off.append(off[-1] + int(n))
    return (torch.tensor(off, dtype=torch.int32, device=device),
            torch.tensor(list(adapters), dtype=torch.int32, device=device))


class AdaptedLinear:
    """y = x . dequant(W)^T + s_a (drop(x) A_a^T) B_a^T for W [N, K] quantized once and a pool of adapters
    A [L, R, K], B [L, N, R] (ranks int32 [L], scales fp32 [L]; bf16 or fp16, the type of x)."""

    def __init__(self, W: torch.Tensor, bits: int, A, B, ranks, scales, group: int | None = None):
        self.N, self.K = W.shape
        self.bits, self.group = bits, group or bq.GROUP_OF_BITS[bits]
        bq._device("W", W)
        with torch.cuda.device_of(W):
            self.weights = bq.bq_quantize(W.contiguous(), self.bits, self.group, "interleaved")
        self.A, self.B, self.ranks, self.scales = A, B, ranks, scales

    def _pools(self, segs):
        return (self.A, self.B, self.ranks, self.scales, *segs)

    def _rows(self, name: str, v, cols: int):
        """v [rows, cols] with dense rows: the frozen layer's calls take their sizes and strides for granted."""
        if v.dim() != 2 or v.shape[1] != cols or v.dtype is not self.A.dtype:
            raise bq._bad(name, f"[rows, {cols}] {self.A.dtype}", v)
        if bq._device(name, v) != self.A.get_device():
            raise bq._bad(name, f"a tensor on {self.A.device}", v)
        return v.contiguous()

    def __call__(self, x: torch.Tensor, segs, out=None) -> torch.Tensor:
        """Serving: every row of x belongs to a segment (rows behind the last get the frozen layer alone)."""
        x = self._rows("x", x, self.K)
        if out is not None and (out.shape != (x.shape[0], self.N) or not out.is_contiguous() or
                                self._rows("out", out, self.N) is not out):
            raise bq._bad("out", f"contiguous [{x.shape[0]}, {self.N}]", out)
        with torch.cuda.device_of(x):
            y = bq.bq_linear(x, *self.weights, self.N, self.bits, self.group, out=out)
            return bq.bq_lora(x, *self._pools(segs), base=y, out=y)

    def forward(self, x: torch.Tensor, segs, p: float = 0.0, rng=None):
        """(y, saved) with dropout p on the adapters' input; saved goes to backward unchanged."""
        x = self._rows("x", x, self.K)
        with torch.cuda.device_of(x):
            y = bq.bq_linear(x, *self.weights, self.N, self.bits, self.group)
            # zero: rows behind the last segment have no t
            t = torch.zeros((x.shape[0], self.A.shape[1]), dtype=torch.float32, device=x.device)
            bq.bq_lora(x, *self._pools(segs), base=y, out=y, p=p, rng=rng, t=t)
        return y, (x, t, segs, p, None if rng is None else rng.clone())

    def backward(self, dy: torch.Tensor, saved):
        """(dx, dA, dB): the gradients of x (dy's type) and of the adapters (fp32)."""
        x, t, segs, p, rng = saved
        dy = self._rows("dy", dy, self.N)
        if dy.shape[0] != x.shape[0]:
            raise bq._bad("dy", f"[{x.shape[0]}, {self.N}]", dy)
        with torch.cuda.device_of(dy):
            dx = bq.bq_linear_grad_input(dy, *self.weights, self.K, self.bits, self.group)
            return bq.bq_lora_grad(dy, x, t, *self._pools(segs), base=dx, out=dx, p=p, rng=rng)
