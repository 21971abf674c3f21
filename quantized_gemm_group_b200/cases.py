"""Single-kernel cases for profiling (ncu) and timing: one shape, a few
launches, then a device-status check.

    python -m quantized_gemm_group_b200.cases gemv  M N K BITS    # decode linear, M <= 16
    python -m quantized_gemm_group_b200.cases gemm  M N K BITS    # prefill linear, M >= 64
    python -m quantized_gemm_group_b200.cases quant N K BITS      # quantizer, interleaved layout
    python -m quantized_gemm_group_b200.cases grad  M N K BITS    # input gradient dx = dy . dequant(W)
    python -m quantized_gemm_group_b200.cases lora  M N K R S     # low-rank adapters, S segments, one adapter each
    python -m quantized_gemm_group_b200.cases lora_grad M N K R S # their gradients
    python -m quantized_gemm_group_b200.cases dropout M K         # dropout of bf16 activations

Weights are synthetic fp16 N(0, 0.02) (N(0, 0.015) for the prefill case),
activations (and dy) bf16 N(0, 1); INT4 uses group 128, INT2 group 64.  Each case runs
its kernel 4 times (3 for the prefill case), so a profiler can skip the first
launches.
"""
from __future__ import annotations

import sys

import torch

from . import bq, synth


def main(argv):
    which = argv[0]
    if which in ("gemv", "gemm"):
        M, N, K, bits = (int(v) for v in argv[1:5])
        g = 128 if bits == 4 else 64
        W = synth.normal((N, K), 0.02 if which == "gemv" else 0.015, seed=1, dtype="f16", device="cuda")
        pk, sc, ze = bq.bq_quantize(W, bits, g, "interleaved")
        x = synth.activations(M, K, seed=2, device="cuda")
        y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        for _ in range(4 if which == "gemv" else 3):
            bq.bq_linear(x, pk, sc, ze, N, bits, g, out=y)
    elif which == "grad":
        M, N, K, bits = (int(v) for v in argv[1:5])
        g = 128 if bits == 4 else 64
        W = synth.normal((N, K), 0.02, seed=1, dtype="f16", device="cuda")
        pk, sc, ze = bq.bq_quantize(W, bits, g, "interleaved")
        dy = synth.activations(M, N, seed=2, device="cuda")
        dx = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
        for _ in range(4):
            bq.bq_linear_grad_input(dy, pk, sc, ze, K, bits, g, out=dx)
    elif which == "quant":
        N, K, bits = (int(v) for v in argv[1:4])
        g = 128 if bits == 4 else 64
        W = synth.normal((N, K), 0.02, seed=1, dtype="f16", device="cuda")
        out = bq.bq_quantize(W, bits, g, "interleaved")
        for _ in range(3):
            bq.bq_quantize(W, bits, g, "interleaved", out=out)
    elif which in ("lora", "lora_grad"):
        M, N, K, R, S = (int(v) for v in argv[1:6])
        x, dy = synth.activations(M, K, seed=2, device="cuda"), synth.activations(M, N, seed=3, device="cuda")
        ad = synth.adapters(S, R, K, N, seed=4, device="cuda")
        segs = (torch.linspace(0, M, S + 1, device="cuda").to(torch.int32),
                torch.arange(S, dtype=torch.int32, device="cuda"))
        y, dx = torch.empty_like(dy), torch.empty_like(x)
        t = torch.empty((M, R), dtype=torch.float32, device="cuda")
        bq.bq_lora(x, *ad, *segs, base=dy, out=y, t=t)
        for _ in range(3):
            if which == "lora":
                bq.bq_lora(x, *ad, *segs, base=dy, out=y)
            else:
                bq.bq_lora_grad(dy, x, t, *ad, *segs, base=x, out=dx)
    elif which == "dropout":
        M, K = (int(v) for v in argv[1:3])
        x = synth.activations(M, K, seed=2, device="cuda")
        rng = torch.tensor([7, 1], dtype=torch.int64, device="cuda")
        for _ in range(4):
            bq.bq_dropout(x, 0.05, rng)
    else:
        raise SystemExit(__doc__)
    torch.cuda.synchronize()
    status = bq.bq_device_status()
    if status != bq.BQ_OK:
        raise SystemExit(f"device status {bq.status_string(status)}")
    print("ok")


if __name__ == "__main__":
    main(sys.argv[1:])
