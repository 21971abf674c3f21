"""Host-side checks of the adapter and dropout entry points: argument validation without a device, the layout of the
argument structs, and the reference implementation's own pins.  No GPU needed."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

from quantized_gemm_group_b200 import bq, build

from . import adapter_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    build.build()
    return bq.lib()


def test_validation_cases_without_a_device(L):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "abi_adapter_cases.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]


@pytest.mark.parametrize("name,fmt", [("bq_lora_args", bq._LORA_ARGS), ("bq_lora_grad_args", bq._LORA_GRAD_ARGS)])
def test_argument_structs_match_the_header(name, fmt):
    """The binding's packed layout is the header's struct: pointers, int64, double, int32, in order and without gaps."""
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "bq.h")).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", src).group(1)
    kinds = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        kind = "Q" if "*" in decl else {"int64_t": "q", "double": "d", "int32_t": "i"}[decl.split()[0]]
        kinds += [kind] * len(decl.split(","))
    assert "".join(kinds) == re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), fmt.format[1:])
    native = {"Q": ctypes.c_void_p, "q": ctypes.c_int64, "d": ctypes.c_double, "i": ctypes.c_int32}

    class S(ctypes.Structure):
        _fields_ = [("f%d" % i, native[k]) for i, k in enumerate(kinds)]

    assert ctypes.sizeof(S) == fmt.size


def test_cpu_tensors_are_refused(L):
    x = torch.zeros((2, 8))
    with pytest.raises(ValueError):
        bq.bq_dropout(x, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        bq.bq_lora(x.half(), torch.zeros((1, 8, 8)).half(), torch.zeros((1, 8, 8)).half(), torch.zeros(1, dtype=torch.int32),
                   torch.zeros(1), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_generator_known_answers():
    """Known answers of Philox 4x32-10, published with the generator: counter and key all zero, all ones, and digits of pi."""
    def words(counter, key):
        u = np.uint64
        c, (k0, k1) = [u(v) for v in counter], key
        for _ in range(10):
            p0, p1 = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
            c = [(p1 >> u(32)) ^ c[1] ^ u(k0), p1 & u(0xFFFFFFFF), (p0 >> u(32)) ^ c[3] ^ u(k1), p0 & u(0xFFFFFFFF)]
            k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
        return [int(v) for v in c]

    assert words([0] * 4, (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 0xFFFFFFFF
    assert words([ones] * 4, (ones, ones)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert words([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
    # the reference's fields are these words' halves, eight columns a block
    got = ref.philox_fields(3, 20, 0x0000000500000007, 0x0000000B00000009)
    for row, blk in ((0, 0), (2, 1), (1, 2)):
        w = words([blk, row, 9, 11], (7, 5))
        want = [v for x in w for v in (x & 0xFFFF, x >> 16)]
        assert got[row, 8 * blk:8 * blk + 8].tolist() == want[:min(8, 20 - 8 * blk)]


def test_reference_gradients_against_differences():
    """The reference's gradients against central differences of its own forward pass, in 64 bits on the CPU."""
    g = torch.Generator().manual_seed(3)
    M, K, N, R = 9, 16, 24, 8
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, dy, A, B = rnd(M, K), rnd(M, N), rnd(2, R, K), rnd(2, N, R)
    tail = (torch.tensor([8, 5]), torch.tensor([0.5, 2.0]), torch.tensor([0, 4, 7, 9]), torch.tensor([1, -1, 0]))
    kw = dict(p=0.3, rng=torch.tensor([11, 2]))
    for v in (ref.HALF_STEP, ref.TINY):
        v.setdefault(torch.float64, 0.0)
    t = ref.lora(x, A, B, *tail, **kw)[2]
    dx, _, dA, _, dB, _ = ref.lora_grad(dy, x, t, A, B, *tail, **kw)
    for i, got in ((0, dx), (1, dA), (2, dB)):
        args = [x, A, B]
        d = rnd(*args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + d, args[i] - d
        q = float((dy * (ref.lora(*up, *tail, **kw)[0] - ref.lora(*down, *tail, **kw)[0])).sum()) / 2
        assert abs(float((got * d).sum()) - q) <= 1e-9 * max(1.0, abs(q))


def test_adapted_linear_refuses_other_shapes():
    """The frozen layer's calls read as many packed bytes as the rows are wide: another width is refused before them."""
    from quantized_gemm_group_b200 import adapters
    ly = object.__new__(adapters.AdaptedLinear)
    ly.N, ly.K, ly.bits, ly.group, ly.weights = 64, 128, 4, 128, (None, None, None)
    ly.A, ly.B = torch.zeros((1, 8, 128)).half(), torch.zeros((1, 64, 8)).half()
    ly.ranks, ly.scales = torch.zeros(1, dtype=torch.int32), torch.zeros(1)
    segs = (torch.tensor([0, 2], dtype=torch.int32), torch.tensor([0], dtype=torch.int32))
    for x in (torch.zeros((2, 256)).half(), torch.zeros((2, 64)).half(), torch.zeros((2, 128)), torch.zeros((1, 2, 128)).half(),
              torch.zeros((2, 128)).half()):            # wider, narrower, another type, three dimensions, not on a GPU
        with pytest.raises(ValueError):
            ly(x, segs)
        with pytest.raises(ValueError):
            ly.forward(x, segs)
    saved = (torch.zeros((2, 128)).half(), torch.zeros((2, 8)), segs, 0.0, None)
    for dy in (torch.zeros((2, 128)).half(), torch.zeros((2, 64))):
        with pytest.raises(ValueError):
            ly.backward(dy, saved)
    with pytest.raises(ValueError):
        adapters.AdaptedLinear(torch.zeros((64, 128)).half(), 4, ly.A, ly.B, ly.ranks, ly.scales)
