"""bq_lora and bq_lora_grad against a plain implementation in 64 bits, element by element within bounds derived from
the kernels' arithmetic (adapter_ref)."""
from __future__ import annotations

import random

import pytest
import torch

from quantized_gemm_group_b200 import bq, synth

from . import adapter_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


class Case:
    """Inputs for one batch.  `lens`: the segments' rows, `ads` their adapters, `tail` rows behind the last segment.
    What a call must not use holds NaN: pools behind their ranks, and rows of x, dy and t without an adapter."""

    def __init__(self, K, N, R, ranks, lens, ads, tail=0, dtype=torch.bfloat16, p=0.0, pad=0, seed=0, scale=1.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + 1000 * K + N + R)
        L, M = len(ranks), sum(lens) + tail

        def rows(n, cols, std):
            w = (torch.randn((n, cols + 2 * pad), generator=g, device=DEV) * std).to(dtype)
            return w[:, pad:pad + cols]

        self.M, self.K, self.N, self.R, self.L, self.p, self.dtype = M, K, N, R, L, p, dtype
        self.x, self.dy, self.base, self.dbase = rows(M, K, 1.0), rows(M, N, 0.5), rows(M, N, 1.0), rows(M, K, 0.5)
        self.A = (torch.randn((L, R, K), generator=g, device=DEV) * max(K, 1) ** -0.5).to(dtype)
        self.B = (torch.randn((L, N, R), generator=g, device=DEV) * 0.1).to(dtype)
        for a, r in enumerate(ranks):
            self.A[a, r:] = NAN
            self.B[a, :, r:] = NAN
        self.ranks = torch.tensor(ranks, dtype=torch.int32, device=DEV)
        self.scales = torch.tensor([scale * (1.5 - a) or 0.75 for a in range(L)], dtype=torch.float32, device=DEV)
        off = [0]
        for n in lens:
            off.append(off[-1] + n)
        self.seg_off = torch.tensor(off, dtype=torch.int32, device=DEV)
        self.seg_adapter = torch.tensor(ads, dtype=torch.int32, device=DEV)
        self.rows = off[-1]
        for m0, m1, a in ref.segments(self.seg_off, self.seg_adapter):
            if a < 0:
                self.x[m0:m1] = NAN
                self.dy[m0:m1] = NAN
        self.x[self.rows:] = NAN
        self.dy[self.rows:] = NAN
        self.rng = torch.tensor([seed + 3, 5], dtype=torch.int64, device=DEV)
        self.pools = (self.A, self.B, self.ranks, self.scales, self.seg_off, self.seg_adapter)

    def forward(self, base=True, **kw):
        return bq.bq_lora(self.x, *self.pools, base=self.base if base else None, p=self.p, rng=self.rng, **kw)

    def grad(self, t, base=True, **kw):
        return bq.bq_lora_grad(self.dy, self.x, t, *self.pools, base=self.dbase if base else None, p=self.p, rng=self.rng,
                               **kw)

    def ref_forward(self, base=True):
        return ref.lora(self.x, *self.pools, base=self.base if base else None, p=self.p, rng=self.rng)

    def ref_grad(self, t, base=True):
        return ref.lora_grad(self.dy, self.x, t, *self.pools, base=self.dbase if base else None, p=self.p, rng=self.rng)

    def check(self, base=True):
        """Forward and gradients; what lies behind the last segment keeps its bits."""
        n = self.rows
        t = torch.full((self.M, self.R), 9.0, device=DEV)
        out = torch.full((self.M, self.N), 7.0, device=DEV).to(self.dtype)
        y = self.forward(base, out=out, t=t)
        w, b, wt, bt = self.ref_forward(base)
        ref.assert_within("t", t[:n], wt[:n], bt[:n])
        ref.assert_within("y", y[:n], w[:n], b[:n])
        assert bool((y[n:] == 7).all()) and bool((t[n:] == 9).all())
        no_t = self.forward(base)
        assert torch.equal(no_t[:n], y[:n])
        for m0, m1, a in ref.segments(self.seg_off, self.seg_adapter):
            if a < 0:
                t[m0:m1] = NAN
        t[n:] = NAN
        for a, r in enumerate(self.ranks.tolist()):  # behind the rank t may hold anything as well
            for m0, m1, b_ in ref.segments(self.seg_off, self.seg_adapter):
                if a == b_:
                    t[m0:m1, r:] = NAN
        out = torch.full((self.M, self.K), 7.0, device=DEV).to(self.dtype)
        dA, dB = torch.full(self.A.shape, 3.0, device=DEV), torch.full(self.B.shape, 3.0, device=DEV)
        dx, gA, gB = self.grad(t, base, out=out, dA=dA, dB=dB)
        wx, bx, wA, bA, wB, bB = self.ref_grad(t, base)
        ref.assert_within("dx", dx[:n], wx[:n], bx[:n])
        assert bool((dx[n:] == 7).all())
        ref.assert_within("dA", gA, wA, bA)
        ref.assert_within("dB", gB, wB, bB)
        assert bq.bq_device_status() == bq.BQ_OK
        return y, dx, dA, dB


DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# lengths around the 16-row and 128-row tiles and around the choice between the two kernels (24 rows a segment)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 24, 25, 31, 33, 64, 65, 127, 128, 129, 257])
def test_one_segment(M, dt):
    Case(264, 200, 16, [16], [M], [0], dtype=DT[dt]).check()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("R,ranks", [(8, [8, 1]), (16, [16, 5]), (24, [17, 24]), (40, [33, 40]), (64, [64, 63]),
                                     (72, [72, 65]), (128, [128, 81]), (128, [16, 128])])
@pytest.mark.parametrize("lens", [[3, 1, 7], [70, 150, 40]])
def test_ranks(R, ranks, lens, dt):
    Case(328, 392, R, ranks, lens, [0, 1, 0], dtype=DT[dt]).check()


@pytest.mark.parametrize("K,N", [(8, 8), (8, 4104), (4104, 8), (64, 64), (72, 56), (1000, 1032), (2048, 520), (520, 4096)])
@pytest.mark.parametrize("lens", [[5, 9], [140, 60]])
def test_sizes(K, N, lens):
    Case(K, N, 32, [32, 20], lens, [1, 0]).check()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("p", [0.05, 0.6])
@pytest.mark.parametrize("lens,ads", [([4, 1, 11], [0, -1, 1]), ([200, 33, 90], [1, -1, 0])])
def test_dropout(p, lens, ads, dt):
    Case(712, 600, 48, [48, 30], lens, ads, tail=3, dtype=DT[dt], p=p).check()


@pytest.mark.parametrize("lens,ads", [
    ([0, 5, 0, 0, 3, 0], [1, 0, 1, -1, 1, 0]),          # empty segments everywhere
    ([0, 0, 0], [0, 1, -1]),                            # nothing but empty segments
    ([300, 0, 200], [0, 1, 0]),                         # one adapter in several segments, another unused
    ([60, 50, 70, 40, 30], [1, -1, 1, 1, -1]),          # the same adapter three times, requests without one
    ([40] * 40, [i % 2 for i in range(40)]),            # more segments than a warp looks at once
    ([1] * 70, [(i * 5) % 3 - 1 for i in range(70)]),   # one token each
    ([200], [-1]),                                      # no adapter at all
])
@pytest.mark.parametrize("tail", [0, 5])
def test_segments(lens, ads, tail):
    Case(200, 264, 24, [24, 9], lens, ads, tail=tail, p=0.1).check()


@pytest.mark.parametrize("lens", [[6, 10], [100, 156]])
def test_rank_zero_adapters(lens):
    Case(136, 264, 16, [0, 16], lens, [0, 1]).check()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("lens", [[5, 9], [130, 77]])
def test_strided_rows_without_base(lens, dt):
    c = Case(264, 520, 16, [16, 12], lens, [0, 1], tail=2, dtype=DT[dt], pad=24)
    c.check()
    c.check(base=False)


@pytest.mark.parametrize("lens", [[5, 9], [130, 77]])
def test_in_place(lens):
    c = Case(264, 520, 40, [40, 12], lens, [0, -1], tail=4)
    y, dx, _, _ = c.check()
    t = torch.zeros((c.M, c.R), device=DEV)
    z = c.base.clone()
    assert bq.bq_lora(c.x, *c.pools, base=z, out=z, t=t) is z
    assert torch.equal(z[:c.rows], y[:c.rows]) and torch.equal(z[c.rows:], c.base[c.rows:])
    z = c.dbase.clone()
    got, _, _ = bq.bq_lora_grad(c.dy, c.x, t, *c.pools, base=z, out=z)
    assert got is z and torch.equal(z[:c.rows], dx[:c.rows]) and torch.equal(z[c.rows:], c.dbase[c.rows:])


@pytest.mark.parametrize("lens", [[5, 9], [130, 77]])
def test_parts_of_the_gradient(lens):
    c = Case(264, 520, 40, [40, 12], lens, [0, 1], p=0.1)
    t = torch.zeros((c.M, c.R), device=DEV)
    c.forward(t=t)
    dx, dA, dB = c.grad(t)
    only, none_a, none_b = c.grad(t, need_weights=False)
    assert none_a is None and none_b is None and torch.equal(only, dx)
    none_x, a2, b2 = c.grad(t, need_dx=False)
    assert none_x is None and torch.equal(a2, dA) and torch.equal(b2, dB)
    # x and t are not looked at when the weights' gradients are not wanted
    only2, _, _ = bq.bq_lora_grad(c.dy, None, None, *c.pools, base=c.dbase, p=c.p, rng=c.rng, need_weights=False)
    assert torch.equal(only2, dx)


@pytest.mark.parametrize("lens", [[4, 3, 9], [300, 129, 65]])
def test_fp16_far_from_one(lens):
    """t and dt outside fp16's range or among its subnormals: the parts carry their own power of two."""
    for scale in (2.0 ** 14, 2.0 ** -13):
        c = Case(512, 256, 32, [32, 17], lens, [0, 1, 0], dtype=torch.float16)
        c.A.mul_(2.0 ** 5 if scale > 1 else 2.0 ** -6)
        c.x.mul_(2.0 ** 9 if scale > 1 else 2.0 ** -3)      # t up to about 2^17, or about 2^-9 and below
        c.B.mul_(2.0 ** -11 if scale > 1 else 1.0)
        c.check()


@pytest.mark.parametrize("lens", [[4, 3], [150, 65]])
def test_infinities_and_nan_stay_in_their_rows(lens):
    c = Case(264, 200, 16, [16, 16], lens, [0, 1])
    y0 = c.forward()
    x1 = c.x.clone()
    x1[1, 7], x1[2, 8] = float("inf"), NAN
    y1 = bq.bq_lora(x1, *c.pools, base=c.base)
    assert not bool(torch.isfinite(y1[1]).any()) and bool(torch.isnan(y1[2]).all())
    keep = [m for m in range(c.M) if m not in (1, 2)]
    assert torch.equal(y1[keep], y0[keep])
    # dropped places may hold anything
    c = Case(264, 200, 16, [16, 16], lens, [0, 1], p=0.5)
    y0 = c.forward()
    f = ref.keep_factor(c.M, c.K, c.p, c.rng)
    c.x[f == 0] = NAN
    assert torch.equal(c.forward(), y0)
    t = torch.zeros((c.M, c.R), device=DEV)
    c.forward(t=t)
    assert all(bool(torch.isfinite(v).all()) for v in c.grad(t))


@pytest.mark.parametrize("lens", [[3] * 12, [130, 200, 77]])
def test_same_bits_every_time(lens):
    c = Case(1032, 776, 64, [64, 40], lens, [i % 2 for i in range(len(lens))], p=0.1)
    first = c.check()
    for _ in range(3):
        assert all(torch.equal(a[:c.rows] if a.dim() == 2 else a, b[:c.rows] if b.dim() == 2 else b)
                   for a, b in zip(first, c.check()))


@pytest.mark.parametrize("lens", [[6, 11], [90, 140]])
def test_against_differences(lens):
    """<gradient, direction> against the central difference of the 64-bit loss <dy, y> along a random direction (y is
    bilinear in the pools and linear in x, so the central difference of each argument alone is exact)."""
    c = Case(136, 104, 16, [16, 9], lens, [0, 1], p=0.2)
    t = torch.zeros((c.M, c.R), device=DEV)
    c.forward(base=False, t=t)
    dx, dA, dB = c.grad(t, base=False)
    wx, bx, wA, bA, wB, bB = c.ref_grad(t, base=False)
    live = torch.arange(c.R, device=DEV)[None, :] < c.ranks[:, None]
    A, B = torch.where(live[:, :, None], c.A.double(), 0.0), torch.where(live[:, None, :], c.B.double(), 0.0)
    x, dy = c.x.double(), c.dy.double()
    f = ref.keep_factor(c.M, c.K, c.p, c.rng)

    def loss(x, A, B):
        total = 0.0
        for m0, m1, a in ref.segments(c.seg_off, c.seg_adapter):
            total += (dy[m0:m1] * (float(c.scales[a]) * ((x[m0:m1] * f[m0:m1]) @ A[a].t()) @ B[a].t())).sum()
        return float(total)

    for got, bound, at in ((dx, bx, 0), (dA, bA, 1), (dB, bB, 2)):
        args = [x, A, B]
        d = torch.randn_like(args[at])
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + d, args[at] - d
        quotient = (loss(*up) - loss(*down)) / 2
        if at:
            d = torch.where(live[:, :, None] if at == 1 else live[:, None, :], d, 0.0)
        inner = float((got.double() * d).sum())
        # dB is taken from the fp32 t: its own bound, plus what t's rounding (SUM(K)) does
        slack = float((bound * d.abs()).sum()) * (1 if at != 2 else 4) + (2.0 ** -12 * abs(quotient) if at == 2 else 0)
        assert abs(inner - quotient) <= slack + 1e-9 * abs(quotient)


def test_many_shapes():
    """Random batches of both kernels' ranges."""
    rnd = random.Random(12)
    for i in range(40):
        L = rnd.randint(1, 5)
        R = 8 * rnd.randint(1, 16)
        S = rnd.randint(1, 9)
        big = rnd.random() < 0.5
        lens = [rnd.choice((0, rnd.randint(1, 300 if big else 20))) for _ in range(S)]
        Case(8 * rnd.randint(1, 90), 8 * rnd.randint(1, 90), R, [rnd.randint(0, R) for _ in range(L)], lens,
             [rnd.randint(-1, L - 1) for _ in range(S)], tail=rnd.randint(0, 6), dtype=DT[rnd.choice(("bf16", "f16"))],
             p=rnd.choice((0.0, 0.2)), pad=rnd.choice((0, 8)), seed=i).check(base=rnd.random() < 0.7)


def test_adapters_of_a_fused_projection():
    """Query and value slices of one fused output get their own adapters in place; the key slice stays as it was."""
    M, K = 70, 256
    fused = torch.randn((M, 256 + 64 + 64), device=DEV).to(torch.bfloat16)
    before = fused.clone()
    x = torch.randn((M, K), device=DEV).to(torch.bfloat16)
    seg = (torch.tensor([0, 30, M], dtype=torch.int32, device=DEV), torch.tensor([1, 0], dtype=torch.int32, device=DEV))
    for lo, hi, seed in ((0, 256, 1), (320, 384, 2)):
        A, B, ranks, scales = synth.adapters(2, 16, K, hi - lo, seed, device=DEV)
        y = fused[:, lo:hi]
        bq.bq_lora(x, A, B, ranks, scales, *seg, base=y, out=y)
        w, b, _, _ = ref.lora(x, A, B, ranks, scales, *seg, base=before[:, lo:hi])
        ref.assert_within("y", y, w, b)
    assert torch.equal(fused[:, 256:320], before[:, 256:320])


# ---------------------------------------------------------------------------
# with the weight-only linear layer, as a model runs them
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("overlap", [0, 1, 2])
@pytest.mark.parametrize("lens", [[1, 1, 1, 1, 1], [90, 60]])
def test_beside_the_linear_layer(overlap, lens):
    """Frozen low-bit projections with adapters, forward and back, back to back on one stream: each call's result
    against the 64-bit adapter on the linear layer's own output, under every launch mode."""
    K, N, M = 512, 256, sum(lens)
    c = Case(K, N, 16, [16, 11], lens, [i % 2 for i in range(len(lens))], p=0.1)
    W = synth.normal((N, K), 0.02, seed=1, dtype="f16", device=DEV)
    pk, sc, ze = bq.bq_quantize(W, 4, 128)
    y0 = bq.bq_linear(c.x, pk, sc, ze, N, 4, 128)
    dx0 = bq.bq_linear_grad_input(c.dy, pk, sc, ze, K, 4, 128)
    t = torch.zeros((M, 16), device=DEV)
    torch.cuda.synchronize()
    old = bq.bq_get_option(bq.BQ_OPT_LINEAR_OVERLAP)
    bq.bq_set_option(bq.BQ_OPT_LINEAR_OVERLAP, overlap)
    try:
        got = []
        for _ in range(5):
            y = bq.bq_linear(c.x, pk, sc, ze, N, 4, 128)
            bq.bq_lora(c.x, *c.pools, base=y, out=y, p=c.p, rng=c.rng, t=t)
            dx = bq.bq_linear_grad_input(c.dy, pk, sc, ze, K, 4, 128)
            _, dA, dB = bq.bq_lora_grad(c.dy, c.x, t, *c.pools, base=dx, out=dx, p=c.p, rng=c.rng)
            got.append((y, dx, dA, dB))
        torch.cuda.synchronize()
    finally:
        bq.bq_set_option(bq.BQ_OPT_LINEAR_OVERLAP, old)
    w, b, _, _ = ref.lora(c.x, *c.pools, base=y0, p=c.p, rng=c.rng)
    wx, bx, wA, bA, wB, bB = ref.lora_grad(c.dy, c.x, t, *c.pools, base=dx0, p=c.p, rng=c.rng)
    for y, dx, dA, dB in got:
        ref.assert_within("y", y, w, b)
        ref.assert_within("dx", dx, wx, bx)
        ref.assert_within("dA", dA, wA, bA)
        ref.assert_within("dB", dB, wB, bB)
    assert bq.bq_device_status() == bq.BQ_OK


# ---------------------------------------------------------------------------
# graphs, streams, addresses
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens,other", [([3, 9, 4], [9, 0, 7]), ([200, 60, 40], [0, 290, 5])])
def test_graph_replays_with_other_segments_and_masks(lens, other):
    """A captured step reads segments, ranks, scales and the generator when it runs."""
    c = Case(264, 200, 24, [24, 10], lens, [0, 1, -1], p=0.2)
    c.x.copy_(torch.randn_like(c.x.float()))
    c.dy.copy_(torch.randn_like(c.dy.float()))
    t, y, dx = torch.zeros((c.M, c.R), device=DEV), torch.zeros_like(c.base), torch.zeros_like(c.dbase)
    dA, dB = torch.zeros(c.A.shape, device=DEV), torch.zeros(c.B.shape, device=DEV)
    ws = torch.zeros((c.M, c.R), device=DEV)

    def step():
        c.forward(out=y, t=t)
        c.grad(t, out=dx, dA=dA, dB=dB, workspace=ws)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g2 = torch.cuda.CUDAGraph()                        # a second graph of the same call allocates its own workspace
    with torch.cuda.graph(g2):
        dx2, dA2, dB2 = c.grad(t)
    for n, ads in ((lens, [0, 1, -1]), (other, [1, -1, 0])):
        off = [0, n[0], n[0] + n[1], n[0] + n[1] + n[2]]
        c.seg_off.copy_(torch.tensor(off, dtype=torch.int32))
        c.seg_adapter.copy_(torch.tensor(ads, dtype=torch.int32))
        c.rng[1] += 1
        g.replay()
        g2.replay()
        rows = off[-1]
        w, b, wt, bt = c.ref_forward()
        ref.assert_within("y", y[:rows], w[:rows], b[:rows])
        wx, bx, wA, bA, wB, bB = c.ref_grad(t)
        ref.assert_within("dx", dx[:rows], wx[:rows], bx[:rows])
        ref.assert_within("dA", dA, wA, bA)
        ref.assert_within("dB", dB, wB, bB)
        assert torch.equal(dx2[:rows], dx[:rows]) and torch.equal(dA2, dA) and torch.equal(dB2, dB)
    assert bq.bq_device_status() == bq.BQ_OK


@pytest.mark.parametrize("lens", [[3, 9], [200, 60]])
def test_two_streams_at_once(lens):
    cs = [Case(520, 264, 64, [64, 33], lens, [0, 1], seed=s) for s in (1, 2)]
    want = [c.check() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for c, s in zip(cs, streams):
            t = torch.zeros((c.M, c.R), device=DEV)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                y = c.forward(t=t)
            got.append((c, y) + c.grad(t, stream=s))
            t.record_stream(s)
    torch.cuda.synchronize()
    for c, y, dx, dA, dB in got:
        for a, b in zip((y, dx, dA, dB), want[cs.index(c)]):
            assert torch.equal(a, b)


def test_results_belong_to_the_stream():
    """A result allocated for another stream is not memory that the current stream's kernels may still use."""
    c = Case(520, 264, 64, [64, 33], [3, 9], [0, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for call, cols in ((lambda: c.forward(stream=s), c.N), (lambda: bq.bq_dropout(c.x, 0.5, c.rng, stream=s), c.K)):
        old = torch.empty((c.M, cols), dtype=c.dtype, device=DEV)
        at = old.data_ptr()
        del old
        out = call()
        assert out.data_ptr() != at
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Rows so far apart that element offsets pass 2^31, with both kernels."""
    for lens in ([2, 3], [120, 50]):
        M = sum(lens)
        stride = ((1 << 31) // (M - 2) + 4096) // 8 * 8
        flat = torch.zeros(M * stride, dtype=torch.bfloat16, device=DEV)
        c = Case(64, 72, 16, [16, 16], lens, [0, 1])
        view = lambda cols, at, v: torch.as_strided(flat, (M, cols), (stride, 1), at).copy_(v)  # noqa: E731
        c.x, c.base, c.dy, c.dbase = view(64, 0, c.x), view(72, 64, c.base), view(72, 136, c.dy), view(64, 208, c.dbase)
        out = torch.as_strided(flat, (M, 72), (stride, 1), 272)
        t = torch.zeros((M, 16), device=DEV)
        c.forward(out=out, t=t)
        w, b, _, _ = c.ref_forward()
        ref.assert_within("y", out, w, b)
        dx, dA, dB = c.grad(t)
        wx, bx, wA, bA, wB, bB = c.ref_grad(t)
        ref.assert_within("dx", dx, wx, bx)
        ref.assert_within("dA", dA, wA, bA)
        ref.assert_within("dB", dB, wB, bB)


def test_pool_past_32_bits():
    """The last adapter of a pool of more than 2^31 elements."""
    L, R, K, N = 1100, 128, 16384, 8
    A = torch.zeros((L, R, K), dtype=torch.bfloat16, device=DEV)
    A[-1] = torch.randn((R, K), device=DEV) / 128
    B = torch.randn((L, N, R), device=DEV).to(torch.bfloat16)
    ranks = torch.full((L,), R, dtype=torch.int32, device=DEV)
    scales = torch.ones(L, device=DEV)
    for M in (3, 130):
        x = torch.randn((M, K), device=DEV).to(torch.bfloat16)
        seg = (torch.tensor([0, M], dtype=torch.int32, device=DEV), torch.tensor([L - 1], dtype=torch.int32, device=DEV))
        y = bq.bq_lora(x, A, B, ranks, scales, *seg)
        w, b, _, _ = ref.lora(x, A, B, ranks, scales, *seg)
        ref.assert_within("y", y, w, b)


# ---------------------------------------------------------------------------
# refusals that only the device can make, empty calls
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens", [[4, 6, 5], [150, 60, 90]])
def test_bad_segments_are_recorded_and_skipped(lens):
    c = Case(136, 200, 16, [16, 8], lens, [0, 1, 0])
    good = c.forward()
    off = c.seg_off.tolist()
    bad = [(dict(seg_adapter=[0, 2, 0]), 1), (dict(seg_adapter=[0, -2, 0]), 1),
           (dict(seg_off=[0, off[1], off[2], c.M + 1]), 2), (dict(seg_off=[-1, off[1], off[2], off[3]]), 0),
           (dict(ranks=[16, 17]), 1), (dict(ranks=[16, -1]), 1)]
    for what, hit in bad:
        v = {"seg_off": c.seg_off, "seg_adapter": c.seg_adapter, "ranks": c.ranks}
        for k, l in what.items():
            v[k] = torch.tensor(l, dtype=torch.int32, device=DEV)
        y = c.base.clone()
        bq.bq_lora(c.x, c.A, c.B, v["ranks"], c.scales, v["seg_off"], v["seg_adapter"], base=y, out=y)
        assert bq.bq_device_status() == bq.BQ_ERR_UNSUPPORTED
        for i in range(3):
            rows = slice(off[i], off[i + 1])
            assert torch.equal(y[rows], c.base[rows] if i == hit else good[rows]), (what, i)
        assert bq.bq_device_status() == bq.BQ_OK
    # descending offsets: the segment that descends is skipped
    y = c.base.clone()
    descending = torch.tensor([off[1], 0, off[2], off[2]], dtype=torch.int32, device=DEV)
    bq.bq_lora(c.x, *c.pools[:4], descending, torch.tensor([0, 1, 0], dtype=torch.int32, device=DEV), base=y, out=y)
    assert bq.bq_device_status() == bq.BQ_ERR_UNSUPPORTED


def test_empty_calls():
    c = Case(64, 72, 16, [16], [4], [0])
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = c.base.clone()
    bq.bq_lora(c.x, c.A, c.B, c.ranks, c.scales, zero, none, base=y, out=y)          # no segments
    assert torch.equal(y, c.base)
    t = torch.zeros((4, 16), device=DEV)
    dx, dA, dB = bq.bq_lora_grad(c.dy, c.x, t, c.A, c.B, c.ranks, c.scales, zero, none)
    assert bool((dA == 0).all()) and bool((dB == 0).all())
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    dx, dA, dB = bq.bq_lora_grad(e(0, 72), e(0, 64), torch.empty((0, 16), device=DEV), *c.pools)   # no rows
    assert dx.shape == (0, 64) and bool((dA == 0).all()) and bool((dB == 0).all())
    bq.bq_device_status()                                                            # offsets leave [0, 0]
    # an empty contraction: y = base, t = 0
    for M in (4, 60):
        seg = (torch.tensor([0, M], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV))
        base = torch.randn((M, 72), device=DEV).to(torch.bfloat16)
        t = torch.full((M, 16), 3.0, device=DEV)
        y = bq.bq_lora(e(M, 0), e(1, 16, 0), c.B, c.ranks, c.scales, *seg, base=base, t=t)
        assert torch.equal(y, base) and bool((t == 0).all())
    assert bq.bq_device_status() == bq.BQ_OK


def test_refused_tensors():
    c = Case(64, 72, 16, [16], [4], [0])
    ok = dict(zip(("A", "B", "ranks", "scales", "seg_off", "seg_adapter"), c.pools))
    for name, v in (("A", c.A.half()), ("A", c.A[:, :, ::2]), ("B", c.B[:, :, :8]), ("ranks", c.ranks.long()),
                    ("scales", c.scales.double()), ("seg_off", c.seg_off.long()), ("seg_off", c.seg_off[:1]),
                    ("seg_adapter", c.seg_adapter.cpu())):
        with pytest.raises(ValueError):
            bq.bq_lora(c.x, *{**ok, name: v}.values())
    for kw in (dict(base=c.base.float()), dict(out=c.base[:2]), dict(t=torch.zeros((4, 8), device=DEV)),
               dict(t=torch.zeros((4, 16), dtype=torch.float16, device=DEV)), dict(p=0.5, rng=torch.zeros(2, device=DEV))):
        with pytest.raises(ValueError):
            bq.bq_lora(c.x, *c.pools, **kw)
    with pytest.raises(ValueError):
        bq.bq_lora(c.x.t().contiguous().t(), *c.pools)                               # columns not contiguous
    for x, kw in ((c.x, dict(p=1.0, rng=c.rng)), (c.x, dict(p=-0.1, rng=c.rng)), (c.x, dict(p=0.5))):
        with pytest.raises(bq.BQError):
            bq.bq_lora(x, *c.pools, **kw)
    wide = torch.zeros((4, 80), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(bq.BQError):
        bq.bq_lora(wide[:, 4:68], *c.pools)                                          # rows not 16-byte aligned
    odd = torch.zeros((4, 68), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(bq.BQError):
        bq.bq_lora(odd[:, :64], *c.pools)                                            # a row stride of 68
    assert bq.bq_device_status() == bq.BQ_OK
