"""bq_lora and bq_lora_grad in every geometry that the host chooses: clusters of every size with one CTA an SM and with
two, more tiles than the GPU holds at once, rings of shared memory that go round several times, in both directions and
types, against the 64-bit implementation."""
from __future__ import annotations

import random

import pytest

from .test_lora_gpu import DT, Case


def ragged(total, parts, seed, empty=0.1):
    """`parts` lengths that add up to `total`, some of them 0."""
    rnd = random.Random(seed)
    w = [0.0 if rnd.random() < empty else rnd.random() + 0.05 for _ in range(parts)]
    w[-1] = max(w[-1], 0.5)
    cuts, at = [0], 0.0
    for v in w:
        at += v
        cuts.append(round(total * at / sum(w)))
    return [b - a for a, b in zip(cuts, cuts[1:])]


pytestmark = pytest.mark.gpu


# Tiles that the host counts for (rows / 128 + segments).  Ranks to 64 take clusters of 8, 6, 5, 4, 3, 2 with one CTA an SM up
# to 15, 22, 26, 33, 45, 74 tiles, then of 3, 2, 1 with two CTAs an SM up to 93, 148 and above; 296 fit at once.  Ranks
# above 64 take clusters of 2 and 1 where those go over to two CTAs an SM.
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("R", [64, 128])
@pytest.mark.parametrize("tiles", [12, 20, 25, 30, 40, 60, 80, 120, 200, 320])
def test_clusters(tiles, R, dt):
    S = 2 * tiles // 3
    M = (tiles - S) * 128
    lens = ragged(M, S, tiles)
    assert M > 24 * S and len(lens) == S and sum(lens) == M
    ranks = [R, R - 5, R // 2 + 1, 3]
    p = 0.1 if tiles in (25, 60, 80, 200) else 0.0
    Case(2056, 1032, R, ranks, lens, [i % 5 - 1 for i in range(S)], dtype=DT[dt], p=p, seed=tiles).check()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("lens,K,N,R", [
    ([5000, 1037], 264, 200, 64),        # clusters of 8, 12 tiles of 64 rows a CTA
    ([5000, 1037], 264, 200, 128),
    ([300, 0, 411], 8200, 11008, 64),    # single CTAs, 12 tiles each
    ([300, 0, 411], 4104, 5504, 128),
])
def test_weight_gradients_of_many_tiles(lens, K, N, R, p, dt):
    Case(K, N, R, [R, 7], lens, [0] * len(lens), dtype=DT[dt], p=p, tail=2).check()


@pytest.mark.parametrize("R", [16, 64, 128])
@pytest.mark.parametrize("S,rows", [(20, 3), (100, 5), (200, 9), (330, 2)])
def test_short_segments_in_clusters_of_every_size(S, rows, R):
    """Tiles of 16 rows: clusters of 8, 2 and 1 and more of them than the GPU holds; up to 33 steps down a CTA."""
    lens = ragged(S * rows, S, S)
    Case(8456, 1032, R, [R, R // 2 + 1, 1], lens, [i % 4 - 1 for i in range(S)], p=0.1 if S == 100 else 0.0, tail=1).check()
