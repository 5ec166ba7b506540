"""CPU model of the MXFP4 product's tile arithmetic (csrc/mxfp4_product.cuh) and of the packed weights' layout
(csrc/mxfp4.cuh): every row x weight row tile once, every offset inside its tile once."""
import random
import re
import os

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_routed_sqrt_b200", "csrc")


def widths():
    """The row tiles' widths, read from the host code."""
    src = open(os.path.join(CSRC, "operators.cu")).read()
    found = sorted({int(m) for m in re.findall(r"MxCfg<(\d+),", src)})
    assert found
    return found


def walk(S, lo, hi, E, MT, NT, index, stride):
    """The tiles (expert, weight row tile, first row, rows) of one CTA: MxTiles."""
    tiles, t, e, end, base = S[E] * MT, index, -1, 0, 0
    out = []
    while t < tiles:
        if t >= end:
            left = e + 1
            step = (E - left + 31) // 32
            hits = [left + lane * step < E and S[min(left + lane * step, E)] * MT <= t for lane in range(32)]
            assert hits[0] and hits == sorted(hits, reverse=True)
            left += (sum(hits) - 1) * step
            hits = [lane < step and left + lane < E and S[min(left + lane, E)] * MT <= t for lane in range(32)]
            assert hits[0]
            e = left + sum(hits) - 1
            base, nt = S[e] * MT, S[e + 1] - S[e]
            end = base + nt * MT
            rows = hi[e] - lo[e]
            per = min(NT, ((rows + nt - 1) // nt + 15) & ~15)
        local = t - base
        m = local // nt
        row = lo[e] + (local - m * nt) * per
        out.append((e, m, row, min(per, hi[e] - row)))
        t += stride
    return out


@pytest.mark.parametrize("NT", widths())
@pytest.mark.parametrize("seed", range(12))
def test_every_row_meets_every_weight_tile_once(NT, seed):
    rng = random.Random(100 * NT + seed)
    E = rng.choice([1, 2, 7, 31, 32, 33, 64, 200, 512])
    counts = [rng.choice([0, 0, 1, 5, 16, 17, NT - 1, NT, NT + 1, 3 * NT + 5, rng.randint(0, 900)]) if rng.random() < 0.6 else 0
              for _ in range(E)]
    MT = rng.randint(1, 9)
    lo, hi, S = [], [], [0]
    for c in counts:
        lo.append(hi[-1] if hi else 0)
        hi.append(lo[-1] + c)
        S.append(S[-1] + (c + NT - 1) // NT)
    stride = rng.choice([1, 3, 148])
    seen = {}
    for cta in range(stride):
        last = -1
        for e, m, row, n in walk(S, lo, hi, E, MT, NT, cta, stride):
            assert 1 <= n <= NT and 0 <= m < MT and lo[e] <= row and row + n <= hi[e] and e >= last
            last = e
            for r in range(row, row + n):
                assert (r, m) not in seen
                seen[r, m] = cta
    assert len(seen) == hi[-1] * MT


def test_packed_tile_is_a_bijection():
    code = {r * 128 + ((c ^ (r & 7)) << 4) for r in range(128) for c in range(8)}
    assert code == set(range(0, 16384, 16))
    scale = {16384 + (b >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3) for r in range(128) for b in range(8)}
    assert scale == set(range(16384, 17408))


def test_scale_warps_never_skip_a_phase():
    """A scale warp waits on every other pair of input tiles; a barrier's parity tells two phases apart, so the
    stages it waits on must be at most a ring apart (the first stage of a pair after the last of the one before)."""
    src = open(os.path.join(CSRC, "operators.cu")).read()
    rings = {(int(s), int(per)) for s, per in re.findall(r"MxCfg<\d+, \d+, \d+, (\d+), (\d+),", src)}
    assert rings
    for stages, per in rings:
        for K_tiles in range(1, 12):
            KS, PT = -(-K_tiles // per), (K_tiles + 1) // 2
            waits = {0: [], 1: []}
            g = it0 = 0
            for _ in range(7):
                for pt in range(PT):
                    waits[g & 1] += [it0 + 2 * pt // per + h for h in range(2 // per) if 2 * pt + h < K_tiles]
                    g += 1
                it0 += KS
            assert sorted(waits[0] + waits[1]) == list(range(it0))
            for w in waits.values():
                assert all(0 < b - a <= stages for a, b in zip(w, w[1:]))
