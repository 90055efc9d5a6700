"""The division of tree attention's key tiles into runs (serving_runs restates it; the GPU tests compare
it with the runs that the kernel notes): every tile once, and what the join relies on."""
import random

import pytest

import shifted_sparse_attention_s2attn_b200 as s2
from serving_runs import SEQ_COST, plan, segments


@pytest.fixture(scope="module")
def lib():
    from shifted_sparse_attention_s2attn_b200 import _build
    _build.build()
    return s2.capi()


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_once_and_a_partial_in_every_run_of_a_sequence(seed):
    rng = random.Random(seed)
    B = rng.choice([1, 2, 7, 40, 300, 1024])
    lens = [rng.choice([0, 1, 63, 64, 65, rng.randint(0, 5000)]) for _ in range(B)]
    new = [rng.choice([0, 1, 128, rng.randint(0, 20)]) for _ in range(B)]
    J = rng.choice([1, 2, 9, 37, 296, 592])
    segs, tiles = segments(lens, new, rng.choice([0, 0, 16]), J)
    seen = [[0] * t for t in tiles]
    slots, runs_of, work = set(), {}, {}
    for j, b, t0, n, total in segs:
        assert 0 <= j < J
        for t in range(t0, t0 + n):
            seen[b][t] += 1
        work[j] = work.get(j, 0) + n
        runs_of.setdefault(b, []).append((j, t0, n))
        if n < total:        # a partial: slot 1 holds a sequence's first tile, slot 0 a later part
            assert (j, t0 == 0) not in slots
            slots.add((j, t0 == 0))
    assert all(c == 1 for row in seen for c in row)
    for b, parts in runs_of.items():
        # neighbouring runs without a gap, in order: the join reads slot 1 of the first, slot 0 of the others
        js = [j for j, _, _ in parts]
        assert js == list(range(js[0], js[-1] + 1))
        assert [t0 == 0 for _, t0, _ in parts] == [True] + [False] * (len(parts) - 1)
    if segs:                 # no run takes much more than its share of tiles and ends
        runs = min(J, sum(tiles))
        assert max(work.values()) <= -(-sum(t + SEQ_COST for t in tiles if t) // runs)


def test_runs_without_tiles_and_cuts_behind_a_sequences_last_tile():
    """Many short sequences: shares that fall into the weight of ends alone."""
    segs, tiles = segments([1] * 50, [1] * 50, 0, 592)
    assert {j for j, *_ in segs} < set(range(100)) and sum(tiles) == 100
    assert len(segs) == len({(b, t0) for _, b, t0, _, _ in segs})


@pytest.mark.parametrize("M,H,Hkv", [(1, 1, 1), (1, 32, 32), (32, 32, 8), (64, 64, 8), (128, 128, 1), (13, 8, 2),
                                     (128, 8, 8), (40, 2, 1), (2, 300, 300), (30, 10, 2), (1, 1024, 1024), (100, 50, 50)])
@pytest.mark.parametrize("B,D", [(1, 64), (7, 128)])
def test_the_workspace_follows_the_plan(lib, M, H, Hkv, B, D):
    up = lambda x: -(-x // 256) * 256
    tok, row_tiles, J, slot_rows = plan(M, H, Hkv)
    rows = Hkv * row_tiles * J * 2 * slot_rows
    want = up(rows * D * 4) + up(rows * 8) + up(B * row_tiles * 8)
    assert lib.s2attn_tree_decode_workspace_bytes(B, M, H, Hkv, D) == want
