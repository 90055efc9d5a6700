"""s2attn_tree_decode where scores are infinite, and where they grow from tile to tile."""
import math

import pytest
import torch

import shifted_sparse_attention_s2attn_b200 as s2
from serving_utils import HALF_STEP, check_close, make_cache, no_device_error
from test_gpu_tree import _case, _run

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s2.clear_device_error()


def _row(q, k, v, dt):
    """o, lse of one row in 64 bits and their bounds as in serving_utils.attend; keys of score -inf have
    weight 0 (and a row that has no others is 0 with lse = -inf)."""
    D = q.shape[0]
    s = (k.double() @ q.double()) / math.sqrt(D)
    keep = s > -math.inf
    if not keep.any():
        z = torch.zeros(D).double()
        return z, z[0] - math.inf, z, z[0]
    s, k, v = s[keep], k[keep].double(), v[keep].double()
    p = torch.exp(s - s.max())
    o, pv = (p @ v) / p.sum(), (p @ v.abs()) / p.sum()
    lse = s.max() + p.sum().log()
    e = D * 2.0 ** -23 * ((k.abs() @ q.double().abs()).max() / math.sqrt(D)) + 2.0 ** -18
    u = HALF_STEP[dt]
    tiny = 2.0 ** -25 if dt is FP else 0.0
    return o, lse, (u * o.abs() + (u + 2 * e) * pv + tiny * (1 + v.abs().sum(0))) * 1.02, e + 2.0 ** -18 * (1 + lse.abs())


def _check_rows(c, see, words, new):
    B, M, H, D = c["q"].shape
    o, lse = _run(c, words, new, True)
    no_device_error()
    Hkv, page = c["k_new"].shape[2], c["k_pages"].shape[1]
    for b in range(B):
        n = int(c["cache_len"][b])
        ids = c["page_table"][b][:-(-n // page)].long()
        for h in range(H):
            g = h * Hkv // H
            kc, vc = (c[x][ids].flatten(0, 1)[:n, g] for x in ("k_pages", "v_pages"))
            for m in range(new[b]):
                on = see[b, m, :new[b]].nonzero()[:, 0]
                wo, wl, bo, bl = _row(c["q"][b, m, h], torch.cat([kc, c["k_new"][b, on, g]]),
                                      torch.cat([vc, c["v_new"][b, on, g]]), c["q"].dtype)
                check_close(o[b, m, h], wo, bo, f"o of sequence {b} token {m} head {h}")
                check_close(lse[b, h, m], wl, bl, f"lse of sequence {b} token {m} head {h}")


# 300 key heads leave one run a unit, a few heads one tile a run
@pytest.mark.parametrize("H,Hkv", [(2, 1), (300, 300)])
@pytest.mark.parametrize("dt", [BF, FP])
def test_scores_of_minus_infinity_have_weight_zero(H, Hkv, dt):
    M, page = 5, 16
    c, see, words, new = _case([0, 200, 64, 3, 130], M, H, Hkv, 64, page, dt, "chain", seed=11)
    c["q"][..., 7] = c["q"][..., 7].abs() + 0.5
    low = -math.inf

    def cached(b, tokens):
        for t in tokens:
            c["k_pages"][c["page_table"][b, t // page].long(), t % page, :, 7] = low
    c["k_new"][0, 0, :, 7] = low          # the first key of all: token 0 sees no other
    cached(1, range(64))                  # a whole first tile
    cached(2, range(64))                  # the whole cache; then the first drafted one
    c["k_new"][2, 0, :, 7] = low
    cached(3, [0, 1])
    cached(4, [5, 64, 65, 129])           # single ones, and the last tile of the cache
    c["k_new"][4, 4, :, 7] = low
    _check_rows(c, see, words, new)


@pytest.mark.parametrize("H,Hkv", [(2, 1), (300, 300)])
def test_a_masked_key_of_minus_infinity_changes_nothing(H, Hkv):
    c, see, words, new = _case([0, 70], 6, H, Hkv, 64, 16, BF, "any", seed=5)
    clean = _run(c, words, new, True)
    c["k_new"][:, 2, :, 3] = -math.inf
    o, lse = _run(c, words, new, True)
    no_device_error()
    blind = ~see[:, :, 2]
    assert torch.equal(o[blind], clean[0][blind])
    assert torch.equal(lse.transpose(1, 2)[blind], clean[1].transpose(1, 2)[blind])


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("step", [0.5, 2.5, 3.0, 5.0, 6.0])
@pytest.mark.parametrize("Hkv", [1, 300])
def test_scores_that_grow_from_tile_to_tile(dt, step, Hkv):
    """Every tile's maximum is `step` nats above the last one's: below and above the growth at which the
    running maximum moves."""
    D, page, n = 64, 64, 640
    c, see, words, new = _case([n], 2, Hkv, Hkv, D, page, dt, "chain", seed=2)
    c["q"][..., 0] = math.sqrt(D)
    for t in range(n // page):
        c["k_pages"][c["page_table"][0, t].long(), :, :, 0] = step * t
    _check_rows(c, see, words, new)
