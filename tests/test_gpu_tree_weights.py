"""s2attn_tree_decode where many small weights make up a row, and with large scores in fp16."""
import math

import pytest
import torch

import shifted_sparse_attention_s2attn_b200 as s2
from serving_utils import HALF_STEP, check_close, make_cache, no_device_error
from test_gpu_tree import _case, _check, _run

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s2.clear_device_error()


def _one_ahead(dt, N, gap, at, M=1, H=1):
    """N cached keys and the drafted ones of score 0 and value 1, one more of score `gap` and value 0 at
    index `at` of the cache: o is the weight of the others."""
    D, page = 64, 128
    kp, vp, table, n = make_cache([N + 1], 0, page, 1, D, dt, 1, fill=0.0)
    kp.zero_()
    vp.fill_(1.0)
    pg, row = int(table[0, at // page]), at % page
    kp[pg, row, :, 0] = gap
    vp[pg, row] = 0.0
    q = torch.zeros(1, M, H, D, dtype=dt)
    q[..., 0] = math.sqrt(D)
    new = torch.zeros(1, M, 1, D, dtype=dt)
    c = dict(q=q, k_new=new, v_new=torch.ones_like(new), k_pages=kp, v_pages=vp, page_table=table, cache_len=n)
    o, lse = _run(c, None, [M], False)
    no_device_error()
    others = N + 1 + torch.arange(M, dtype=torch.float64)
    want, want_lse = others / (others + math.exp(gap)), (others + math.exp(gap)).log()
    # P is held in the input's type, in fp16 scaled so that its largest is at least 2^11: an element is off
    # by half a step or, where it is subnormal, by 2^-25, which is 2^-36 of the sum; o is rounded once
    # more; exponentials are off by 2^-18, each of at most 700 additions to a running sum by 2^-23
    bound = (2 * HALF_STEP[dt] + 2.0 ** -18 + 700 * 2.0 ** -23) * want * 1.02
    if dt is FP:
        bound += 2.0 ** -36 * others + 2.0 ** -25
    check_close(o, want[None, :, None, None].expand(o.shape), bound[None, :, None, None].expand(o.shape), "o")
    check_close(lse, want_lse.expand(lse.shape), (2.0 ** -18 * (1 + want_lse) + 700 * 2.0 ** -23).expand(lse.shape), "lse")


GAPS = [2.5, 5.25, 8.0, 14.0, 16.0, 17.0, 17.5, 18.0, 20.0]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("at", [0, 51000, 102400])
def test_many_small_weights_are_not_lost(dt, gap, at):
    """102401 weights of e^-gap beside one of 1, over many runs."""
    _one_ahead(dt, 102400, gap, at)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("at", [0, 700, 9000, 20000])
def test_many_small_weights_in_one_run(dt, gap, at):
    """128 row tiles (of one token of 128 heads) leave two runs of 10000 keys each."""
    _one_ahead(dt, 20000, gap, at, M=128, H=128)


@pytest.mark.parametrize("D,q_scale", [(64, 30.0), (128, 3.0), (128, 30.0)])
def test_large_scores_in_fp16(D, q_scale):
    """The running maximum moves in most tiles."""
    _check(*_case([500, 130], 4, 4, 2, D, 16, FP, "tree", q_scale=q_scale), ragged=False)
