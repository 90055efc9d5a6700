"""s2attn_tree_mask and s2attn_tree_decode against 64-bit attention over the gathered cache.

The pools' unused rows and pages hold NaN, so that a key that must not be seen shows.  The
bounds are derived in serving_utils.attend.
"""
import random

import pytest
import torch

import shifted_sparse_attention_s2attn_b200 as s2
from serving_utils import (attend, check_close, make_cache, no_device_error, random_parents, tree_see, words_of)

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s2.clear_device_error()


@pytest.mark.parametrize("B,M", [(1, 1), (3, 2), (2, 13), (1, 63), (2, 64), (1, 65), (2, 128)])
def test_tree_mask(B, M):
    rng = random.Random(M)
    trees = random_parents(B, M, rng)
    trees[0] = list(range(-1, M - 1))      # a chain, the deepest tree
    see, depth = tree_see(trees)
    mask = torch.full((B, M, (M + 63) // 64), -1, dtype=torch.int64, device="cuda")
    dep = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    par = torch.tensor(trees, dtype=torch.int32, device="cuda")
    s2.s2attn_tree_mask(par, mask, dep)
    no_device_error()
    assert torch.equal(mask.cpu(), words_of(see)) and torch.equal(dep.cpu(), depth)
    mask.zero_()
    s2.s2attn_tree_mask(par, mask)
    no_device_error()
    assert torch.equal(mask.cpu(), words_of(see))


def test_tree_mask_records_bad_parents():
    par = torch.tensor([[-1, 0, 2, 1], [-1, 0, 1, 2], [-2, 0, 0, 9]], dtype=torch.int32, device="cuda")
    mask = torch.zeros(3, 4, 1, dtype=torch.int64, device="cuda")
    s2.s2attn_tree_mask(par, mask)
    torch.cuda.synchronize()
    assert s2.get_device_error() == (-6, 0x640)
    s2.clear_device_error()
    assert mask[1, :, 0].tolist() == [1, 3, 7, 15]
    assert mask[0, :, 0].tolist() == [1, 3, 4, 11] and mask[2, :, 0].tolist() == [1, 3, 5, 8]


def _case(lens, M, H, Hkv, D, page, dt, mask, new=None, seed=0, fill=float("nan"), q_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    rnd = lambda *s: torch.randn(s, generator=g).to(dt)
    kp, vp, table, n = make_cache(lens, 0, page, Hkv, D, dt, seed + 1, fill=fill)
    c = dict(q=(rnd(B, M, H, D) * q_scale), k_new=rnd(B, M, Hkv, D), v_new=rnd(B, M, Hkv, D), k_pages=kp, v_pages=vp,
             page_table=table, cache_len=n)
    rng = random.Random(seed)
    if mask == "chain":
        see, words = torch.ones(M, M, dtype=torch.bool).tril().expand(B, M, M), None
    elif mask == "tree":
        see, _ = tree_see(random_parents(B, M, rng))
        words = words_of(see)
    else:      # any bits: later tokens seen, own token not, rows that see nothing
        see = torch.rand(B, M, M, generator=g) < 0.4
        see[:, ::3] = False
        words = words_of(see)
    new = [M] * B if new is None else new
    for b, m in enumerate(new):     # rows that do not exist hold NaN too
        for t in ("q", "k_new", "v_new"):
            c[t][b, m:] = float("nan")
    return c, see, words, new


def _run(c, words, new, ragged, o_fill=7.0):
    d = {n: t.cuda() for n, t in c.items()}
    B, M, H, D = c["q"].shape
    o = torch.full_like(d["q"], o_fill)
    lse = torch.full((B, H, M), o_fill, dtype=torch.float32, device="cuda")
    ws = torch.empty(s2.s2attn_tree_decode_workspace_bytes(B, M, H, c["k_new"].shape[2], D), dtype=torch.uint8,
                     device="cuda").fill_(0xff)
    s2.s2attn_tree_decode(d["q"], d["k_new"], d["v_new"], d["k_pages"], d["v_pages"], d["page_table"], d["cache_len"],
                          o, lse, ws, tree_mask=None if words is None else words.cuda(),
                          new_len=torch.tensor(new, dtype=torch.int32, device="cuda") if ragged else None)
    return o.cpu(), lse.cpu()


def _check(c, see, words, new, ragged=True):
    o, lse = _run(c, words, new, ragged)
    no_device_error()
    wo, wl, bo, bl = attend(c["q"], c["k_new"], c["v_new"], c["k_pages"], c["v_pages"], c["page_table"], c["cache_len"],
                            see, new)
    for b, m in enumerate(new):
        assert (o[b, m:] == 7).all() and (lse[b, :, m:] == 7).all(), "rows behind the last drafted token changed"
        check_close(o[b, :m], wo[b, :m], bo[b, :m], f"o of sequence {b}")
        check_close(lse[b, :, :m], wl[b, :, :m], bl[b, :, :m], f"lse of sequence {b}")
    return o, lse


@pytest.mark.parametrize("lens,M,H,Hkv,D,page,dt", [
    ([0], 1, 1, 1, 128, 16, BF),                       # nothing cached, one token
    ([1], 1, 1, 1, 64, 16, FP),
    ([63, 64, 65], 1, 4, 4, 128, 64, BF),              # tile borders
    ([15, 16, 17, 0, 130], 3, 8, 2, 64, 16, FP),       # pages that end inside a tile
    ([300, 7], 13, 8, 1, 128, 32, BF),
    ([200], 64, 8, 8, 128, 128, FP),
    ([129, 31], 65, 2, 1, 64, 256, BF),                # two drafted tiles
    ([70], 128, 3, 3, 128, 16, BF),
    ([90, 1], 30, 10, 2, 128, 16, FP),                 # five heads a key head: row tiles of 25 tokens
    ([100], 40, 8, 1, 64, 64, BF),                     # three row tiles
    ([40], 2, 128, 1, 128, 16, BF),                    # one token a row tile
    ([33], 5, 7, 1, 64, 16, FP),
    ([2900], 2, 2, 1, 128, 64, BF),                    # one sequence over many runs
    ([1, 700, 0, 64, 0, 200, 33, 5], 4, 2, 1, 64, 16, FP),
])
@pytest.mark.parametrize("mask", ["chain", "tree", "any"])
def test_attention(lens, M, H, Hkv, D, page, dt, mask):
    _check(*_case(lens, M, H, Hkv, D, page, dt, mask), ragged=False)


@pytest.mark.parametrize("mask", ["chain", "tree", "any"])
def test_ragged_batches(mask):
    rng = random.Random(5)
    for seed, B, M, H, Hkv, D in [(1, 9, 20, 4, 2, 64), (2, 3, 70, 8, 1, 64), (3, 40, 3, 2, 2, 128)]:
        lens = [rng.choice([0, 1, 64, rng.randint(0, 400)]) for _ in range(B)]
        new = [rng.choice([0, 1, M, rng.randint(0, M)]) for _ in range(B)]
        new[0] = 0
        _check(*_case(lens, M, H, Hkv, D, 16, BF, mask, new=new, seed=seed))


def test_nothing_to_do():
    c, see, words, new = _case([40, 0], 3, 2, 1, 64, 16, BF, "chain", new=[0, 0])
    _check(c, see, words, new)


def test_large_scores():
    """Scores up to several hundred: the running maximum moves in most tiles."""
    _check(*_case([500, 130], 4, 4, 2, 128, 16, BF, "tree", q_scale=30.0), ragged=False)


def test_masked_rows_that_hold_infinities_reach_nobody_else():
    """Drafted rows with inf and NaN reach exactly the tokens whose mask shows them."""
    for H, M, mask in [(2, 6, "tree"), (8, 70, "any"), (1, 5, "chain")]:
        c, see, words, new = _case([70, 0], M, H, 1, 64, 16, FP, mask, seed=4)
        bad = M - 2
        c["v_new"][:, bad, :, 3] = float("inf")
        c["v_new"][:, bad, :, 40] = float("nan")
        o, lse = _run(c, words, new, False)
        no_device_error()
        clean = {n: t.clone() for n, t in c.items()}
        clean["v_new"][:, bad, :, 3] = clean["v_new"][:, bad, :, 40] = 0.0
        wo, wl, bo, bl = attend(clean["q"], clean["k_new"], clean["v_new"], clean["k_pages"], clean["v_pages"],
                                clean["page_table"], clean["cache_len"], see, new)
        hit = see[:, :, bad]
        wo[..., 3] = torch.where(hit[:, :, None], float("inf"), wo[..., 3])
        wo[..., 40] = torch.where(hit[:, :, None], float("nan"), wo[..., 40])
        check_close(o, wo, bo, "o")
        check_close(lse, wl, bl, "lse")
        # a key of NaN makes the scores of those who see it NaN, of nobody else
        c["v_new"][:, bad] = 1.0
        c["k_new"][:, bad] = float("nan")
        o, lse = _run(c, words, new, False)
        no_device_error()
        assert torch.equal(o.isnan().all(-1).all(-1), hit) and torch.equal(o.isnan().any(-1).any(-1), hit)
        assert torch.equal(lse.isnan().all(1), hit)


def test_bad_pages_and_lengths_are_recorded_and_stay_in_their_sequence():
    c, see, words, new = _case([100, 200, 150], 3, 4, 2, 64, 16, BF, "chain")
    wo, wl, bo, bl = attend(*[c[n] for n in ("q", "k_new", "v_new", "k_pages", "v_pages", "page_table", "cache_len")],
                            see, new)
    for what, value in [("page", -1), ("page", 10 ** 9), ("page", c["k_pages"].shape[0]), ("len", -5), ("len", 10 ** 9)]:
        x = {n: t.clone() for n, t in c.items()}
        if what == "page":
            x["page_table"][1, 3] = value
        else:
            x["cache_len"][1] = value
            if value > 0:      # the clamped length meets the table's unused entries
                x["page_table"][1][x["page_table"][1] < 0] = 0
        o, lse = _run(x, words, new, False)
        torch.cuda.synchronize()
        assert s2.get_device_error() == (-6, 0x640), (what, value)
        s2.clear_device_error()
        for b in (0, 2):
            check_close(o[b], wo[b], bo[b], f"o of sequence {b} beside {what} {value}")
            check_close(lse[b], wl[b], bl[b], f"lse of sequence {b}")
    # drafted counts outside 0..M
    for value in (-1, 4):
        o, lse = _run(c, words, [3, value, 3], True)
        torch.cuda.synchronize()
        assert s2.get_device_error() == (-6, 0x640)
        s2.clear_device_error()
        check_close(o[2], wo[2], bo[2], "o of sequence 2")
    no_device_error()


def test_repeats_are_bitwise_equal():
    c, see, words, new = _case([900, 64, 333], 9, 8, 2, 128, 16, BF, "tree")
    a = _run(c, words, new, False)
    for _ in range(3):
        b = _run(c, words, new, False)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_call_follows_the_lengths():
    """A captured call on a stream of its own, replayed after the cache has grown, while another call
    with a workspace of its own runs on a second stream."""
    page, Hkv, D, H, M, B = 16, 2, 64, 4, 2, 3
    lens = [10, 60, 0]
    c, see, words, new = _case(lens, M, H, Hkv, D, page, BF, "chain")
    kp, vp, table, n = make_cache(lens, 200, page, Hkv, D, BF, 9, fill=0.25)
    c.update(k_pages=kp, v_pages=vp, page_table=table, cache_len=n)
    d = {x: t.cuda() for x, t in c.items()}
    o, o2 = torch.empty_like(d["q"]), torch.empty_like(d["q"])
    lse, lse2 = (torch.empty(B, H, M, device="cuda") for _ in range(2))
    ws, ws2 = (torch.empty(s2.s2attn_tree_decode_workspace_bytes(B, M, H, Hkv, D), dtype=torch.uint8, device="cuda")
               for _ in range(2))
    names = ("q", "k_new", "v_new", "k_pages", "v_pages", "page_table", "cache_len")
    args = [d[x] for x in names]
    st, st2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        s2.s2attn_tree_decode(*args, o, lse, ws)
    for grown in ([10, 60, 0], [11, 62, 130], [200, 190, 64]):
        d["cache_len"].copy_(torch.tensor(grown, dtype=torch.int32))
        torch.cuda.synchronize()
        with torch.cuda.stream(st2):
            s2.s2attn_tree_decode(*args, o2, lse2, ws2)
        with torch.cuda.stream(st):
            g.replay()
        no_device_error()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        wo, wl, bo, bl = attend(*[c[x] for x in names[:-1]], torch.tensor(grown), see, new)
        check_close(o, wo, bo, "o")
        check_close(lse, wl, bl, "lse")


def test_agrees_with_the_contiguous_decoding_step():
    """The same sequence as a contiguous cache through s2attn_decode: both within their bounds, so
    within the sum of two output roundings and two P roundings of each other."""
    N, M, H, D, page = 1000, 4, 4, 128, 64
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(1, n, H, D, generator=g).bfloat16().cuda() for n in (M, N, N))
    o, lse = torch.empty_like(q), torch.empty(1, H, M, device="cuda")
    ws = torch.empty(s2.s2attn_decode_workspace_bytes(1, M, N, H, D), dtype=torch.uint8, device="cuda")
    s2.s2attn_decode(q, k, v, o, lse, ws)
    n = N - M
    pages = -(-n // page)
    kp, vp = (torch.zeros(pages * page, H, D, dtype=BF, device="cuda") for _ in range(2))
    kp[:n], vp[:n] = k[0, :n], v[0, :n]
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    ws2 = torch.empty(s2.s2attn_tree_decode_workspace_bytes(1, M, H, H, D), dtype=torch.uint8, device="cuda")
    s2.s2attn_tree_decode(q, k[:, n:].contiguous(), v[:, n:].contiguous(), kp.view(pages, page, H, D),
                          vp.view(pages, page, H, D), torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                          torch.tensor([n], dtype=torch.int32, device="cuda"), o2, lse2, ws2)
    no_device_error()
    # sum p|v| <= max over keys of |v| < 5 times the sum of p; measured outputs are far smaller
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -8 * 2 * (o.float().abs().max() + 1)
    assert (lse - lse2).abs().max() <= 1e-4


def test_every_mask_bit_set():
    """Bits of tokens that do not exist (j >= new_len, j >= M) show nothing."""
    B, M = 3, 70
    c, _, _, new = _case([20, 0, 129], M, 4, 2, 64, 16, BF, "chain", new=[70, 33, 1])
    see = torch.ones(B, M, M, dtype=torch.bool)
    words = torch.full((B, M, 2), -1, dtype=torch.int64)
    _check(c, see, words, new)


def test_pages_behind_the_first_four_gigabytes():
    """A pool of more than 2^32 bytes and 2^31 elements: the sequence's pages are its last ones."""
    page, Hkv, D, H, M, n = 64, 8, 128, 8, 2, 150
    n_pages = (2 ** 31 + 2 ** 24) // (page * Hkv * D)
    c, see, words, new = _case([n], M, H, Hkv, D, page, BF, "chain", seed=3)
    used = -(-n // page)
    pools = []
    for name in ("k_pages", "v_pages"):
        pool = torch.zeros(n_pages, page, Hkv, D, dtype=BF, device="cuda")
        ids = c["page_table"][0, :used].long()
        pool[n_pages - used:] = c[name][ids].cuda()
        pools.append(pool)
    table = torch.arange(n_pages - used, n_pages, dtype=torch.int32, device="cuda")[None]
    q, kn, vn, ln = (c[x].cuda() for x in ("q", "k_new", "v_new", "cache_len"))
    o, lse = torch.empty_like(q), torch.empty(1, H, M, device="cuda")
    ws = torch.empty(s2.s2attn_tree_decode_workspace_bytes(1, M, H, Hkv, D), dtype=torch.uint8, device="cuda")
    s2.s2attn_tree_decode(q, kn, vn, *pools, table, ln, o, lse, ws)
    no_device_error()
    wo, wl, bo, bl = attend(*[c[x] for x in ("q", "k_new", "v_new", "k_pages", "v_pages", "page_table", "cache_len")],
                            see, new)
    check_close(o, wo, bo, "o")
    check_close(lse, wl, bl, "lse")
    # appended rows and copied pages beyond the same border
    s2.s2attn_cache_append(kn, vn, *pools, table, ln)
    s2.s2attn_cache_copy_pages(pools, [(n_pages - 1, 0), (1, n_pages - 2)])
    no_device_error()
    for pool, new_rows in zip(pools, (kn, vn)):
        assert torch.equal(pool[n_pages - 1, n % page:n % page + M], new_rows[0])
        assert torch.equal(pool[0].nan_to_num(), pool[n_pages - 1].nan_to_num()) and (pool[n_pages - 2] == 0).all()


_FIRST_CALL = """
import torch
import shifted_sparse_attention_s2attn_b200 as s2
B, M, H, Hk, D = 1, 2, 4, 2, 64
q, kn = (torch.randn(B, M, h, D, device="cuda").half() for h in (H, Hk))
pages = torch.randn(4, 16, Hk, D, device="cuda").half()
table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
n = torch.tensor([40], dtype=torch.int32, device="cuda")
o, lse = torch.zeros_like(q), torch.zeros(B, H, M, device="cuda")
f = s2.rope_inv_freq(D)[0].cuda()
ws = torch.empty(s2.s2attn_tree_decode_workspace_bytes(B, M, H, Hk, D), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    s2.qk_norm_rope_fwd(q, kn, q, kn, f, pos0=40)
    s2.s2attn_tree_decode(q, kn, kn, pages, pages, table, n, o, lse, ws)
    s2.s2attn_cache_append(kn, kn, pages, pages, table, n)
g.replay()
torch.cuda.synchronize()
assert s2.get_device_error() == (0, 0)
assert o.abs().sum() > 0 and torch.equal(pages[2, 8:10], kn[0])
print("captured first call ok")
"""


def test_the_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALL], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "captured first call ok" in r.stdout, r.stderr[-2000:]


def test_two_host_threads_at_once():
    """Two threads, each with its own stream, workspace and inputs."""
    import threading
    cases = [_case([300, 40], 5, 8, 2, 128, 16, BF, "tree", seed=s) for s in (1, 2)]
    want = [_run(c, w, n, False) for c, _, w, n in cases]
    got = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got[i] = _run(cases[i][0], cases[i][2], cases[i][3], False)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    no_device_error()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


@pytest.mark.parametrize("lens,M,H,Hkv,D,page", [
    ([i % 37 for i in range(1024)], 1, 2, 1, 64, 16),       # the most sequences a call takes
    ([10, 5000, 4096], 3, 6, 2, 128, 4096),                 # pages far larger than a tile
    ([9000], 1, 1, 1, 64, 16),                              # one row, hundreds of runs of one tile
    ([50], 1, 300, 300, 64, 16),                            # more units than CTAs fit: one run each
])
def test_sizes_at_the_ends(lens, M, H, Hkv, D, page):
    _check(*_case(lens, M, H, Hkv, D, page, BF, "chain"), ragged=False)
