"""s2attn_cache_append and s2attn_cache_copy_pages: exact copies, nothing else touched."""
import random

import pytest
import torch

import shifted_sparse_attention_s2attn_b200 as s2
from serving_utils import make_cache, no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s2.clear_device_error()


def _expect(pool, new, table, lens, rows, n_rows, page):
    pool = pool.clone()
    for b in range(new.shape[0]):
        for j in range(n_rows[b]):
            pos = int(lens[b]) + j
            pool[int(table[b, pos // page]), pos % page] = new[b, rows[b][j]]
    return pool


@pytest.mark.parametrize("lens,M,page,Hkv,D,dt", [
    ([0], 1, 16, 1, 64, torch.bfloat16), ([5, 16, 0], 3, 16, 2, 64, torch.float16),
    ([31, 100], 40, 32, 8, 128, torch.bfloat16), ([0, 1, 2, 3], 17, 64, 3, 80, torch.float32),
    ([700], 1500, 256, 1, 128, torch.bfloat16), ([3], 5, 16, 40, 128, torch.bfloat16),
])
@pytest.mark.parametrize("picked", [False, True])
def test_append(lens, M, page, Hkv, D, dt, picked):
    rng = random.Random(M)
    kp, vp, table, n = make_cache(lens, M, page, Hkv, D, dt, 1, fill=0.5)
    g = torch.Generator().manual_seed(2)
    kn, vn = (torch.randn(len(lens), M, Hkv, D, generator=g).to(dt) for _ in range(2))
    rows = [list(range(M)) for _ in lens]
    counts = [M] * len(lens)
    r = c = None
    if picked:      # any order, the same row twice, no row, counts above the width
        A = min(M, 6)
        rows = [[rng.randrange(M) for _ in range(A)] for _ in lens]
        counts = [rng.choice([0, A, rng.randint(0, A)]) for _ in lens]
        r = torch.tensor(rows, dtype=torch.int32).cuda()
        c = torch.tensor([x if x < A else 10 ** 6 for x in counts], dtype=torch.int32).cuda()
        if counts[0] == 0:
            c[0] = -3
    dk, dv = kp.cuda(), vp.cuda()
    s2.s2attn_cache_append(kn.cuda(), vn.cuda(), dk, dv, table.cuda(), n.cuda(), rows=r, n_rows=c)
    no_device_error()
    assert torch.equal(dk.cpu(), _expect(kp, kn, table, n, rows, counts, page))
    assert torch.equal(dv.cpu(), _expect(vp, vn, table, n, rows, counts, page))


def test_append_records_what_is_out_of_range_and_skips_it():
    kp, vp, table, n = make_cache([10, 20, 3], 4, 16, 2, 64, torch.bfloat16, 1, fill=0.5)
    kn = torch.randn(3, 4, 2, 64).bfloat16()
    ok = _expect(kp, kn, table, n, [[0, 1, 2, 3]] * 3, [0, 4, 0], 16)
    # a page outside the pool; a negative length; a row outside the new ones
    for change, where in [("table", 99), ("table", -1), ("len", -40), ("len", 10 ** 9), ("row", 4), ("row", -1)]:
        t, l, r = table.clone(), n.clone(), torch.tensor([[0, 1, 2, 3]] * 3, dtype=torch.int32)
        counts = torch.tensor([4, 4, 0], dtype=torch.int32)
        if change == "table":
            t[0, 0] = where
        elif change == "len":
            l[0] = where
        else:
            r[0] = where
        dk, dv = kp.cuda(), vp.cuda()
        s2.s2attn_cache_append(kn.cuda(), kn.cuda(), dk, dv, t.cuda(), l.cuda(), rows=r.cuda(), n_rows=counts.cuda())
        torch.cuda.synchronize()
        assert s2.get_device_error() == (-6, 0x740), change
        s2.clear_device_error()
        assert torch.equal(dk.cpu(), ok), change       # sequence 1's rows, nothing of sequence 0
    no_device_error()


@pytest.mark.parametrize("n_pages,page,Hkv,D,dt,n_pools,n_pairs", [
    (2, 16, 1, 64, torch.bfloat16, 1, 1), (9, 16, 8, 128, torch.bfloat16, 3, 4), (1100, 1, 1, 8, torch.float16, 2, 500),
    (40, 64, 3, 80, torch.float32, 128, 20), (1000, 2, 1, 16, torch.bfloat16, 1, 460),
])
def test_copy_pages(n_pages, page, Hkv, D, dt, n_pools, n_pairs):
    g = torch.Generator().manual_seed(n_pages)
    pools = [torch.randn(n_pages, page, Hkv, D, generator=g).to(dt) for _ in range(n_pools)]
    order = random.Random(1).sample(range(n_pages), 2 * n_pairs)
    pairs = list(zip(order[::2], order[1::2]))
    dev = [p.cuda() for p in pools]
    s2.s2attn_cache_copy_pages(dev, pairs)
    no_device_error()
    for p, d in zip(pools, dev):
        for a, b in pairs:
            p[b] = p[a]
        assert torch.equal(d.cpu(), p)


def test_copy_one_page_to_many_and_nothing():
    pool = torch.randn(6, 16, 2, 64).cuda()
    want = pool.clone()
    s2.s2attn_cache_copy_pages([pool], [])
    assert torch.equal(pool, want)
    s2.s2attn_cache_copy_pages([pool], [(2, 0), (2, 5), (2, 3)])
    want[[0, 5, 3]] = want[2].clone()
    no_device_error()
    assert torch.equal(pool, want)
