"""CPU checks of the rotary norm, tree attention and paged-cache calls: refusals of the C entry
points and of the binding (no GPU is touched), rotary frequencies, and the division of a
batch's key tiles into runs restated on the host."""
import ctypes
import math

import pytest
import torch

import shifted_sparse_attention_s2attn_b200 as s2

P = 0x10000      # an aligned fake device address: these calls fail before any launch
NULL = None


@pytest.fixture(scope="module")
def lib():
    from shifted_sparse_attention_s2attn_b200 import _build
    _build.build()
    return s2.capi()


# ---- qk_norm_rope -----------------------------------------------------------------------

def _fwd(lib, q=P, k=P, wq=NULL, wk=NULL, pos=NULL, f=P, qo=P, ko=P, B=1, N=8, Hq=4, Hk=2, D=128, R=128, inter=0,
         norm=1, eps=1e-6, af=1.0, pos0=0, dtype=0):
    return lib.qk_norm_rope_fwd(q, k, wq, wk, pos, f, qo, ko, B, N, Hq, Hk, D, R, inter, norm, eps, af, pos0, dtype,
                                NULL)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(N=0), dict(Hq=0), dict(Hk=16385), dict(D=120), dict(D=272), dict(D=8, R=8), dict(R=144), dict(R=24), dict(R=-16),
    dict(dtype=3), dict(dtype=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(af=float("inf")), dict(f=NULL),
    dict(q=NULL), dict(qo=NULL), dict(q=NULL, qo=NULL, k=NULL, ko=NULL), dict(q=P + 8), dict(ko=P + 4), dict(pos=P + 2),
    dict(wq=P, norm=0), dict(wk=P + 8), dict(B=1 << 16, N=1 << 15), dict(pos0=2 ** 31 - 4),
])
def test_norm_rope_refusals(lib, bad):
    assert _fwd(lib, **bad) == -1


@pytest.mark.parametrize("bad,status", [
    (dict(ws=NULL), -3), (dict(ws=P + 16), -3), (dict(n=16), -3), (dict(dwq=P, norm=0), -1), (dict(q=NULL), -1),
    (dict(dq=NULL), -1), (dict(dq_out=NULL), -1), (dict(dk_out=P + 2), -1),
])
def test_norm_rope_bwd_refusals(lib, bad, status):
    a = dict(q=P, k=P, dq_out=P, dk_out=P, dq=P, dk=P, dwq=P, dwk=NULL, norm=1, ws=P, n=1 << 22)
    a.update(bad)
    rc = lib.qk_norm_rope_bwd(a["q"], a["k"], a["dq_out"], a["dk_out"], NULL, NULL, NULL, P, a["dq"], a["dk"], a["dwq"],
                              a["dwk"], 1, 8, 4, 2, 128, 128, 0, a["norm"], 1e-6, 1.0, 0, 0, a["ws"], a["n"], NULL)
    assert rc == status


def test_norm_rope_workspace(lib):
    assert lib.qk_norm_rope_bwd_workspace_bytes(128) == 1024 * 128 * 4
    assert lib.qk_norm_rope_bwd_workspace_bytes(100) == 0


def test_norm_rope_binding_refusals():
    q, k = torch.zeros(1, 4, 4, 64), torch.zeros(1, 4, 2, 64)
    f = torch.zeros(32)
    ok = dict(wq=None, wk=None)
    with pytest.raises(ValueError):   # CPU tensors
        s2.qk_norm_rope_fwd(q, k, q, k, f, **ok)
    with pytest.raises(ValueError):   # neither side
        s2.qk_norm_rope_fwd(None, None, None, None, f)
    with pytest.raises(ValueError):   # an output without its input
        s2.qk_norm_rope_fwd(q, None, q, k, f)
    with pytest.raises(ValueError):   # other length
        s2.qk_norm_rope_fwd(q, torch.zeros(1, 5, 2, 64), q, torch.zeros(1, 5, 2, 64), f)
    with pytest.raises(ValueError):   # other type of the output
        s2.qk_norm_rope_fwd(q, k, q.half(), k, f)
    with pytest.raises(ValueError):   # not contiguous
        s2.qk_norm_rope_fwd(q.transpose(1, 2), k, q, k, f)
    with pytest.raises(ValueError):   # 64-bit positions
        s2.qk_norm_rope_fwd(q, k, q, k, f, positions=torch.zeros(1, 4, dtype=torch.int64))
    with pytest.raises(ValueError):   # a weight without the norm
        s2.qk_norm_rope_fwd(q, k, q, k, f, wq=torch.ones(64), norm=False)
    with pytest.raises(ValueError):   # pos0 past 32 bits
        s2.qk_norm_rope_fwd(q, k, q, k, f, pos0=2 ** 31)
    with pytest.raises(ValueError):   # dwq without a workspace
        s2.qk_norm_rope_bwd(q, k, q, k, q, k, f, dwq=torch.zeros(64))
    with pytest.raises(ValueError):   # the forward's input is missing
        s2.qk_norm_rope_bwd(None, k, q, k, q, k, f)


def test_rope_inv_freq():
    R, base, L0 = 128, 10000.0, 4096
    f = [base ** (-2 * i / R) for i in range(R // 2)]
    near = lambda got, want: all(abs(a - b) <= 2 ** -23 * b for a, b in zip(got.tolist(), want))
    got, af = s2.rope_inv_freq(R)
    assert near(got, f) and af == 1.0
    got, af = s2.rope_inv_freq(R, scaling="linear", factor=8.0)
    assert near(got, [x / 8 for x in f]) and af == 1.0
    got, af = s2.rope_inv_freq(R, scaling="ntk", factor=4.0)
    b2 = base * 4.0 ** (R / (R - 2))
    assert near(got, [b2 ** (-2 * i / R) for i in range(R // 2)]) and af == 1.0
    # the lowest frequency of the larger base is the interpolated one
    assert abs(got[-1].item() - f[-1] / 4) < 1e-6 * f[-1]
    got, af = s2.rope_inv_freq(R, scaling="yarn", factor=8.0, original_len=L0)
    assert abs(af - (0.1 * math.log(8.0) + 1)) < 1e-6
    turns = [L0 * x / (2 * math.pi) for x in f]
    for i in range(R // 2):
        if turns[i] > 32 * base ** (2 / R):     # a step beyond the border on either side
            assert abs(got[i].item() - f[i]) <= 2 ** -23 * f[i]
        elif turns[i] < base ** (-2 / R):
            assert abs(got[i].item() - f[i] / 8) <= 2 ** -23 * f[i]
        else:
            assert f[i] / 8 * (1 - 1e-6) <= got[i].item() <= f[i] * (1 + 1e-6)
    assert s2.rope_inv_freq(2)[0].tolist() == [1.0]


@pytest.mark.parametrize("kw", [dict(R=0), dict(R=3), dict(R=258), dict(R=2, scaling="ntk"), dict(R=64, factor=0.5),
                                dict(R=64, base=1.0), dict(R=64, scaling="yarn", original_len=0), dict(R=64, scaling="log"),
                                dict(R=64, scaling="yarn", beta_fast=1.0, beta_slow=2.0)])
def test_rope_inv_freq_refusals(kw):
    with pytest.raises((ValueError, s2.S2AttnError)):
        s2.rope_inv_freq(**kw)


# ---- tree attention ---------------------------------------------------------------------

def _tree(lib, ptrs=None, B=2, M=4, H=8, Hkv=2, D=128, n_pages=10, page=16, width=5, dtype=0, ws=P, n=1 << 30):
    a = dict(q=P, kn=P, vn=P, kp=P, vp=P, table=P, len=P, new=NULL, mask=NULL, o=P, lse=P)
    a.update(ptrs or {})
    return lib.s2attn_tree_decode(*a.values(), B, M, H, Hkv, D, n_pages, page, width, dtype, ws, n, NULL)


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), -1), (dict(M=0), -1), (dict(H=7), -1), (dict(Hkv=0), -1), (dict(dtype=2), -1), (dict(n_pages=0), -1),
    (dict(width=0), -1), (dict(width=1 << 30, B=600), -2), (dict(B=1025), -2), (dict(M=129), -2), (dict(D=96), -2), (dict(D=256), -2),
    (dict(H=129, Hkv=1), -2), (dict(page=24), -2), (dict(page=8), -2), (dict(n_pages=1 << 27, page=16), -2),
    (dict(ws=NULL), -3), (dict(ws=P + 64), -3), (dict(n=100), -3),
    (dict(ptrs=dict(q=NULL)), -1), (dict(ptrs=dict(vp=P + 8)), -1), (dict(ptrs=dict(len=NULL)), -1),
    (dict(ptrs=dict(mask=P + 4)), -1), (dict(ptrs=dict(new=P + 2)), -1), (dict(ptrs=dict(lse=NULL)), -1),
])
def test_tree_refusals(lib, bad, status):
    assert _tree(lib, **bad) == status


def test_tree_mask_refusals(lib):
    assert lib.s2attn_tree_mask(P, P, NULL, 0, 4, NULL) == -1
    assert lib.s2attn_tree_mask(P, P, NULL, 1, 129, NULL) == -2
    assert lib.s2attn_tree_mask(NULL, P, NULL, 1, 4, NULL) == -1
    assert lib.s2attn_tree_mask(P, P + 4, NULL, 1, 4, NULL) == -1


def test_tree_workspace(lib):
    assert lib.s2attn_tree_decode_workspace_bytes(1, 129, 8, 8, 128) == 0
    assert lib.s2attn_tree_decode_workspace_bytes(1, 4, 8, 3, 128) == 0
    # one key head, one row: all runs of two waves at most, two partials each
    assert 0 < lib.s2attn_tree_decode_workspace_bytes(1, 1, 1, 1, 128) <= 592 * 2 * 130 * 4 + 768
    for M, H, Hkv in [(1, 32, 32), (64, 64, 8), (128, 128, 1), (1, 1024, 1024)]:
        assert lib.s2attn_tree_decode_workspace_bytes(4, M, H, Hkv, 128) < 200 << 20


def test_tree_binding_refusals():
    B, M, H, Hk, D = 2, 4, 8, 2, 64
    t = dict(q=torch.zeros(B, M, H, D, dtype=torch.float16), k_new=torch.zeros(B, M, Hk, D, dtype=torch.float16),
             k_pages=torch.zeros(6, 16, Hk, D, dtype=torch.float16), page_table=torch.zeros(B, 3, dtype=torch.int32),
             cache_len=torch.zeros(B, dtype=torch.int32), lse=torch.zeros(B, H, M),
             workspace=torch.zeros(256, dtype=torch.uint8))
    t.update(v_new=t["k_new"], v_pages=t["k_pages"], o=t["q"])
    for change in [dict(), dict(q=t["q"].float()), dict(k_new=t["k_new"][:, :3]), dict(v_pages=t["k_pages"][:5]),
                   dict(k_pages=t["k_pages"].bfloat16()), dict(page_table=t["page_table"].long()),
                   dict(cache_len=t["cache_len"][:1]), dict(lse=t["lse"].half()), dict(o=t["q"].transpose(1, 2)),
                   dict(tree_mask=torch.zeros(B, M, 2, dtype=torch.int64)), dict(new_len=torch.zeros(B, 1, dtype=torch.int32)),
                   dict(workspace=None)]:
        with pytest.raises(ValueError):
            s2.s2attn_tree_decode(**{**t, **change})     # with no change: CPU tensors


def _runs(lens, new, first_tok, J, min_run):
    """The kernel's division of a unit's key tiles: [(run, sequence, first tile, tiles, total)]."""
    tiles = [(-(-n // 64) + -(-m // 64)) if m > first_tok else 0 for n, m in zip(lens, new)]
    W = sum(tiles)
    runs = min(J, max(1, W // min_run))
    out = []
    for j in range(J):
        w0, w1 = (W * j // runs, W * (j + 1) // runs) if j < runs else (0, 0)
        before = 0
        for b, t in enumerate(tiles):
            a, z = max(w0, before), min(w1, before + t)
            if a < z:
                out.append((j, b, a - before, z - a, t))
            before += t
    return out, tiles


@pytest.mark.parametrize("seed", range(20))
def test_runs_visit_every_tile_once_and_leave_two_partials_at_most(seed):
    import random
    rng = random.Random(seed)
    B = rng.choice([1, 2, 7, 40, 300])
    lens = [rng.choice([0, 1, 63, 64, 65, rng.randint(0, 5000)]) for _ in range(B)]
    new = [rng.randint(0, 20) for _ in range(B)]
    segs, tiles = _runs(lens, new, rng.choice([0, 16]), rng.choice([1, 9, 37, 296]), rng.choice([1, 2, 4]))
    seen = [[0] * t for t in tiles]
    partial = {}
    for j, b, t0, n, total in segs:
        for t in range(t0, t0 + n):
            seen[b][t] += 1
        if n < total:      # slot 1: it holds the sequence's first tile; slot 0: a later part
            key = (j, 1 if t0 == 0 else 0)
            assert key not in partial
            partial[key] = b
    assert all(c == 1 for row in seen for c in row)


# ---- cache ------------------------------------------------------------------------------

@pytest.mark.parametrize("bad,status", [
    (dict(B=0), -1), (dict(A=3), -1), (dict(es=3), -1), (dict(page=20), -2), (dict(Hkv=1, D=4), -2), (dict(kn=NULL), -1),
    (dict(vp=P + 8), -1), (dict(table=P + 1), -1), (dict(n_pages=0), -1), (dict(rows=P + 2, A=3), -1),
])
def test_append_refusals(lib, bad, status):
    a = dict(kn=P, vn=P, kp=P, vp=P, table=P, len=P, rows=NULL, n_rows=NULL, B=2, M=4, A=4, Hkv=2, D=64, n_pages=9,
             page=16, width=4, es=2)
    a.update(bad)
    assert lib.s2attn_cache_append(*a.values(), NULL) == status


def _copy(lib, pairs, n_pages=8, n_pools=1, page_bytes=64, pool=P):
    pools = (ctypes.c_void_p * 200)(*[pool] * 200)
    flat = (ctypes.c_int * max(1, 2 * len(pairs)))(*[x for p in pairs for x in p])
    return lib.s2attn_cache_copy_pages(pools, n_pools, flat, len(pairs), n_pages, page_bytes, NULL)


@pytest.mark.parametrize("pairs", [[(0, 8)], [(-1, 2)], [(0, -1)], [(8, 0)], [(3, 3)], [(0, 1), (2, 1)],
                                   [(0, 1), (1, 2)], [(2, 0), (1, 2)], [(i, i + 4) for i in range(4)] * 3])
def test_copy_refuses_bad_pairs(lib, pairs):
    assert _copy(lib, pairs) == -1


def test_copy_refusals(lib):
    assert _copy(lib, []) == 0                       # nothing to do
    assert _copy(lib, [(0, 1)], n_pools=0) == -1
    assert _copy(lib, [(0, 1)], n_pools=129) == -1
    assert _copy(lib, [(0, 1)], page_bytes=24) == -2
    assert _copy(lib, [(0, 1)], pool=P + 8) == -1
    x = torch.zeros(4, 16, 2, 64)
    for pools, pairs in [([], [(0, 1)]), ([x], [(0, 1)]), ([x, x[:3]], [(0, 1)]), ([x], [(0, 4)]), ([x], [(2 ** 32, 1)]),
                         ([x], [(0, 1, 2)])]:
        with pytest.raises(ValueError):
            s2.s2attn_cache_copy_pages(pools, pairs)


def test_append_binding_refusals():
    kn = torch.zeros(2, 4, 2, 64)
    pages = torch.zeros(5, 16, 2, 64)
    table, n = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for args, kw in [((kn, kn, pages, pages, table, n), {}), ((kn, kn.half(), pages, pages, table, n), {}),
                     ((kn, kn, pages, pages[:, :8], table, n), {}), ((kn, kn, pages, pages, table[:1], n), {}),
                     ((kn, kn, pages, pages, table, n), dict(rows=torch.zeros(2, 3))),
                     ((kn, kn, pages, pages, table, n), dict(n_rows=torch.zeros(3, dtype=torch.int32)))]:
        with pytest.raises(ValueError):
            s2.s2attn_cache_append(*args, **kw)


def test_sizes_that_do_not_fit_the_c_call_are_refused():
    """Expanded host tensors (no memory): sizes past 32 bits never reach a 32-bit argument."""
    big = torch.zeros(1).expand(2 ** 20, 2 ** 12, 1, 16)
    with pytest.raises(ValueError, match="2\\^30"):
        s2.qk_norm_rope_fwd(big, None, big, None, torch.zeros(8))
    with pytest.raises(ValueError, match="2\\^31"):
        s2.s2attn_cache_copy_pages([torch.zeros(1).expand(2 ** 32 + 2, 16)], [(0, 1)])
    with pytest.raises(ValueError, match="2\\^30"):
        s2.s2attn_cache_append(big, big, big, big, None, None)
    pool = torch.zeros(1).expand(2 ** 30, 16, 1, 16)
    kn = torch.zeros(1, 1, 1, 16)
    with pytest.raises(ValueError, match="2\\^31"):
        s2.s2attn_cache_append(kn, kn, pool, pool, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
