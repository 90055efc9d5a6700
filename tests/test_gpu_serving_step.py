"""The serving calls together, as a decoding step uses them: drafted tokens of a tree are normed
and rotated at their positions, attend over the paged cache, the accepted rows are appended, a
sequence is forked, and the next step runs on both; and the training direction: norm, rotation,
S^2-Attn and back."""
import random

import pytest
import torch

import shifted_sparse_attention_s2attn_b200 as s2
from serving_utils import (HALF_STEP, attend, cached, check_close, make_cache, no_device_error, norm_rope,
                           norm_rope_grad, random_parents, tree_see, words_of)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s2.clear_device_error()


def test_draft_verify_append_fork():
    B, M, H, Hkv, D, page = 2, 7, 8, 2, 128, 16
    lens = [45, 18]
    kp, vp, table, n = make_cache(lens, 40, page, Hkv, D, BF, 3, fill=float("nan"), spare=6)
    width = table.shape[1]
    d_kp, d_vp, d_table, d_len = kp.cuda(), vp.cuda(), table.cuda(), n.cuda()
    free = sorted(set(range(kp.shape[0])) - set(table[table >= 0].tolist()))
    g = torch.Generator().manual_seed(0)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(BF) for _ in range(2))
    inv, af = s2.rope_inv_freq(D, scaling="yarn", factor=4.0)
    ws = torch.empty(s2.s2attn_tree_decode_workspace_bytes(3, M, H, Hkv, D), dtype=torch.uint8, device="cuda")
    rng = random.Random(2)
    for step in range(3):
        B = d_table.shape[0]
        trees = random_parents(B, M, rng)
        see, depth = tree_see(trees)
        new = [M, 3, 5][:B]
        q, k, v = (torch.randn(B, M, h, D, generator=g).to(BF) for h in (H, Hkv, Hkv))
        mask = torch.empty(B, M, 1, dtype=torch.int64, device="cuda")
        dep = torch.empty(B, M, dtype=torch.int32, device="cuda")
        s2.s2attn_tree_mask(torch.tensor(trees, dtype=torch.int32, device="cuda"), mask, dep)
        pos = d_len[:, None] + dep
        qr, kr = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
        s2.qk_norm_rope_fwd(q.cuda(), k.cuda(), qr, kr, inv.cuda(), wq=wq.cuda(), wk=wk.cuda(), positions=pos,
                            attn_factor=af)
        vn = v.cuda()
        o = torch.zeros(B, M, H, D, dtype=BF, device="cuda")
        lse = torch.zeros(B, H, M, device="cuda")
        d_new = torch.tensor(new, dtype=torch.int32, device="cuda")
        s2.s2attn_tree_decode(qr, kr, vn, d_kp, d_vp, d_table, d_len, o, lse, ws, tree_mask=mask, new_len=d_new)
        no_device_error()
        assert torch.equal(mask.cpu(), words_of(see)) and torch.equal(dep.cpu(), depth)
        for got, x, w in ((qr, q, wq), (kr, k, wk)):
            want, scale = norm_rope(x, w, pos.cpu(), inv, True, 1e-6, af, False)
            check_close(got, want, HALF_STEP[BF] * want.abs() + 64 * 2.0 ** -24 * scale, "norm and rotation")
        wo, wl, bo, bl = attend(qr.cpu(), kr.cpu(), v, d_kp.cpu(), d_vp.cpu(), d_table.cpu(), d_len.cpu(), see, new)
        for b in range(B):
            check_close(o[b, :new[b]], wo[b, :new[b]], bo[b, :new[b]], "o")
            check_close(lse[b, :, :new[b]], wl[b, :, :new[b]], bl[b, :, :new[b]], "lse")
        # accept the path to a random drafted token
        paths = [see[b, rng.randrange(new[b])].nonzero()[:, 0].tolist() for b in range(B)]
        A = max(len(p) for p in paths)
        rows = torch.tensor([p + [0] * (A - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        count = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        s2.s2attn_cache_append(kr, vn, d_kp, d_vp, d_table, d_len, rows=rows, n_rows=count)
        old = d_len.tolist()
        d_len += count
        no_device_error()
        for b, p in enumerate(paths):
            for pool, x in ((d_kp, kr), (d_vp, vn)):
                got = cached(pool, d_table[b], old[b] + len(p), page)[old[b]:]
                assert torch.equal(got, x[b, p])
        if step == 0:       # fork sequence 0: full pages shared, the last one copied, room of its own behind it
            length = int(d_len[0])
            full = length // page
            child = d_table[0].tolist()
            own = -(-(length + 30) // page) - full
            fresh = [free.pop() for _ in range(own)]
            child[full:full + own] = fresh
            s2.s2attn_cache_copy_pages([d_kp, d_vp], [(int(d_table[0, full]), fresh[0])])
            d_table = torch.cat([d_table, torch.tensor([child[:width]], dtype=torch.int32, device="cuda")])
            d_len = torch.cat([d_len, d_len[:1]])
            no_device_error()
            assert torch.equal(cached(d_kp, d_table[2], length, page), cached(d_kp, d_table[0], length, page))


def test_training_step():
    """Norm and rotation before S^2-Attn, and the whole gradient back to q, k and the norm weights."""
    import oracle
    from parity_utils import device_to_bits, rel_l2
    B, N, H, D, G, SH = 1, 512, 4, 128, 256, 2
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(B, N, H, D, generator=g).to(BF) for _ in range(4))
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(BF) for _ in range(2))
    inv, af = s2.rope_inv_freq(D, scaling="linear", factor=8.0)
    pos = torch.arange(N).expand(B, N)
    dev = lambda t: t.cuda()
    qr, kr, o = (torch.empty(B, N, H, D, dtype=BF, device="cuda") for _ in range(3))
    lse = torch.empty(B, H, N, device="cuda")
    s2.qk_norm_rope_fwd(dev(q), dev(k), qr, kr, dev(inv), wq=dev(wq), wk=dev(wk), attn_factor=af)
    s2.s2attn_fwd(qr, kr, dev(v), o, lse, G, SH)
    dqr, dkr, dv = (torch.empty_like(o) for _ in range(3))
    ws = torch.empty(s2.s2attn_bwd_workspace_bytes(B, N, H, D), dtype=torch.uint8, device="cuda")
    s2.s2attn_bwd(qr, kr, dev(v), o, dev(do), lse, dqr, dkr, dv, G, SH, ws)
    g_q, g_k = dqr.cpu(), dkr.cpu()
    dwq, dwk = dev(wq).clone(), dev(wk).clone()
    ws2 = torch.empty(s2.qk_norm_rope_bwd_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    s2.qk_norm_rope_bwd(dev(q), dev(k), dqr, dkr, dqr, dkr, dev(inv), wq=dev(wq), wk=dev(wk), dwq=dwq, dwk=dwk,
                        attn_factor=af, workspace=ws2)
    no_device_error()
    ro, _ = oracle.s2attn_fwd(device_to_bits(qr), device_to_bits(kr), device_to_bits(v), G, SH)
    assert abs(o.float().cpu().numpy() - ro).max() <= 2e-2
    rdq, rdk, _ = oracle.s2attn_bwd(device_to_bits(qr), device_to_bits(kr), device_to_bits(v), device_to_bits(do), G, SH)
    assert rel_l2(g_q.float().numpy(), rdq) <= 2e-2 and rel_l2(g_k.float().numpy(), rdk) <= 2e-2
    u = HALF_STEP[BF]
    for got, dw, x, w, gy in ((dqr, dwq, q, wq, g_q), (dkr, dwk, k, wk, g_k)):
        dx, scale, wdw, wscale = norm_rope_grad(x, w, gy, pos, inv, True, 1e-6, af, False)
        check_close(got, dx, u * dx.abs() + 128 * 2.0 ** -24 * scale, "dx")
        check_close(dw, wdw, u * wdw.abs() + (64 + N * H) * 2.0 ** -24 * wscale, "dw")
