"""64-bit definitions (torch on the CPU) of the rotary norm and of attention over a paged cache, and
helpers that lay out a paged cache; shared by the GPU tests of those calls."""
import math
import random

import torch

import shifted_sparse_attention_s2attn_b200 as s2

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}   # half of fp16's smallest step


def no_device_error():
    torch.cuda.synchronize()
    rc, detail = s2.get_device_error()
    assert rc == 0, f"device error word set: {detail:#x}"


# ---- rotary norm ------------------------------------------------------------------------

def cos_sin(pos, inv_freq, af):
    angle = pos.double()[..., None] * inv_freq.double()
    return angle.cos()[:, :, None] * af, angle.sin()[:, :, None] * af


def rotate(x, c, s, R, interleaved):
    y = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def partner(x, R, interleaved):
    """|x| of an element plus |x| of the other element of its pair."""
    m = x.abs()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y = m.clone()
    y[..., a] = y[..., b] = m[..., a] + m[..., b]
    return y


def norm_rope(x, w, pos, inv_freq, norm, eps, af, interleaved):
    """(y, scale): the result in 64 bits and the magnitude its fp32 roundings are relative to."""
    R = 2 * inv_freq.numel()
    x = x.double()
    if norm:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
        if w is not None:
            x = x * w.double()
    c, s = cos_sin(pos, inv_freq, af)
    return rotate(x, c, s, R, interleaved), partner(x, R, interleaved) * max(1.0, abs(af))


def norm_rope_grad(x, w, dy, pos, inv_freq, norm, eps, af, interleaved):
    """(dx, scale of dx, dw, scale of dw) in 64 bits, from the formula."""
    R, D = 2 * inv_freq.numel(), dy.shape[-1]
    c, s = cos_sin(pos, inv_freq, af)
    g = rotate(dy.double(), c, -s, R, interleaved)
    gs = partner(dy.double(), R, interleaved) * max(1.0, abs(af))
    if not norm:
        return g, gs, None, None
    x = x.double()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    xhat = x * r
    wd = torch.ones(D, dtype=torch.float64, device=dy.device) if w is None else w.double()
    gx = g * wd
    dx = r * (gx - xhat * (gx * xhat).mean(-1, keepdim=True))
    scale = r * (gs * wd.abs() + xhat.abs() * (gs * wd.abs() * xhat.abs()).mean(-1, keepdim=True))
    return dx, scale, (g * xhat).sum((0, 1, 2)), (gs * xhat.abs()).sum((0, 1, 2))


# ---- attention over a paged cache -------------------------------------------------------

def words_of(see):
    """[B, M, M] bool -> [B, M, ceil(M/64)] int64."""
    B, M, _ = see.shape
    out = torch.zeros(B, M, (M + 63) // 64, dtype=torch.int64)
    for j in range(M):
        bit = 1 << (j % 64)
        bit = bit - (1 << 64) if bit >= 1 << 63 else bit
        out[:, :, j // 64] |= see[:, :, j].long() * bit
    return out


def tree_see(parents):
    """[B][M] parents -> [B, M, M] bool, and depths [B, M]."""
    B, M = len(parents), len(parents[0])
    see = torch.zeros(B, M, M, dtype=torch.bool)
    for b in range(B):
        for m in range(M):
            a = m
            while a >= 0:
                see[b, m, a] = True
                a = parents[b][a]
    return see, see.sum(-1).to(torch.int32) - 1


def random_parents(B, M, rng):
    return [[-1] + [rng.choice([-1, m - 1, rng.randint(0, m - 1)]) for m in range(1, M)] for _ in range(B)]


def make_cache(lens, room, page, Hkv, D, dtype, seed, fill=float("nan"), spare=2):
    """A pool whose pages hold `lens` tokens (and have room for `room` more), in random page order;
    rows behind a sequence's last token, and spare pages, hold `fill`.  CPU tensors."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-(n + room) // page) for n in lens]
    width = max(1, max(used))
    n_pages = sum(used) + spare
    order = random.Random(seed).sample(range(n_pages), sum(used))
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    pools = []
    for _ in range(2):
        pool = torch.full((n_pages, page, Hkv, D), fill, dtype=torch.float32)
        at = 0
        for b, n in enumerate(lens):
            ids = order[at:at + used[b]]
            at += used[b]
            table[b, :used[b]] = torch.tensor(ids, dtype=torch.int32)
            for i, pg in enumerate(ids):
                rows = max(0, min(page, n - i * page))
                pool[pg, :rows] = torch.randn(rows, Hkv, D, generator=g)
        pools.append(pool.to(dtype))
    return pools[0], pools[1], table, torch.tensor(lens, dtype=torch.int32)


def cached(pool, table_row, n, page):
    """The n cached rows of a sequence, [n, Hkv, D]."""
    ids = table_row[:-(-n // page)].long()
    return pool[ids].flatten(0, 1)[:n]


def attend(q, k_new, v_new, k_pages, v_pages, table, lens, see, new):
    """o [B,M,H,D], lse [B,H,M] in 64 bits and bounds on what the kernel may be off by; rows from
    new[b] on are None-like zeros.

    Bound of o: P and o are each rounded by half a step u, so u |o| + u sum p |v|, where fp16's
    smallest step adds half of it per key (P's largest element is at least 1, the sum too);
    scores are sums of D products in fp32, each partial sum off by 2^-23 of at most sum |q k|
    (D additions), and an error e of a score scales p by 1 + e, twice in the quotient; exp2 and
    the sums in fp32 add 2^-18.
    """
    B, M, H, D = q.shape
    Hkv, page = k_new.shape[2], k_pages.shape[1]
    u, tiny = HALF_STEP[q.dtype], TINY[q.dtype]
    o = torch.zeros(B, M, H, D, dtype=torch.float64)
    bo = torch.zeros_like(o)
    lse = torch.full((B, H, M), -math.inf, dtype=torch.float64)
    bl = torch.zeros_like(lse)
    for b in range(B):
        n, m = int(lens[b]), int(new[b])
        if m == 0:
            continue
        kk = torch.cat([cached(k_pages, table[b], n, page), k_new[b, :m]]).double()
        vv = torch.cat([cached(v_pages, table[b], n, page), v_new[b, :m]]).double()
        vis = torch.cat([torch.ones(m, n, dtype=torch.bool), see[b, :m, :m]], 1)
        for h in range(H):
            k, v = kk[:, h * Hkv // H], vv[:, h * Hkv // H]
            for i in range(m):
                keys = vis[i]
                if not keys.any():
                    continue
                s = (k[keys] @ q[b, i, h].double()) / math.sqrt(D)
                mag = (k[keys].abs() @ q[b, i, h].double().abs()).max() / math.sqrt(D)
                top = s.max()
                p = torch.exp(s - top)
                o[b, i, h] = (p @ v[keys]) / p.sum()
                lse[b, h, i] = top + p.sum().log()
                e = D * 2.0 ** -23 * mag + 2.0 ** -18
                pv = (p @ v[keys].abs()) / p.sum()
                bo[b, i, h] = (u * o[b, i, h].abs() + (u + 2 * e) * pv + tiny * (1 + v[keys].abs().sum(0))) * 1.02
                bl[b, h, i] = e + 2.0 ** -18 * (1 + lse[b, h, i].abs())
    return o, lse, bo, bl


def check_close(got, want, bound, name):
    got = got.double().cpu()
    same = (got == want) | (got.isnan() & want.isnan())      # infinities and NaN
    bad = ~(same | ((got - want).abs() <= bound))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; at {i}: {got[i]} for {want[i]}, "
                             f"bound {bound[i]}")
