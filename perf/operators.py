"""Measured cases of the operators around a decoding step on a paged key/value cache.

    qk_norm_rope     RMS norm of every q and k head and the rotary embedding in one pass
                     (forward, and forward with backward)
    tree_decode      attention of a tree of drafted tokens over a paged cache
    cache_append     new keys and values written to their pages (all of them, or accepted rows)
    cache_copy       whole pages copied inside the cache's pools (forks, moves)

`run` computes an operator in plain torch operations (own = False) or through the library
(own = True); `exact` computes it in 64 bits from its definition.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ------------------------------------------------------------------------------

def listed():
    return [
        # one new token of each of 16 sequences being decoded, at its own position: latency
        dict(name="norm_rope_token", op="rope", B=16, N=1, Hq=32, Hk=8, D=128, R=128, dtype="bf16",
             interleaved=False, norm=True, bwd=False, scaling="none", factor=1.0, pos0=5000),
        # q and k of a 32k prompt at the 7B layer's heads, positions interpolated from 4096
        dict(name="norm_rope_prompt_32k", op="rope", B=1, N=32768, Hq=32, Hk=32, D=128, R=128, dtype="bf16",
             interleaved=False, norm=True, bwd=False, scaling="linear", factor=8.0, pos0=0),
        # a training step's norm and rotation at 8k with shared key heads, forward and backward
        dict(name="norm_rope_train_8k", op="rope", B=1, N=8192, Hq=32, Hk=8, D=128, R=128, dtype="bf16",
             interleaved=False, norm=True, bwd=True, scaling="yarn", factor=2.0, pos0=0),
        # odd lengths, interleaved pairs over half of a 64-wide head, fp16, forward and backward
        dict(name="norm_rope_train_odd", op="rope", B=3, N=1001, Hq=14, Hk=2, D=64, R=32, dtype="fp16",
             interleaved=True, norm=True, bwd=True, scaling="ntk", factor=4.0, pos0=0),
        # two short chats with a fresh 13-token tree: its mask is built, then attended with
        dict(name="tree_small", op="tree", B=2, M=13, Hq=8, Hk=2, D=64, page=16, dtype="fp16", min_len=37,
             max_len=300, len_seed=1, tree="built", ragged=True),
        # one token of one sequence against a 32k cache at the 7B layer's heads: plain decoding
        dict(name="tree_token_32k", op="tree", B=1, M=1, Hq=32, Hk=32, D=128, page=64, dtype="bf16", min_len=32768,
             max_len=32768, len_seed=1, tree="chain", ragged=False),
        # a serving batch of 16 requests of very different lengths, 32 drafted tokens each at most
        dict(name="tree_batch_16k", op="tree", B=16, M=32, Hq=32, Hk=8, D=128, page=16, dtype="bf16", min_len=100,
             max_len=16384, len_seed=2, tree="mask", ragged=True),
        # the longest context, 100k tokens, 64 drafted tokens and 64 query heads over 8 key heads
        dict(name="tree_100k", op="tree", B=1, M=64, Hq=64, Hk=8, D=128, page=128, dtype="bf16", min_len=102400,
             max_len=102400, len_seed=1, tree="mask", ragged=False),
        # after verification: the accepted rows of each of 32 requests go to their pages: latency
        dict(name="append_accepted", op="append", B=32, M=16, Hk=8, D=128, page=16, dtype="bf16", max_len=4000,
             len_seed=3, picked=True),
        # the keys and values of a 32k prompt go to their pages
        dict(name="append_prompt_32k", op="append", B=1, M=32768, Hk=8, D=128, page=64, dtype="bf16", max_len=0,
             len_seed=1, picked=False),
        # eight sequences are forked: the partly filled last page of each is copied in 16 layers' pools
        dict(name="copy_forks", op="copy", pools=32, pages=64, pairs=8, page=16, Hk=8, D=128, dtype="bf16"),
        # a long cache is moved to other pages (500 pages of 64 tokens in the pools of two layers)
        dict(name="copy_move", op="copy", pools=4, pages=1100, pairs=500, page=64, Hk=8, D=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "append", "copy"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "rope":
        D = rng.choice([64, 80, 128, 128, 256])
        hk = rng.choice([1, 2, 4, 8, 10])
        return dict(op=op, B=_log_int(rng, 1, 16), N=_log_int(rng, 1, 32768), Hq=hk * rng.choice([1, 3, 4, 8]), Hk=hk,
                    D=D, R=rng.choice([16 * rng.randint(1, D // 16), D]), dtype=rng.choice([dtype, dtype, "fp32"]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.75, bwd=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0]),
                    pos0=rng.choice([0, 0, rng.randint(1, 100000)]))
    if op == "tree":
        hk = rng.choice([1, 2, 4, 8, 10])
        max_len = _log_int(rng, 1, 102400)
        return dict(op=op, B=_log_int(rng, 1, 32), M=_log_int(rng, 1, 128), Hq=hk * rng.choice([1, 1, 4, 5, 8]), Hk=hk,
                    D=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128, 256]), dtype=dtype,
                    min_len=rng.choice([0, max_len // 2]), max_len=max_len, len_seed=rng.randint(1, 10 ** 6),
                    tree=rng.choice(["chain", "mask", "built"]), ragged=rng.random() < 0.5)
    if op == "append":
        picked = rng.random() < 0.5
        return dict(op=op, B=_log_int(rng, 1, 32), M=_log_int(rng, 1, 128 if picked else 32768),
                    Hk=rng.choice([1, 2, 8, 10]), D=rng.choice([64, 128]), page=rng.choice([16, 64, 256]), dtype=dtype,
                    max_len=rng.choice([0, rng.randint(1, 8000)]), len_seed=rng.randint(1, 10 ** 6), picked=picked)
    pages = _log_int(rng, 4, 1100)
    return dict(op=op, pools=_log_int(rng, 1, 64), pages=pages, pairs=rng.randint(1, pages // 2),
                page=rng.choice([16, 64]), Hk=rng.choice([1, 8, 10]), D=rng.choice([64, 128]), dtype=dtype)


def _footprint(case):
    """Bytes of the case's largest buffers (the whole pools of a cache)."""
    if case["op"] == "copy":
        return case["pools"] * case["pages"] * case["page"] * case["Hk"] * case["D"] * 2
    if case["op"] == "append":
        return (case["max_len"] + case["M"]) * case["B"] * case["Hk"] * case["D"] * 4
    return 0


def draw(rng):
    """One more case of the listed ones' ranges that costs no more than the largest of its operator."""
    most = {}
    for c in listed():
        w = work(c)
        b, f, s = most.get(c["op"], (0, 0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]), max(s, _footprint(c)))
    while True:
        c = _draw(rng)
        w = work(c)
        b, f, s = most[c["op"]]
        if w["bytes"] <= b and w["flops"] <= f and _footprint(c) <= s:
            return c


# ---- sizes that follow from a case ------------------------------------------------------

def _lens(case):
    """Cached tokens of each sequence: the ends of the range are always met."""
    rng = random.Random(case["len_seed"])
    lo, hi = case.get("min_len", 0), case["max_len"]
    out = [hi] + [int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1
                  for _ in range(case["B"] - 1)]
    return [min(max(x, lo), hi) for x in out]


def _new(case):
    """Drafted tokens of each sequence."""
    rng = random.Random(case["len_seed"] + 1)
    if not case["ragged"]:
        return [case["M"]] * case["B"]
    return [case["M"]] + [rng.randint(0, case["M"]) for _ in range(case["B"] - 1)]


def _accepted(case):
    """Rows that go to the cache, of each sequence (None: all M in order)."""
    if not case["picked"]:
        return None
    rng = random.Random(case["len_seed"] + 2)
    return [sorted(rng.sample(range(case["M"]), rng.randint(0, min(case["M"], 8)))) for _ in range(case["B"])]


def _esize(case):
    return 4 if case["dtype"] == "fp32" else 2


def work(case):
    es = _esize(case)
    if case["op"] == "rope":
        rows = case["B"] * case["N"] * (case["Hq"] + case["Hk"])
        x = rows * case["D"] * es
        passes = 5 if case["bwd"] else 2      # read and write; backward: read x and dy, write dx
        if case["bwd"] and not case["norm"]:
            passes = 4                        # a rotation's backward does not need x
        return {"bytes": passes * x + case["B"] * case["N"] * 4, "flops": (14 if case["bwd"] else 6) * rows * case["D"]}
    if case["op"] == "tree":
        H, Hk, D = case["Hq"], case["Hk"], case["D"]
        nb, fl = 0, 0
        for n, m in zip(_lens(case), _new(case)):
            if m:
                nb += 2 * (n + m) * Hk * D * es + 2 * m * H * D * es + m * H * 4 + -(-n // case["page"]) * 4
                fl += 4 * m * H * D * n + 4 * H * D * m * (m + 1) // 2
        return {"bytes": nb, "flops": fl}
    row = case["Hk"] * case["D"] * es
    if case["op"] == "append":
        acc = _accepted(case)
        n = case["B"] * case["M"] if acc is None else sum(len(a) for a in acc)
        return {"bytes": 4 * n * row, "flops": 0}
    return {"bytes": 2 * case["pools"] * case["pairs"] * case["page"] * row, "flops": 0}


# ---- inputs -----------------------------------------------------------------------------

def _inv_freq(R, scaling, factor, base=10000.0, original=4096):
    """Rotary frequencies of a context stretched by `factor`, and the factor on cos and sin."""
    i = torch.arange(R // 2, dtype=torch.float64)
    if scaling == "ntk" and R > 2:
        base = base * factor ** (R / (R - 2))
    f = base ** (-2.0 * i / R)
    if scaling == "linear":
        return (f / factor).float(), 1.0
    if scaling == "yarn":
        turn = lambda n: R * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), R // 2 - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return (f / factor * ramp + f * (1 - ramp)).float(), 0.1 * math.log(factor) + 1.0
    return f.float(), 1.0


def _parents(case, seed):
    """Trees of drafted tokens: node 0 follows the cache, the others a random earlier node."""
    rng = random.Random(seed * 1000003 + case["len_seed"])
    return [[-1] + [rng.randint(max(0, m - 8), m - 1) for m in range(1, case["M"])] for _ in range(case["B"])]


def _mask_of(parents):
    """[B, M, ceil(M/64)] int64: bit j of row m is set where j is m or one of its ancestors."""
    B, M = len(parents), len(parents[0])
    out = torch.zeros((B, M, -(-M // 64)), dtype=torch.int64)
    for b in range(B):
        sets = []
        for m in range(M):
            sets.append((sets[parents[b][m]] if parents[b][m] >= 0 else 0) | (1 << m))
            for w in range(out.shape[2]):
                x = (sets[m] >> (64 * w)) & ((1 << 64) - 1)
                out[b, m, w] = x - (1 << 64) if x >= 1 << 63 else x
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, dev = _DT[case["dtype"]], "cuda"
    rnd = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.float32).to(dt)
    st = {"case": case}
    if case["op"] == "rope":
        B, N, Hq, Hk, D = (case[x] for x in ("B", "N", "Hq", "Hk", "D"))
        st["q"], st["k"] = rnd(B, N, Hq, D), rnd(B, N, Hk, D)
        f, st["attn_factor"] = _inv_freq(case["R"], case["scaling"], case["factor"])
        st["inv_freq"] = f.to(dev)
        start = torch.randint(0, case["pos0"] + 1, (B, 1), generator=g, device=dev)
        st["positions"] = (start + torch.arange(N, device=dev)).to(torch.int32)
        if case["norm"]:
            st["wq"], st["wk"] = ((1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt) for _ in range(2))
        else:
            st["wq"] = st["wk"] = None
        st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        if case["bwd"]:
            st["dq_out"], st["dk_out"] = rnd(B, N, Hq, D), rnd(B, N, Hk, D)
            st["dq"], st["dk"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
            if case["norm"]:
                st["dwq"], st["dwk"] = torch.empty_like(st["wq"]), torch.empty_like(st["wk"])
            if own:
                import shifted_sparse_attention_s2attn_b200 as s2
                st["workspace"] = torch.empty(s2.qk_norm_rope_bwd_workspace_bytes(D), dtype=torch.uint8, device=dev)
        return st
    if case["op"] == "copy":
        P = case["pages"]
        st["pools"] = [rnd(P, case["page"], case["Hk"], case["D"]) for _ in range(case["pools"])]
        order = random.Random(seed).sample(range(P), 2 * case["pairs"])
        st["pairs"] = list(zip(order[::2], order[1::2]))
        return st
    # a paged cache: the pages of the sequences lie in random order among a few spare ones
    B, M, Hk, D, ps = (case[x] for x in ("B", "M", "Hk", "D", "page"))
    lens = _lens(case)
    grow = M if case["op"] == "append" else 0
    used = [-(-(n + grow) // ps) for n in lens]
    width = max(max(used), 1)
    n_pages = sum(used) + 3
    st["k_pages"], st["v_pages"] = rnd(n_pages, ps, Hk, D), rnd(n_pages, ps, Hk, D)
    ids = random.Random(seed).sample(range(n_pages), sum(used))
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b in range(B):
        table[b, :used[b]] = torch.tensor(ids[sum(used[:b]):sum(used[:b]) + used[b]], dtype=torch.int32)
    st["page_table"] = table.to(dev)
    st["cache_len"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["k_new"], st["v_new"] = rnd(B, M, Hk, D), rnd(B, M, Hk, D)
    st["lens"] = lens
    if case["op"] == "append":
        acc = _accepted(case)
        st["rows"] = st["n_rows"] = None
        if acc is not None:
            A = max(1, max(len(a) for a in acc))
            st["rows"] = torch.tensor([a + [0] * (A - len(a)) for a in acc], dtype=torch.int32, device=dev)
            st["n_rows"] = torch.tensor([len(a) for a in acc], dtype=torch.int32, device=dev)
        st["counts"] = [M] * B if acc is None else [len(a) for a in acc]
        return st
    H = case["Hq"]
    st["q"] = rnd(B, M, H, D)
    st["new"] = _new(case)
    st["new_len"] = torch.tensor(st["new"], dtype=torch.int32, device=dev) if case["ragged"] else None
    st["parents"] = st["mask"] = None
    if case["tree"] != "chain":
        parents = _parents(case, seed)
        if case["tree"] == "built":
            st["parents"] = torch.tensor(parents, dtype=torch.int32, device=dev)
            st["mask"] = torch.zeros((B, M, -(-M // 64)), dtype=torch.int64, device=dev)
            st["depth"] = torch.zeros((B, M), dtype=torch.int32, device=dev)
        else:
            st["mask"] = _mask_of(parents).to(dev)
    st["o"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros((B, H, M), dtype=torch.float32, device=dev)
    if own:
        import shifted_sparse_attention_s2attn_b200 as s2
        st["workspace"] = torch.empty(s2.s2attn_tree_decode_workspace_bytes(B, M, H, Hk, D), dtype=torch.uint8,
                                      device=dev)
    return st


# ---- one pass ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _rope_outputs(s):
    c = s["case"]
    out = [s["q_out"], s["k_out"]]
    if c["bwd"]:
        out += [s["dq"], s["dk"]]
        if c["norm"]:
            out += [s["dwq"], s["dwk"]]
    return out


def _own_rope(s):
    import shifted_sparse_attention_s2attn_b200 as s2
    c = s["case"]
    how = dict(wq=s["wq"], wk=s["wk"], norm=c["norm"], eps=1e-6, positions=s["positions"],
               attn_factor=s["attn_factor"], interleaved=c["interleaved"])
    s2.qk_norm_rope_fwd(s["q"], s["k"], s["q_out"], s["k_out"], s["inv_freq"], **how)
    if c["bwd"]:
        s2.qk_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["dq"], s["dk"], s["inv_freq"],
                            dwq=s.get("dwq"), dwk=s.get("dwk"), workspace=s["workspace"], **how)
    return _rope_outputs(s)


def _own_tree(s):
    import shifted_sparse_attention_s2attn_b200 as s2
    out = [s["o"], s["lse"]]
    if s["parents"] is not None:
        s2.s2attn_tree_mask(s["parents"], s["mask"], s["depth"])
        out += [s["mask"], s["depth"]]
    s2.s2attn_tree_decode(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["page_table"],
                          s["cache_len"], s["o"], s["lse"], s["workspace"], tree_mask=s["mask"],
                          new_len=s["new_len"])
    return out


def _own_append(s):
    import shifted_sparse_attention_s2attn_b200 as s2
    s2.s2attn_cache_append(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["page_table"], s["cache_len"],
                           rows=s["rows"], n_rows=s["n_rows"])
    return [s["k_pages"], s["v_pages"]]


def _own_copy(s):
    import shifted_sparse_attention_s2attn_b200 as s2
    s2.s2attn_cache_copy_pages(s["pools"], s["pairs"])
    return s["pools"]


_OWN = {"rope": _own_rope, "tree": _own_tree, "append": _own_append, "copy": _own_copy}


def _rotate(x, cos, sin, R, interleaved):
    """Pairs of the first R elements turned by the angles of cos, sin [..., 1, R/2]."""
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, x[..., R:]), dim=-1)


def _plain_rope(s):
    c, R = s["case"], s["case"]["R"]
    angle = s["positions"].double()[:, :, None, None] * s["inv_freq"].double()
    cos = (angle.cos() * s["attn_factor"]).float()
    sin = (angle.sin() * s["attn_factor"]).float()
    out, grads, wgrads = [], [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq_out")), (s["k"], s["wk"], s.get("dk_out"))):
        x32 = x.float()
        if c["norm"]:
            rstd = (x32.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
            xhat = x32 * rstd
            y = xhat * w.float()
        else:
            y = x32
        out.append(_rotate(y, cos, sin, R, c["interleaved"]).to(x.dtype))
        if c["bwd"]:
            gr = _rotate(dy.float(), cos, -sin, R, c["interleaved"])
            if c["norm"]:
                gx = gr * w.float()
                dx = rstd * (gx - xhat * (gx * xhat).mean(-1, keepdim=True))
                wgrads.append((gr * xhat).sum((0, 1, 2)).to(x.dtype))
            else:
                dx = gr
            grads.append(dx.to(x.dtype))
    return out + grads + wgrads


def _gather(pages, table_row, n):
    """The first n cached rows of a sequence, [Hk, n, D] in 32 bits."""
    used = -(-n // pages.shape[1])
    return pages[table_row[:used].long()].flatten(0, 1)[:n].permute(1, 0, 2).float()


def _plain_tree(s):
    c = s["case"]
    M, H, Hk, D = c["M"], c["Hq"], c["Hk"], c["D"]
    G = H // Hk
    extra = []
    dev = s["q"].device
    if s["parents"] is not None:
        par = s["parents"].long()
        seen = torch.zeros((c["B"], M, M), dtype=torch.bool, device=dev)
        for m in range(M):
            up = seen.gather(1, par[:, m].clamp(min=0)[:, None, None].expand(-1, 1, M))[:, 0]
            seen[:, m] = up & (par[:, m] >= 0)[:, None]
            seen[:, m, m] = True
        weight = torch.ones(64, dtype=torch.int64, device=dev) << torch.arange(64, device=dev)
        padded = torch.nn.functional.pad(seen.long(), (0, -M % 64)).view(c["B"], M, -1, 64)
        mask = (padded * weight).sum(-1)
        depth = (seen.sum(-1) - 1).to(torch.int32)
        extra = [mask, depth]
    elif s["mask"] is not None:
        bit = torch.arange(M, device=dev)
        seen = ((s["mask"][:, :, bit // 64] >> (bit % 64)) & 1).bool()
    else:
        seen = torch.ones((M, M), dtype=torch.bool, device=dev).tril().expand(c["B"], M, M)
    for b in range(c["B"]):
        n, m = s["lens"][b], s["new"][b]
        if m == 0:
            continue
        q = s["q"][b, :m].float().view(m, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * m, D)
        k = torch.cat((_gather(s["k_pages"], s["page_table"][b], n), s["k_new"][b, :m].permute(1, 0, 2).float()), 1)
        v = torch.cat((_gather(s["v_pages"], s["page_table"][b], n), s["v_new"][b, :m].permute(1, 0, 2).float()), 1)
        score = (q @ k.transpose(1, 2)) * (1.0 / math.sqrt(D))
        score.view(Hk, G, m, n + m)[..., n:].masked_fill_(~seen[b, :m, :m], float("-inf"))
        top = score.amax(-1, keepdim=True)
        p = (score - top).exp_()
        total = p.sum(-1, keepdim=True)
        o = (p @ v) / total
        s["o"][b, :m] = o.view(Hk, G, m, D).permute(2, 0, 1, 3).reshape(m, H, D).to(s["o"].dtype)
        s["lse"][b, :, :m] = (top + total.log()).view(H, m)
    return [s["o"], s["lse"]] + extra


def _plain_append(s):
    ps = s["case"]["page"]
    B, M = s["case"]["B"], s["case"]["M"]
    dev = s["k_new"].device
    if s["rows"] is None:
        src = torch.arange(M, device=dev).expand(B, M)
        live = torch.ones((B, M), dtype=torch.bool, device=dev)
    else:
        src = s["rows"].long()
        live = torch.arange(src.shape[1], device=dev) < s["n_rows"][:, None]
    b, j = live.nonzero(as_tuple=True)
    pos = s["cache_len"].long()[b] + j
    page = s["page_table"].long()[b, pos // ps]
    s["k_pages"][page, pos % ps] = s["k_new"][b, src[b, j]]
    s["v_pages"][page, pos % ps] = s["v_new"][b, src[b, j]]
    return [s["k_pages"], s["v_pages"]]


def _plain_copy(s):
    pairs = torch.tensor(s["pairs"], device=s["pools"][0].device)
    for pool in s["pools"]:
        pool[pairs[:, 1]] = pool[pairs[:, 0]]
    return s["pools"]


_PLAIN = {"rope": _plain_rope, "tree": _plain_tree, "append": _plain_append, "copy": _plain_copy}


# ---- 64-bit definitions -----------------------------------------------------------------

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_rope(case, s):
    """y = R(pos) (w x / rms(x)): each pair is a complex number times attn_factor e^{i pos f};
    the gradients by differentiating that in 64 bits."""
    R, D = case["R"], case["D"]
    turn = torch.polar(torch.tensor(float(s["attn_factor"]), dtype=torch.float64, device="cuda").expand(
        case["B"], case["N"], R // 2), s["positions"].double().unsqueeze(-1) * s["inv_freq"].double()).unsqueeze(2)
    outs, grads, wgrads = [], [], []
    for x, w, dy in (("q", "wq", "dq_out"), ("k", "wk", "dk_out")):
        xd = s[x].double().requires_grad_(case["bwd"])
        wd = None if s[w] is None else s[w].double().requires_grad_(case["bwd"])
        y = xd
        if wd is not None:
            y = xd / torch.sqrt((xd * xd).sum(-1, keepdim=True) / D + 1e-6) * wd
        head, tail = y[..., :R], y[..., R:]
        if case["interleaved"]:
            z = turn * torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous())
            head = torch.view_as_real(z).reshape(head.shape)
        else:
            z = turn * torch.complex(head[..., :R // 2].contiguous(), head[..., R // 2:].contiguous())
            head = torch.cat((z.real, z.imag), -1)
        y = torch.cat((head, tail), -1)
        outs.append(y.detach())
        if case["bwd"]:
            got = torch.autograd.grad(y, [xd] if wd is None else [xd, wd], s[dy].double())
            grads.append(got[0])
            wgrads += list(got[1:])
        del y, z, head, tail, xd
    return outs + grads + wgrads


def _exact_tree(case, s):
    M, H, Hk, D, ps = case["M"], case["Hq"], case["Hk"], case["D"], case["page"]
    B = case["B"]
    o = torch.zeros((B, M, H, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, H, M), dtype=torch.float64, device="cuda")
    table = s["page_table"].tolist()
    if s["parents"] is not None:
        words = _mask_of(s["parents"].tolist())
    elif s["mask"] is not None:
        words = s["mask"].cpu()
    else:
        words = _mask_of([list(range(-1, M - 1))] * B)
    words_list = words.tolist()
    depth = torch.zeros((B, M), dtype=torch.int64)
    for b in range(B):
        n, m = s["lens"][b], s["new"][b]
        see = torch.zeros((M, M), dtype=torch.bool)
        for i in range(M):
            for j in range(M):
                see[i, j] = bool((words_list[b][i][j // 64] >> (j % 64)) & 1)
        depth[b] = see.sum(-1) - 1
        if m == 0:
            continue
        off = torch.where(see[:m, :m], 0.0, -math.inf).cuda().double()
        for h in range(H):
            kh = h // (H // Hk)
            if h % (H // Hk) == 0:
                pieces = [(s["k_pages"][table[b][i], :, kh], s["v_pages"][table[b][i], :, kh])
                          for i in range((n + ps - 1) // ps)]
                kk = torch.cat([p[0] for p in pieces])[:n].double() if n else s["k_new"][b, :0, kh].double()
                vv = torch.cat([p[1] for p in pieces])[:n].double() if n else s["v_new"][b, :0, kh].double()
                kk = torch.cat((kk, s["k_new"][b, :m, kh].double()))
                vv = torch.cat((vv, s["v_new"][b, :m, kh].double()))
            a = torch.einsum("md,nd->mn", s["q"][b, :m, h].double(), kk) / math.sqrt(D)
            a[:, n:] += off
            l = torch.logsumexp(a, -1)
            o[b, :m, h] = torch.exp(a - l[:, None]) @ vv
            lse[b, h, :m] = l
    out = [o, lse]
    if s["parents"] is not None:
        out += [words.cuda(), depth.to(torch.int32).cuda()]
    return out


def _exact_append(case, s):
    """A copy of the rows one sequence at a time; nothing is computed."""
    ps, table = case["page"], s["page_table"].tolist()
    pools = [s["k_pages"].double(), s["v_pages"].double()]
    for b, count in enumerate(s["counts"]):
        src = list(range(case["M"])) if s["rows"] is None else s["rows"][b].tolist()
        j = 0
        while j < count:      # the rows that fall into one page
            pos = s["lens"][b] + j
            n = min(count - j, ps - pos % ps)
            for pool, new in zip(pools, (s["k_new"], s["v_new"])):
                pool[table[b][pos // ps], pos % ps:pos % ps + n] = new[b, torch.tensor(src[j:j + n]).cuda()].double()
            j += n
    return pools


def _exact_copy(case, s):
    out = []
    for pool in s["pools"]:
        y = pool.double()
        for a, b in s["pairs"]:
            y[b] = pool[a].double()
        out.append(y)
    return out


_EXACT = {"rope": _exact_rope, "tree": _exact_tree, "append": _exact_append, "copy": _exact_copy}
