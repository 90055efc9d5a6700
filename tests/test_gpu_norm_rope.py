"""qk_norm_rope_fwd / _bwd against the 64-bit definition.

Bounds: one rounding to the type (half a step of the value), and fp32 roundings relative to
the magnitudes that meet in a sum: the rotation's two products with cos and sin (each off by
up to 2 ulp and 2^-24 of the reduced turn: 4 * 2^-22 together), the norm's sum of D squares
(D/16 lanes of 16: 16 + 4 additions, halved by the root), rsqrtf (2 ulp) and the products by
rstd and w: below 64 * 2^-24 in all; twice that for dx, which has a second sum.  dw adds its
rows one after another in fp32: 2^-24 of the sum of magnitudes a row.
"""
import pytest
import torch

import shifted_sparse_attention_s2attn_b200 as s2
from serving_utils import HALF_STEP, TINY, check_close, no_device_error, norm_rope, norm_rope_grad

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s2.clear_device_error()


def _inputs(B, N, Hq, Hk, D, R, dt, norm, weights, seed=0, pos_max=200000):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g).to(dt)
    x = dict(q=rnd(B, N, Hq, D), k=rnd(B, N, Hk, D), dq_out=rnd(B, N, Hq, D), dk_out=rnd(B, N, Hk, D))
    x["wq"] = (1 + 0.3 * torch.randn(D, generator=g)).to(dt) if norm and weights else None
    x["wk"] = (1 + 0.3 * torch.randn(D, generator=g)).to(dt) if norm and weights else None
    x["positions"] = torch.randint(-5, pos_max, (B, N), generator=g, dtype=torch.int32)
    x["inv_freq"] = s2.rope_inv_freq(R, scaling="linear", factor=2.0)[0] if R else torch.zeros(0)
    return x


def _dev(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def _fwd_check(x, q_out, k_out, norm, eps, af, inter, pos=None):
    pos = x["positions"] if pos is None else pos
    for name, got, src, w in (("q", q_out, x["q"], x["wq"]), ("k", k_out, x["k"], x["wk"])):
        if got is None:
            continue
        want, scale = norm_rope(src, w, pos, x["inv_freq"], norm, eps, af, inter)
        u = HALF_STEP[src.dtype]
        check_close(got, want, u * want.abs() + 64 * 2.0 ** -24 * scale + TINY[src.dtype], name)


SHAPES = [  # B, N, Hq, Hk, D, R
    (1, 1, 1, 1, 16, 16), (1, 1, 32, 8, 128, 128), (2, 3, 5, 1, 64, 32), (3, 37, 7, 7, 80, 48), (1, 130, 4, 2, 256, 256),
    (2, 65, 3, 2, 112, 112), (1, 301, 2, 1, 32, 16), (1, 5, 3, 3, 48, 0), (4, 700, 1, 1, 128, 64), (1, 2, 200, 3, 96, 96),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dt", [BF, FP, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm,weights", [(True, True), (True, False), (False, False)])
def test_forward_and_backward(shape, dt, inter, norm, weights):
    B, N, Hq, Hk, D, R = shape
    x = _inputs(B, N, Hq, Hk, D, R, dt, norm, weights)
    d = _dev(x)
    how = dict(wq=d["wq"], wk=d["wk"], norm=norm, eps=1e-5, positions=d["positions"], attn_factor=1.25, interleaved=inter)
    q_out, k_out = torch.empty_like(d["q"]), torch.empty_like(d["k"])
    s2.qk_norm_rope_fwd(d["q"], d["k"], q_out, k_out, d["inv_freq"], **how)
    no_device_error()
    _fwd_check(x, q_out, k_out, norm, 1e-5, 1.25, inter)

    dq, dk = torch.empty_like(d["q"]), torch.empty_like(d["k"])
    dwq = torch.empty(D, dtype=dt, device="cuda") if weights else None
    dwk = torch.empty(D, dtype=dt, device="cuda") if weights else None
    ws = torch.empty(s2.qk_norm_rope_bwd_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    s2.qk_norm_rope_bwd(d["q"], d["k"], d["dq_out"], d["dk_out"], dq, dk, d["inv_freq"], dwq=dwq, dwk=dwk, workspace=ws,
                        **how)
    no_device_error()
    u = HALF_STEP[dt]
    for name, got, src, w, dy, dw in (("q", dq, x["q"], x["wq"], x["dq_out"], dwq),
                                      ("k", dk, x["k"], x["wk"], x["dk_out"], dwk)):
        want, scale, wdw, wscale = norm_rope_grad(src, w, dy, x["positions"], x["inv_freq"], norm, 1e-5, 1.25, inter)
        check_close(got, want, u * want.abs() + 128 * 2.0 ** -24 * scale + TINY[dt], "d" + name)
        if dw is not None:
            rows = B * N * src.shape[2]
            check_close(dw, wdw, u * wdw.abs() + (64 + rows) * 2.0 ** -24 * wscale + TINY[dt], "dw" + name)


def test_gradient_against_differences():
    """Central differences of the 64-bit definition: the analytic oracle that the kernel is held to."""
    x = _inputs(1, 3, 2, 1, 32, 16, F32, True, True)
    args = (x["positions"], x["inv_freq"], True, 1e-5, 1.1, True)
    dx, _, dw, _ = norm_rope_grad(x["q"], x["wq"], x["dq_out"], *args)
    f = lambda q, w: (norm_rope(q, w, *args)[0] * x["dq_out"].double()).sum()
    h = 1e-5
    q, w = x["q"].double(), x["wq"].double()
    for i in [(0, 0, 0, 0), (0, 1, 1, 17), (0, 2, 0, 31), (0, 0, 1, 8)]:
        e = torch.zeros_like(q)
        e[i] = h
        assert abs(((f(q + e, w) - f(q - e, w)) / (2 * h) - dx[i]).item()) < 1e-7
    for j in (0, 7, 31):
        e = torch.zeros_like(w)
        e[j] = h
        assert abs(((f(q, w + e) - f(q, w - e)) / (2 * h) - dw[j]).item()) < 1e-7


@pytest.mark.parametrize("pos0", [0, 131072, 2 ** 31 - 60, -9])
def test_consecutive_positions(pos0):
    x = _inputs(2, 50, 3, 2, 64, 64, F32, True, True)
    d = _dev(x)
    q_out, k_out = torch.empty_like(d["q"]), torch.empty_like(d["k"])
    s2.qk_norm_rope_fwd(d["q"], d["k"], q_out, k_out, d["inv_freq"], wq=d["wq"], wk=d["wk"], pos0=pos0)
    no_device_error()
    # a turn of 2^31 / 2 pi is off by up to 2^-53 * 2 of itself in 64 bits, which the oracle shares
    pos = (pos0 + torch.arange(50)).expand(2, 50)
    _fwd_check(x, q_out, k_out, True, 1e-6, 1.0, False, pos=pos)


def test_one_side_only_and_in_place():
    x = _inputs(2, 9, 4, 2, 128, 128, BF, True, True)
    d = _dev(x)
    q_out, k_out = torch.empty_like(d["q"]), torch.empty_like(d["k"])
    how = dict(positions=d["positions"], eps=1e-6)
    s2.qk_norm_rope_fwd(d["q"], d["k"], q_out, k_out, d["inv_freq"], wq=d["wq"], wk=d["wk"], **how)
    only_q, only_k = torch.empty_like(q_out), torch.empty_like(k_out)
    s2.qk_norm_rope_fwd(d["q"], None, only_q, None, d["inv_freq"], wq=d["wq"], **how)
    s2.qk_norm_rope_fwd(None, d["k"], None, only_k, d["inv_freq"], wk=d["wk"], **how)
    assert torch.equal(only_q, q_out) and torch.equal(only_k, k_out)
    s2.qk_norm_rope_fwd(d["q"], d["k"], d["q"], d["k"], d["inv_freq"], wq=d["wq"], wk=d["wk"], **how)
    assert torch.equal(d["q"], q_out) and torch.equal(d["k"], k_out)
    no_device_error()


def test_backward_one_side_in_place_and_deterministic():
    x = _inputs(1, 600, 8, 2, 128, 64, BF, True, True)
    d = _dev(x)
    ws = torch.empty(s2.qk_norm_rope_bwd_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    how = dict(positions=d["positions"], workspace=ws)

    def both():
        out = [torch.empty_like(d[n]) for n in ("q", "k", "wq", "wk")]
        s2.qk_norm_rope_bwd(d["q"], d["k"], d["dq_out"], d["dk_out"], out[0], out[1], d["inv_freq"], wq=d["wq"],
                            wk=d["wk"], dwq=out[2], dwk=out[3], **how)
        return out
    a, b = both(), both()
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    dk = torch.empty_like(d["k"])
    s2.qk_norm_rope_bwd(None, d["k"], None, d["dk_out"], None, dk, d["inv_freq"], wk=d["wk"], positions=d["positions"])
    assert torch.equal(dk, a[1])
    g = d["dq_out"].clone()
    s2.qk_norm_rope_bwd(d["q"], None, g, None, g, None, d["inv_freq"], wq=d["wq"], positions=d["positions"])
    assert torch.equal(g, a[0])
    no_device_error()


def test_rows_of_zeros_and_infinities_stay_in_their_row():
    x = _inputs(1, 6, 2, 1, 64, 64, F32, True, False)
    x["q"][0, 1] = 0.0
    x["q"][0, 2, 0, 5] = float("inf")
    x["q"][0, 3, 1, 9] = float("nan")
    d = _dev(x)
    q_out = torch.empty_like(d["q"])
    s2.qk_norm_rope_fwd(d["q"], None, q_out, None, d["inv_freq"], positions=d["positions"], eps=1e-6)
    no_device_error()
    assert (q_out[0, 1] == 0).all()
    assert q_out[0, 3, 1].isnan().all() and q_out[0, 2, 0].isnan().any()
    clean = torch.ones(6, 2, dtype=torch.bool)
    clean[2, 0] = clean[3, 1] = False
    assert q_out[0][clean.cuda()].isfinite().all()


def test_matches_rope_pi_on_the_half_layout():
    """Without the norm and with interpolated positions this is rope_pi_apply's rotation; that one
    rounds t * pos_scale and the angle to fp32 (angles up to 4096: off by 2^-24 * 4096 * 2)."""
    N = 4096
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, N, 2, 128, generator=g).bfloat16().cuda()
    f, af = s2.rope_inv_freq(128, scaling="linear", factor=4.0)
    out = torch.empty_like(q)
    s2.qk_norm_rope_fwd(q, None, out, None, f.cuda(), norm=False, attn_factor=af)
    pi = q.clone()
    s2.rope_pi_apply(pi, None, 0.25)
    torch.cuda.synchronize()
    bound = 2 * 2.0 ** -8 * out.double().abs() + 2.0 ** -11 * 16
    assert ((out.double() - pi.double()).abs() <= bound).all()


def test_captured_on_a_stream_and_replayed():
    x = _inputs(2, 40, 4, 2, 128, 128, BF, True, True)
    d = _dev(x)
    q_out, k_out = torch.empty_like(d["q"]), torch.empty_like(d["k"])
    want = torch.empty_like(q_out), torch.empty_like(k_out)
    how = dict(wq=d["wq"], wk=d["wk"], positions=d["positions"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        s2.qk_norm_rope_fwd(d["q"], d["k"], q_out, k_out, d["inv_freq"], **how)
    d["q"].normal_()
    d["positions"].add_(17)
    g.replay()
    s2.qk_norm_rope_fwd(d["q"], d["k"], *want, d["inv_freq"], **how)
    no_device_error()
    assert torch.equal(q_out, want[0]) and torch.equal(k_out, want[1])


def test_more_than_two_to_the_31_elements():
    """The last rows of a tensor of more than 2^31 elements, forward and backward."""
    N, H, D = 132000, 128, 128
    assert N * H * D > 2 ** 31
    q = torch.zeros(1, N, H, D, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(0)
    tail = torch.randn(1, 3, H, D, generator=g).to(BF)
    q[:, -3:] = tail.cuda()
    f = s2.rope_inv_freq(D)[0]
    out = torch.empty_like(q)
    s2.qk_norm_rope_fwd(q, None, out, None, f.cuda())
    no_device_error()
    pos = torch.arange(N - 3, N)[None]
    want, scale = norm_rope(tail, None, pos, f, True, 1e-6, 1.0, False)
    check_close(out[:, -3:], want, HALF_STEP[BF] * want.abs() + 64 * 2.0 ** -24 * scale, "q")
    s2.qk_norm_rope_bwd(q, None, q, None, out, None, f.cuda())
    no_device_error()
    want, scale, _, _ = norm_rope_grad(tail, None, tail, pos, f, True, 1e-6, 1.0, False)
    check_close(out[:, -3:], want, HALF_STEP[BF] * want.abs() + 128 * 2.0 ** -24 * scale, "dq")


def test_heads_at_the_limit():
    """16384 heads (the division of a row by H is exact there) beside one."""
    x = _inputs(1, 9, 16384, 1, 16, 16, F32, True, True)
    d = _dev(x)
    q_out, k_out = torch.empty_like(d["q"]), torch.empty_like(d["k"])
    s2.qk_norm_rope_fwd(d["q"], d["k"], q_out, k_out, d["inv_freq"], wq=d["wq"], wk=d["wk"], positions=d["positions"],
                        eps=1e-5)
    no_device_error()
    _fwd_check(x, q_out, k_out, True, 1e-5, 1.0, False)
