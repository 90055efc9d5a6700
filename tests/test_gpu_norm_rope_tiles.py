"""qk_norm_rope_fwd / _bwd where a CTA holds several tokens' angles at a time, and refills them.

Bounds as in test_gpu_norm_rope; dw by the number of fp32 additions one of its terms passes: a thread's
rows one after another, the CTA's threads, then the CTAs' partials in 32 slices and the slices."""
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


def _near(got, want, bound, name):
    """check_close on the device."""
    bad = ~((got.double() - want).abs() <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; at {i}: {got[i]} for {want[i]}")


@pytest.mark.parametrize("H,tokens", [(16383, 7104), (16384, 7104), (16381, 5000), (7919, 9001), (200, 60000)])
def test_every_token_of_a_tile_turns_by_its_own_angle(H, tokens):
    """16 tokens of 16383 heads are the most that a tile takes: the row's token is row / H there."""
    D = R = 16
    g = torch.Generator(device="cuda").manual_seed(H)
    q = torch.randn(1, tokens, H, D, generator=g, device="cuda", dtype=BF)
    f = s2.rope_inv_freq(R, base=100.0)[0].cuda()
    pos = torch.randint(0, 100000, (1, tokens), generator=g, device="cuda", dtype=torch.int32)
    out = torch.empty_like(q)
    u = HALF_STEP[BF]
    s2.qk_norm_rope_fwd(q, None, out, None, f, positions=pos, eps=1e-5)
    no_device_error()
    for t in range(0, tokens, 200):
        want, scale = norm_rope(q[:, t:t + 200], None, pos[:, t:t + 200], f, True, 1e-5, 1.0, False)
        _near(out[:, t:t + 200], want, u * want.abs() + 64 * 2.0 ** -24 * scale, f"tokens from {t}")
    s2.qk_norm_rope_bwd(q, None, q, None, out, None, f, positions=pos, eps=1e-5)
    no_device_error()
    for t in range(0, tokens, 200):
        x = q[:, t:t + 200]
        want, scale, _, _ = norm_rope_grad(x, None, x, pos[:, t:t + 200], f, True, 1e-5, 1.0, False)
        _near(out[:, t:t + 200], want, u * want.abs() + 128 * 2.0 ** -24 * scale, f"gradient of tokens from {t}")


@pytest.mark.parametrize("B,N,Hq,Hk,D,R,dt,inter", [
    (1, 60000, 2, 1, 64, 64, F32, False),      # a side's CTA: about 200 tokens, its tile 64
    (3, 20001, 3, 2, 128, 128, BF, True),      # tiles of 32
    (2, 9000, 4, 4, 256, 256, FP, False),      # tiles of 16
    (1, 50001, 1, 5, 80, 32, BF, False),       # tiles of 128
])
def test_backward_with_weights_over_several_tiles(B, N, Hq, Hk, D, R, dt, inter):
    g = torch.Generator(device="cuda").manual_seed(N)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
    x = dict(q=rnd(B, N, Hq, D), k=rnd(B, N, Hk, D))
    dy = dict(q=rnd(B, N, Hq, D), k=rnd(B, N, Hk, D))
    w = dict(q=1 + 0.3 * rnd(D), k=1 + 0.3 * rnd(D))
    pos = torch.randint(0, 200000, (B, N), generator=g, device="cuda", dtype=torch.int32)
    f = s2.rope_inv_freq(R, scaling="linear", factor=2.0)[0].cuda()
    dx, dw = {n: torch.empty_like(t) for n, t in x.items()}, {n: torch.empty_like(t) for n, t in w.items()}
    out = {n: torch.empty_like(t) for n, t in x.items()}
    ws = torch.empty(s2.qk_norm_rope_bwd_workspace_bytes(D), dtype=torch.uint8, device="cuda").fill_(0xff)
    how = dict(wq=w["q"], wk=w["k"], positions=pos, eps=1e-5, attn_factor=1.25, interleaved=inter)
    s2.qk_norm_rope_fwd(x["q"], x["k"], out["q"], out["k"], f, **how)
    s2.qk_norm_rope_bwd(x["q"], x["k"], dy["q"], dy["k"], dx["q"], dx["k"], f, dwq=dw["q"], dwk=dw["k"], workspace=ws,
                        **how)
    no_device_error()
    u = HALF_STEP[dt]
    for n in ("q", "k"):
        want, scale = norm_rope(x[n], w[n], pos, f, True, 1e-5, 1.25, inter)
        _near(out[n], want, u * want.abs() + 64 * 2.0 ** -24 * scale + TINY[dt], n)
        want, scale, wdw, wscale = norm_rope_grad(x[n], w[n], dy[n], pos, f, True, 1e-5, 1.25, inter)
        _near(dx[n], want, u * want.abs() + 128 * 2.0 ** -24 * scale + TINY[dt], "d" + n)
        lanes = 4 if D <= 64 else 8 if D <= 128 else 16
        rows = 256 // lanes
        # at least 40 CTAs take a side (its share of 296), 296 at most
        adds = -(-B * N // 40) * x[n].shape[2] // rows + 1 + rows + 296 // 32 + 1 + 32
        check_close(dw[n], wdw.cpu(), (u * wdw.abs() + (64 + adds) * 2.0 ** -24 * wscale + TINY[dt]).cpu(), "dw" + n)
