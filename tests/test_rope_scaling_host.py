"""rope_inv_freq by wavelength: every value on the ramp, at short and long original lengths (host only)."""
import math

import pytest

import shifted_sparse_attention_s2attn_b200 as s2


def by_wavelength(R, base, factor, original_len, beta_fast=32.0, beta_slow=1.0):
    index = lambda n: R * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(base))
    lo, hi = max(0, math.floor(index(beta_fast))), min(R - 1, math.ceil(index(beta_slow)))
    out = []
    for i in range(R // 2):
        f = base ** (-2.0 * i / R)
        r = min(1.0, max(0.0, (i - lo) / (hi - lo))) if hi > lo else float(i > lo)
        out.append(f / factor * r + f * (1.0 - r))
    return out


@pytest.mark.parametrize("R,base,factor,original_len", [
    (128, 10000.0, 8.0, 4096), (128, 10000.0, 4.0, 131072), (64, 10000.0, 4.0, 65536), (128, 10000.0, 2.0, 65536),
    (128, 500000.0, 4.0, 131072), (16, 10000.0, 4.0, 1000000), (2, 10000.0, 4.0, 131072), (256, 100.0, 16.0, 32768),
    (128, 10000.0, 4.0, 200), (64, 10000.0, 4.0, 5), (128, 1.5, 4.0, 1 << 30),
])
def test_every_value_of_the_ramp(R, base, factor, original_len):
    """One rounding of the result to fp32 (2^-24); base and factor are exact in fp32, the rest is in 64 bits."""
    got, af = s2.rope_inv_freq(R, base=base, scaling="yarn", factor=factor, original_len=original_len)
    want = by_wavelength(R, base, factor, original_len)
    assert len(got) == R // 2 and abs(af - (0.1 * math.log(factor) + 1)) <= 2.0 ** -23
    for i, (g, w) in enumerate(zip(got.tolist(), want)):
        assert abs(g - w) <= (2.0 ** -24 + 1e-12) * w, (i, g, w)


def test_what_turns_more_than_beta_slow_times_is_never_divided_in_full():
    """The last frequency still turns more than once within a long original length."""
    R, base, factor, L = 128, 10000.0, 4.0, 131072
    got, _ = s2.rope_inv_freq(R, base=base, scaling="yarn", factor=factor, original_len=L)
    f = base ** (-2.0 * (R // 2 - 1) / R)
    assert L * f / (2 * math.pi) > 1.0
    assert got[-1].item() > f / factor * 1.05
