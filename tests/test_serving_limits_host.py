"""The size limits that the header states, from both sides (no GPU: what is within them fails on the missing
workspace, which is checked behind the sizes, or on a bad pointer)."""
import pytest

import shifted_sparse_attention_s2attn_b200 as s2

P = 0x10000      # an aligned fake device address: these calls fail before any launch
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from shifted_sparse_attention_s2attn_b200 import _build
    _build.build()
    return s2.capi()


@pytest.mark.parametrize("B,width,page,rc", [
    # B * (width * page / 64 + 16) < 2^30
    (2, 2 ** 31 - 65, 16, WORKSPACE), (2, 2 ** 31 - 64, 16, UNSUPPORTED),
    (4, 2 ** 28 - 17, 64, WORKSPACE), (4, 2 ** 28 - 16, 64, UNSUPPORTED),
    (1024, 2 ** 18 - 5, 256, WORKSPACE), (1024, 2 ** 18 - 4, 256, UNSUPPORTED),
    (1, 2 ** 31 - 1, 16, WORKSPACE),
])
def test_tree_decode_table_limit(lib, B, width, page, rc):
    assert lib.s2attn_tree_decode(*[P] * 7, None, None, P, P, B, 1, 1, 1, 64, 4, page, width, 0, None, 0, None) == rc


@pytest.mark.parametrize("B,M,H,rc", [(1024, 128, 2 ** 14 - 1, WORKSPACE), (1024, 128, 2 ** 14, UNSUPPORTED)])
def test_tree_decode_rows_limit(lib, B, M, H, rc):
    """B * M * H < 2^31."""
    assert lib.s2attn_tree_decode(*[P] * 7, None, None, P, P, B, M, H, H, 64, 4, 16, 4, 0, None, 0, None) == rc


@pytest.mark.parametrize("n_pages,page,rc", [(2 ** 27 - 16, 16, WORKSPACE), (2 ** 27 - 15, 16, UNSUPPORTED),
                                             (2 ** 23 - 1, 256, WORKSPACE), (2 ** 23, 256, UNSUPPORTED)])
def test_pool_limit(lib, n_pages, page, rc):
    """n_pages * page_size <= 2^31 - 256."""
    assert lib.s2attn_tree_decode(*[P] * 7, None, None, P, P, 1, 1, 1, 1, 64, n_pages, page, 4, 0, None, 0, None) == rc


@pytest.mark.parametrize("B,M,A,Hkv,D,es,rc", [
    (1, 2 ** 30 - 1, 4, 1, 64, 2, INVALID), (1, 2 ** 30, 4, 1, 64, 2, UNSUPPORTED),          # B * M < 2^30
    (2, 4, 2 ** 29 - 1, 1, 64, 2, INVALID), (2, 4, 2 ** 29, 1, 64, 2, UNSUPPORTED),          # B * A < 2^30
    (1, 4, 4, 2 ** 11, 128, 4, INVALID), (1, 4, 4, 2 ** 11 + 1, 128, 4, UNSUPPORTED),        # a row of 2^20 bytes
])
def test_append_limits(lib, B, M, A, Hkv, D, es, rc):
    """Within the limits the misaligned rows are what is refused."""
    assert lib.s2attn_cache_append(P, P, P, P, P, P, P + 2, None, B, M, A, Hkv, D, 4, 16, 4, es, None) == rc


@pytest.mark.parametrize("page_bytes,rc", [(2 ** 40, INVALID), (2 ** 40 + 16, UNSUPPORTED)])
def test_copy_limit(lib, page_bytes, rc):
    import ctypes
    pools = (ctypes.c_void_p * 1)(P + 8)       # misaligned
    assert lib.s2attn_cache_copy_pages(pools, 1, (ctypes.c_int * 2)(0, 1), 1, 2, page_bytes, None) == rc


def test_binding_refuses_every_size_past_32_bits():
    """The C calls' sizes are 32-bit: one of 2^32 + x must not reach them as x.  Tensors without memory."""
    import torch

    def big(*shape, dtype=torch.bfloat16):
        if max(shape) < 2 ** 31:
            return torch.zeros(shape, dtype=dtype)
        return torch.zeros(1, dtype=dtype).expand(*shape)
    W = 2 ** 32 + 16
    f, i32 = torch.zeros(8), torch.int32
    calls = [
        lambda: s2.qk_norm_rope_fwd(big(1, 1, W, 16), None, big(1, 1, W, 16), None, f),
        lambda: s2.qk_norm_rope_fwd(None, big(1, 1, 4, W), None, big(1, 1, 4, W), f),
        lambda: s2.qk_norm_rope_fwd(big(1, 1, 4, 16), big(1, 1, W, 16), big(1, 1, 4, 16), big(1, 1, W, 16), f),
        lambda: s2.qk_norm_rope_bwd(None, None, big(1, 1, W, 16), None, big(1, 1, W, 16), None, f, norm=False),
        lambda: s2.s2attn_tree_mask(big(W, 1, dtype=i32), big(W, 1, 1, dtype=torch.int64)),
        lambda: s2.s2attn_tree_decode(big(W, 1, 1, 64), big(W, 1, 1, 64), big(W, 1, 1, 64), big(2, 16, 1, 64),
                                      big(2, 16, 1, 64), big(W, 1, dtype=i32), big(W, dtype=i32), big(W, 1, 1, 64),
                                      big(W, 1, 1, dtype=torch.float32), torch.zeros(1)),
        lambda: s2.s2attn_tree_decode(big(1, 1, W, 64), big(1, 1, W, 64), big(1, 1, W, 64), big(2, 16, W, 64),
                                      big(2, 16, W, 64), big(1, 1, dtype=i32), big(1, dtype=i32), big(1, 1, W, 64),
                                      big(1, W, 1, dtype=torch.float32), torch.zeros(1)),
        lambda: s2.s2attn_cache_append(big(1, 2, 1, W), big(1, 2, 1, W), big(2, 16, 1, W), big(2, 16, 1, W),
                                       big(1, 1, dtype=i32), big(1, dtype=i32)),
        lambda: s2.s2attn_cache_append(big(1, 2, W, 16), big(1, 2, W, 16), big(2, 16, W, 16), big(2, 16, W, 16),
                                       big(1, 1, dtype=i32), big(1, dtype=i32)),
        lambda: s2.s2attn_cache_append(big(1, 2, 1, 16), big(1, 2, 1, 16), big(2, 16, 1, 16), big(2, 16, 1, 16),
                                       big(1, 1, dtype=i32), big(1, dtype=i32), rows=big(1, W, dtype=i32)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError) as e:
            call()
        assert "2^3" in str(e.value), i
