"""s2attn_cache_append: a length that is out of range writes nothing, near zero too."""
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


@pytest.mark.parametrize("length", [-1, -3, -16, -2 ** 31])
def test_append_at_a_negative_length_writes_nothing(length):
    """Rows behind position -1 would land in the sequence's first page, which forks share."""
    kp, vp, table, n = make_cache([20, 20], 40, 16, 2, 64, torch.bfloat16, 1, fill=0.5)
    table[1, 0] = table[0, 0]
    n[1] = length
    new = torch.randn(2, 17, 2, 64).bfloat16()
    dk, dv = kp.cuda(), vp.cuda()
    counts = torch.tensor([0, 17], dtype=torch.int32).cuda()
    s2.s2attn_cache_append(new.cuda(), new.cuda(), dk, dv, table.cuda(), n.cuda(), n_rows=counts)
    torch.cuda.synchronize()
    assert s2.get_device_error() == (-6, 0x740)
    s2.clear_device_error()
    assert torch.equal(dk.cpu(), kp) and torch.equal(dv.cpu(), vp)
    no_device_error()
