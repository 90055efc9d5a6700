"""The runs that s2attn_tree_decode notes in its workspace are those of serving_runs."""
import random

import pytest
import torch

import shifted_sparse_attention_s2attn_b200 as s2
from serving_runs import plan, segments
from serving_utils import no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s2.clear_device_error()


def _cases():
    rng = random.Random(9)
    out = [([0], [1], 1, 1, 1), ([32768], [1], 1, 32, 32), ([1] * 50, [1] * 50, 1, 1, 1),
           ([i % 130 for i in range(1024)], [i % 2 for i in range(1024)], 1, 2, 1), ([5000, 0, 0, 64], [40, 0, 40, 7], 40, 8, 1),
           ([100] * 9, [128] * 9, 128, 4, 2)]
    for _ in range(30):
        B, M = rng.choice([1, 2, 7, 33, 40, 300]), rng.choice([1, 2, 13, 65, 128])
        Hkv = rng.choice([1, 2, 8])
        lens = [rng.choice([0, 1, 63, 64, 65, rng.randint(0, 3000)]) for _ in range(B)]
        out.append((lens, [rng.choice([0, 1, M, rng.randint(0, M)]) for _ in range(B)], M, Hkv * rng.choice([1, 2, 5]), Hkv))
    return out


@pytest.mark.parametrize("lens,new,M,H,Hkv", _cases())
def test_first_and_last_run_of_every_sequence(lens, new, M, H, Hkv):
    B, D, page = len(lens), 64, 64
    tok, row_tiles, J, _ = plan(M, H, Hkv)
    width = max(1, -(-max(lens) // page))
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = torch.empty(s2.s2attn_tree_decode_workspace_bytes(B, M, H, Hkv, D), dtype=torch.uint8, device="cuda").fill_(0xff)
    s2.s2attn_tree_decode(z(B, M, H, D), z(B, M, Hkv, D), z(B, M, Hkv, D), z(2, page, Hkv, D), z(2, page, Hkv, D),
                          torch.zeros(B, width, dtype=torch.int32, device="cuda"), i32(lens), z(B, M, H, D),
                          torch.zeros(B, H, M, device="cuda"), ws, new_len=i32(new))
    no_device_error()
    noted = ws[-(-(-B * row_tiles * 8 // 256) * 256):][:B * row_tiles * 8].view(torch.int32).view(B, row_tiles, 2).tolist()
    for rt in range(row_tiles):
        segs, tiles = segments(lens, new, rt * tok, J)
        want = [[-1, -1] for _ in lens]
        for j, b, t0, n, total in segs:
            if t0 == 0:
                want[b][0] = j
            if t0 + n == total:
                want[b][1] = j
        assert [row[rt] for row in noted] == want


def test_lengths_that_change_while_calls_run_leave_the_next_call_right():
    """Every block takes its run and its keys from one reading of the lengths: a call whose lengths another
    stream changes may mix their results, but ends, and the next call is as ever."""
    B, M, H, D, page = 40, 3, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    rng = random.Random(1)
    lens = [torch.tensor([rng.randint(0, 2000) for _ in range(B)], dtype=torch.int32, device="cuda") for _ in range(2)]
    news = [torch.tensor([rng.randint(0, M) for _ in range(B)], dtype=torch.int32, device="cuda") for _ in range(2)]
    kp, vp = rnd(200, page, 1, D), rnd(200, page, 1, D)
    table = torch.randint(0, 200, (B, 125), generator=g, device="cuda", dtype=torch.int32)
    q, kn, vn = rnd(B, M, H, D), rnd(B, M, 1, D), rnd(B, M, 1, D)
    n, new = lens[0].clone(), news[0].clone()
    ws = torch.empty(s2.s2attn_tree_decode_workspace_bytes(B, M, H, 1, D), dtype=torch.uint8, device="cuda").fill_(0xff)

    def call():
        o, lse = torch.zeros_like(q), torch.zeros(B, H, M, device="cuda")
        s2.s2attn_tree_decode(q, kn, vn, kp, vp, table, n, o, lse, ws, new_len=new)
        return o, lse
    want = call()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for i in range(200):
        with torch.cuda.stream(other):
            for j in range(4):
                n.copy_(lens[j % 2])
                new.copy_(news[j % 2])
        call()
    torch.cuda.synchronize()
    n.copy_(lens[0])
    new.copy_(news[0])
    got = call()
    no_device_error()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
