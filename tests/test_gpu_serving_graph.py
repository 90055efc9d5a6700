"""The serving calls and the norm's backward captured into one graph, replayed on new inputs, and run on
several streams at once, against the same calls made eagerly: equal bits."""
import pytest
import torch

import shifted_sparse_attention_s2attn_b200 as s2
from serving_utils import no_device_error

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s2.clear_device_error()


class Step:
    """Norm and rotation forward and backward, a tree's mask and attention, rows appended, a page copied."""

    def __init__(self):
        self.B, self.M, self.H, self.Hk, self.D, self.page = 3, 9, 8, 2, 128, 16
        z = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")
        B, M, H, Hk, D = self.B, self.M, self.H, self.Hk, self.D
        self.inputs = dict(q=z(B, M, H, D), k=z(B, M, Hk, D), v=z(B, M, Hk, D), dq=z(B, M, H, D), dk=z(B, M, Hk, D),
                           w=z(D), kp=z(60, self.page, Hk, D), vp=z(60, self.page, Hk, D))
        self.len = z(B, dt=torch.int32)
        self.parents = z(B, M, dt=torch.int32)
        self.table = torch.arange(57, dtype=torch.int32, device="cuda").view(3, 19)
        self.inv = s2.rope_inv_freq(D)[0].cuda()
        self.mask, self.depth = z(B, M, 1, dt=torch.int64), z(B, M, dt=torch.int32)
        self.out = dict(q=z(B, M, H, D), k=z(B, M, Hk, D), dq=z(B, M, H, D), dk=z(B, M, Hk, D), dwq=z(D), dwk=z(D),
                        o=z(B, M, H, D), lse=z(B, H, M, dt=torch.float32))
        self.ws = z(s2.s2attn_tree_decode_workspace_bytes(B, M, H, Hk, D), dt=torch.uint8)
        self.ws2 = z(s2.qk_norm_rope_bwd_workspace_bytes(D), dt=torch.uint8)

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in self.inputs.values():
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        self.len.copy_(torch.randint(0, 19 * self.page - self.M, (self.B,), generator=g, device="cuda"))
        par = torch.randint(0, 1000, (self.B, self.M), generator=g, device="cuda")
        self.parents.copy_(par % torch.arange(1, self.M + 1, device="cuda") - 1)
        for t in self.out.values():
            t.fill_(5)

    def run(self, stream=None):
        x, o = self.inputs, self.out
        s2.s2attn_tree_mask(self.parents, self.mask, self.depth, stream=stream)
        s2.qk_norm_rope_fwd(x["q"], x["k"], o["q"], o["k"], self.inv, wq=x["w"], wk=x["w"], positions=self.depth,
                            stream=stream)
        s2.qk_norm_rope_bwd(x["q"], x["k"], x["dq"], x["dk"], o["dq"], o["dk"], self.inv, wq=x["w"], wk=x["w"],
                            dwq=o["dwq"], dwk=o["dwk"], positions=self.depth, workspace=self.ws2, stream=stream)
        s2.s2attn_tree_decode(o["q"], o["k"], x["v"], x["kp"], x["vp"], self.table, self.len, o["o"], o["lse"], self.ws,
                              tree_mask=self.mask, stream=stream)
        s2.s2attn_cache_append(o["k"], x["v"], x["kp"], x["vp"], self.table, self.len, stream=stream)
        s2.s2attn_cache_copy_pages([x["kp"], x["vp"]], [(0, 57), (0, 59), (20, 58)], stream=stream)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (*self.out.values(), self.inputs["kp"], self.inputs["vp"], self.mask, self.depth)]


def _eager(seeds):
    out = []
    for seed in seeds:
        s = Step()
        s.fill(seed)
        s.run()
        out.append(s.results())
    no_device_error()
    return out


def test_a_captured_step_replayed_on_new_inputs():
    want = _eager([1, 2, 3])
    s = Step()
    s.fill(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for seed, w in zip([1, 2, 3], want):
        s.fill(seed)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w)), seed
    no_device_error()


def test_steps_on_several_streams_at_once():
    """Four steps at once, each on a stream of its own with its own workspaces; a stream given as an object
    and as an address."""
    want = _eager([1, 2, 3, 4])
    steps, streams = [Step() for _ in range(4)], [torch.cuda.Stream() for _ in range(4)]
    for _ in range(5):
        for i, s in enumerate(steps):
            s.fill(i + 1)
        torch.cuda.synchronize()
        for i, (s, st) in enumerate(zip(steps, streams)):
            s.run(stream=st if i % 2 else st.cuda_stream)
        for s, w in zip(steps, want):
            assert all(torch.equal(a, b) for a, b in zip(s.results(), w))
    no_device_error()
