"""The serving calls together, as a speculative decode loop uses them: the new tokens' K/V quantised
into each sequence's cache (sd_q8_append), their attention over that cache and the prefix that the batch
shares (sd_cache_attend), the drafts checked against the probabilities that follow (sd_verify_drafts),
and the positions moved on by what was accepted.  Every step is held to the 64-bit restatements."""
import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_sparse_decode_gqa_gb300 import build
    build.build()


def sd():
    from top_sparse_decode_gqa_gb300 import binding
    return binding


class Loop:
    """B sequences behind one prefix; every step proposes V - 1 drafts after the last token."""

    def __init__(self, code, B=4, V=4, Hq=8, Hkv=2, d=128, T=64, P=200, N=600, seed=0):
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.B, self.V, self.Hq, self.Hkv, self.d, self.N = B, V, Hq, Hkv, d, N
        self.cache = sd().q8_cache(B, Hkv, T, d, code)
        self.kp, self.vp = (torch.randn(Hkv, P, d, device="cuda", generator=self.g).bfloat16() for _ in range(2))
        self.head = torch.randn(Hq * d, N, device="cuda", generator=self.g) * 0.3
        self.qpos = torch.zeros(B, V, dtype=torch.int32, device="cuda")
        self.q = torch.zeros(B, V, Hq, d, dtype=torch.bfloat16, device="cuda")
        self.kv = torch.zeros(B, V, 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")
        self.count = torch.full((B,), V, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        c = self.cache
        self.args, self.out, self.lse = sd().make_cache_attend_args(
            self.q, c[0], c[1], self.qpos, k_scale=c[2], v_scale=c[3], k_prefix=self.kp, v_prefix=self.vp,
            err_word=self.err)
        self.ws = sd().cache_attend_workspace(self.args)
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def draw(self):
        """The next tokens' inputs (in place), their drafts and the random numbers."""
        B, V, N = self.B, self.V, self.N
        self.q.normal_(generator=self.g)
        self.kv.normal_(generator=self.g)
        self.qprob = torch.softmax(2 * torch.randn(B, V - 1, N, device="cuda", generator=self.g), -1)
        self.draft = self.qprob.argmax(-1).to(torch.int32)
        self.u = 0.2 * torch.rand(B, V - 1, device="cuda", generator=self.g)
        self.un = torch.rand(B, device="cuda", generator=self.g)

    def step(self, stream=None):
        Hkv = self.Hkv
        self.qpos.copy_(self.lens[:, None] + torch.arange(self.V, device="cuda", dtype=torch.int32))
        self.qpos.masked_fill_(torch.arange(self.V, device="cuda") >= self.count[:, None], -1)
        k_new, v_new = self.kv[:, :, :Hkv].transpose(1, 2), self.kv[:, :, Hkv:].transpose(1, 2)
        sd().sd_q8_append(k_new, v_new, *self.cache, self.lens, count=self.count, err_word=self.err, stream=stream)
        sd().sd_cache_attend(self.args, stream=stream)
        self.p = torch.softmax(self.out.reshape(self.B, self.V, -1) @ self.head, -1)
        # half of the drafts' mass moved onto the draft's own choice, so that some are accepted
        self.p[:, :-1] = 0.5 * self.p[:, :-1] + 0.5 * self.qprob
        self.tokens, self.accepted = sd().sd_verify_drafts(self.p, self.qprob, self.draft, self.u, self.un,
                                                           count=(self.count - 1).clamp(min=0), err_word=self.err,
                                                           stream=stream)
        self.lens = self.lens + torch.where(self.count > 0, self.accepted + 1, torch.zeros_like(self.accepted))

    def check(self):
        c = self.cache
        r = ref.attend(self.q, c[0], c[1], self.qpos, c[2], c[3], kp=self.kp, vp=self.vp)
        ref.check_attend(self.out, self.lse, r, f16=False)
        t, a = ref.verify(self.p, self.qprob, self.draft, self.u, self.un, (self.count - 1).clamp(min=0).cpu())
        assert np.array_equal(self.tokens.cpu().numpy(), t) and np.array_equal(self.accepted.cpu().numpy(), a)
        assert int(self.err) == 0


@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
def test_a_speculative_loop(code):
    loop = Loop(code)
    loop.count[2] = 2          # a sequence with fewer drafts
    loop.count[3] = 0          # a finished one: sees the prefix alone
    rows = [[] for _ in range(loop.B)]
    taken = 0
    for _ in range(5):
        loop.draw()
        before = loop.lens.clone()
        loop.step()
        torch.cuda.synchronize()
        loop.check()
        moved = (loop.lens - before).tolist()
        for b, m in enumerate(moved):
            rows[b] += [loop.kv[b, i].clone() for i in range(m)]
        taken += int(loop.accepted.sum())
    assert taken > 0 and int(loop.lens[3]) == 0
    # the cache holds the accepted tokens' rows, whatever rejected ones were there in between
    for b in range(loop.B):
        for i, kv in enumerate(rows[b]):
            v, s = ref.quantise(kv.cpu(), code)
            got = torch.cat([loop.cache[0][b, :, i].float(), loop.cache[1][b, :, i].float()]).cpu().double()
            assert torch.equal(got, v)
            assert torch.equal(torch.cat([loop.cache[2][b, :, i], loop.cache[3][b, :, i]]).cpu().double(), s)


def test_the_loop_on_a_stream_of_its_own_beside_another():
    """Two loops with their own workspaces on two streams at once; the streams given as arguments."""
    loops = [Loop(torch.int8, seed=1), Loop(torch.float8_e4m3fn, P=3000, seed=2)]
    streams = [torch.cuda.Stream() for _ in loops]
    for _ in range(4):
        for loop, s in zip(loops, streams):
            with torch.cuda.stream(s):
                loop.draw()
                loop.step(stream=s)
        torch.cuda.synchronize()
        for loop in loops:
            loop.check()


def test_a_whole_step_captured_and_replayed():
    loop = Loop(torch.float8_e4m3fn, seed=3)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        loop.draw()
        loop.step()
        torch.cuda.synchronize()
        loop.lens.zero_()
        lens = loop.lens
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            loop.step()
            lens.copy_(loop.lens)
    for _ in range(4):
        q, kv = torch.randn_like(loop.q, dtype=torch.float32), torch.randn_like(loop.kv, dtype=torch.float32)
        loop.q.copy_(q)
        loop.kv.copy_(kv)
        loop.u.uniform_(0, 0.2)
        loop.un.uniform_(0, 0.999)
        graph.replay()
        torch.cuda.synchronize()
        loop.check()
    assert int(lens.max()) >= 4


def test_one_workspace_serves_calls_of_different_sizes():
    """The same workspace under calls of other sizes in between, prefix or not: nothing is kept in it."""
    g = torch.Generator("cuda").manual_seed(4)
    big = torch.empty(64 << 20, dtype=torch.uint8, device="cuda").random_(0, 255, generator=g)
    for B, V, Hkv, T, P in ((1, 1, 1, 40, 0), (5, 2, 2, 900, 300), (40, 1, 4, 70, 0), (2, 8, 1, 3000, 1000), (1, 1, 1, 40, 0)):
        cache = sd().q8_cache(B, Hkv, T, 128)
        x = torch.randn(B, Hkv, T, 128, device="cuda", generator=g)
        sd().sd_q8_append(x, -x, *cache, torch.zeros(B, dtype=torch.int32, device="cuda"))
        q = torch.randn(B, V, 4 * Hkv, 128, device="cuda", generator=g).bfloat16()
        qpos = torch.full((B, V), T - 1, dtype=torch.int32, device="cuda")
        pre = {}
        if P:
            pre = {n: torch.randn(Hkv, P, 128, device="cuda", generator=g).bfloat16() for n in ("k_prefix", "v_prefix")}
        out, lse = sd().cache_attend(q, cache[0], cache[1], qpos, workspace=big, k_scale=cache[2], v_scale=cache[3], **pre)
        torch.cuda.synchronize()
        r = ref.attend(q, cache[0], cache[1], qpos, cache[2], cache[3], kp=pre.get("k_prefix"), vp=pre.get("v_prefix"))
        ref.check_attend(out, lse, r, f16=not P)
