"""sd_cache_attend against exact attention in 64 bits over the values the cache stands for, held to
bounds that follow from the kernel's arithmetic (serving_ref.check_attend)."""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3", "bf16"]
DT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_sparse_decode_gqa_gb300 import build
    build.build()


def sd():
    from top_sparse_decode_gqa_gb300 import binding
    return binding


def make(kind, B, V, Hq, Hkv, d, T, lens, seed=0, spread=1.0):
    """q, a cache whose rows at or past each sequence's length hold garbage (NaN or the largest
    codes, NaN scales), qpos."""
    g = torch.Generator("cuda").manual_seed(1000 + seed)
    q = torch.randn(B, V, Hq, d, device="cuda", generator=g).bfloat16()
    lens = np.asarray(lens)
    x = [torch.randn(B, Hkv, T, d, device="cuda", generator=g) for _ in range(2)]
    if spread != 1.0:  # rows of very different sizes
        x = [t * torch.exp(math.log(spread) * (2 * torch.rand(B, Hkv, T, 1, device="cuda", generator=g) - 1)) for t in x]
    kw = {}
    if kind == "bf16":
        k, v = (t.bfloat16() for t in x)
        for b in range(B):
            k[b, :, lens[b]:] = math.nan
            v[b, :, lens[b]:] = math.inf
    else:
        k, v, ks, vs = sd().q8_cache(B, Hkv, T, d, DT[kind])
        sd().sd_q8_append(x[0], x[1], k, v, ks, vs, torch.zeros(B, dtype=torch.int32, device="cuda"))
        for b in range(B):
            k.view(torch.uint8)[b, :, lens[b]:] = 0x7f
            v.view(torch.uint8)[b, :, lens[b]:] = 0x7f
            ks[b, :, lens[b]:] = math.nan
            vs[b, :, lens[b]:] = math.inf
        kw = dict(k_scale=ks, v_scale=vs)
    qpos = torch.from_numpy((lens[:, None] - V + np.arange(V)[None, :]).astype(np.int32)).cuda()
    return q, k, v, qpos, kw


def run_and_check(q, k, v, qpos, kw, out_dtype, **more):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = sd().cache_attend(q, k, v, qpos, out_dtype=out_dtype, err_word=err, **kw, **more)
    torch.cuda.synchronize()
    assert int(err) == 0
    r = ref.attend(q, k, v, qpos, kw.get("k_scale"), kw.get("v_scale"), more.get("idx"), more.get("block", 1),
                   more.get("k_prefix"), more.get("v_prefix"))
    ref.check_attend(out, lse, r, f16=bool(kw))
    return out, lse


SHAPES = [  # B, V, Hq, Hkv, d, T, lens
    (1, 1, 4, 1, 128, 1, [1]),
    (1, 1, 1, 1, 64, 17, [16]),
    (2, 1, 8, 2, 128, 70, [0, 65]),
    (5, 1, 28, 4, 128, 300, [0, 1, 63, 64, 300]),
    (3, 4, 32, 8, 128, 401, [2, 4, 401]),          # some drafts before the first row: empty rows
    (2, 8, 32, 8, 128, 333, [333, 200]),           # 32 query rows
    (2, 3, 21, 3, 64, 129, [129, 128]),            # 21 query rows, d = 64
    (2, 5, 6, 2, 64, 500, [499, 7]),               # 15 query rows
    (130, 1, 4, 2, 64, 40, [i % 41 for i in range(130)]),   # more sequences than threads of a CTA
    (1, 1, 8, 1, 128, 9000, [8999]),               # one group over many CTAs
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:6])))
def test_own_rows(kind, shape, out_dtype):
    run_and_check(*make(kind, *shape), out_dtype)


MANY = [  # 17 to 32 query rows a KV head: B, V, Hq, Hkv, d, T, lens
    (1, 8, 4, 1, 128, 8, [8]),
    (1, 17, 1, 1, 128, 129, [129]),
    (1, 32, 2, 2, 128, 128, [127]),
    (4, 8, 32, 8, 128, 1500, [1500, 8, 700, 4]),      # drafts before the first row
    (3, 5, 16, 4, 128, 6000, [6000, 0, 257]),         # 20 rows; an empty sequence
    (40, 8, 8, 2, 128, 300, [(i * 37) % 301 for i in range(40)]),   # more sequences than lanes
    (1, 8, 4, 1, 128, 40000, [39999]),                # one group over every SM
    (2, 6, 3, 1, 128, 5000, [4000, 5000]),            # 18 rows
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", MANY, ids=lambda s: "-".join(map(str, s[:6])))
def test_many_query_rows(kind, shape, out_dtype):
    run_and_check(*make(kind, *shape, seed=shape[1]), out_dtype)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_many_query_rows_with_growing_logits_and_scales(kind):
    """Every tile's largest logit, and its V scales, far above those before: the maxima move at every tile."""
    B, V, Hq, Hkv, d, T = 1, 8, 4, 1, 128, 3000
    q, k, v, qpos, kw = make(kind, B, V, Hq, Hkv, d, T, [T], seed=31)
    x = [torch.randn(1, 1, T, d, device="cuda") for _ in range(2)]
    ramp = torch.linspace(0, 1, T, device="cuda")[None, None, :, None]
    x[0] = x[0] * 0.05 + 3.0 * ramp
    x[1] = x[1] * torch.exp2(40 * ramp - 20)
    q.copy_((0.3 * q.float() + 0.7).bfloat16())
    q[0, 3] *= -1.0     # for these the logits fall
    sd().sd_q8_append(x[0].contiguous(), x[1].contiguous(), k, v, kw["k_scale"], kw["v_scale"],
                      torch.zeros(1, dtype=torch.int32, device="cuda"))
    run_and_check(q, k, v, qpos, kw, torch.float32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,Hq,Hkv,d,T,block,n_idx", [(1, 8, 2, 128, 640, 1, 100), (1, 4, 4, 64, 640, 16, 7),
                                                      (3, 12, 3, 128, 640, 5, 50), (8, 8, 2, 128, 640, 64, 10)])
def test_selected_rows(kind, V, Hq, Hkv, d, T, block, n_idx):
    B = 3
    x = make(kind, B, V, Hq, Hkv, d, T, [640, 333, 0], seed=n_idx)
    g = torch.Generator("cuda").manual_seed(n_idx)
    idx = torch.rand(B, Hkv, T // block, device="cuda", generator=g).topk(n_idx, -1).indices.to(torch.int32)
    idx[0, 0, 1] = -1
    idx[1, 0, 2] = idx[1, 0, 3]   # given twice: counts twice
    run_and_check(*x, torch.float32, idx=idx.contiguous(), block=block)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,Hq,Hkv,d,block", [(1, 8, 2, 128, 1), (1, 4, 2, 64, 5), (8, 4, 2, 128, 5), (4, 8, 2, 64, 1)])
def test_rows_that_are_not_selected_may_hold_anything(kind, V, Hq, Hkv, d, block, out_dtype):
    """NaN, infinities and the largest codes in every row that idx leaves out, row 0 first of all: an empty
    slot, a list that ends inside a step and one without any row read nothing of them."""
    B, T, n_idx = 3, 200, 7
    q, k, v, qpos, kw = make(kind, B, V, Hq, Hkv, d, T, [200, 150, 200], seed=40 + V)
    g = torch.Generator("cuda").manual_seed(41)
    idx = (torch.rand(B, Hkv, T // block - 1, device="cuda", generator=g).topk(n_idx, -1).indices + 1).to(torch.int32)
    idx[0, 0, 2] = -1
    idx[2, 1] = -1          # nothing selected at all
    out_of = torch.ones(B, Hkv, T, dtype=torch.bool, device="cuda")
    for b in range(B):
        for h in range(Hkv):
            e = idx[b, h][idx[b, h] >= 0].long()
            out_of[b, h, (e[:, None] * block + torch.arange(block, device="cuda")).reshape(-1)] = False
    assert bool(out_of[:, :, 0].all())
    if kind == "bf16":
        k[out_of], v[out_of] = math.nan, math.inf
    else:
        k.view(torch.uint8)[out_of], v.view(torch.uint8)[out_of] = 0x7f, 0x7f   # e4m3: NaN
        kw["k_scale"][out_of], kw["v_scale"][out_of] = math.nan, math.inf
    run_and_check(q, k, v, qpos, kw, out_dtype, idx=idx, block=block)


def test_bad_indices_are_skipped_and_reported():
    q, k, v, qpos, kw = make("int8", 1, 1, 4, 1, 128, 64, [64])
    idx = torch.tensor([[[3, 64, 9, -2, 2147483647, 5]]], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = sd().cache_attend(q, k, v, qpos, idx=idx, err_word=err, **kw)
    assert int(err) == sd().SD_DEVERR_INDEX
    good = torch.tensor([[[3, 9, 5]]], dtype=torch.int32, device="cuda")
    ref.check_attend(out, lse, ref.attend(q, k, v, qpos, kw["k_scale"], kw["v_scale"], good), True)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("spread", [1e3, 1e12])
def test_rows_of_very_different_scales(kind, spread):
    """Row scales over many orders of magnitude: weights are kept relative to their own largest
    product with the scale, so small-scale rows keep their precision where they count."""
    x = make(kind, 2, 2, 8, 2, 128, 700, [700, 100], seed=5, spread=spread)
    x[0].mul_(1e-3 if spread < 1e6 else 1e-12)   # logits of ordinary size
    run_and_check(*x, torch.float32)


@pytest.mark.parametrize("kind", KINDS)
def test_a_sink_and_a_long_flat_tail(kind):
    """One key whose logit is far above all others, which are alike: the tail's small weights add up
    to a visible share and must not be lost one by one."""
    d, T = 128, 20000
    q, k, v, qpos, kw = make(kind, 1, 1, 4, 1, d, T, [T], seed=6)
    q[:] = 1.0
    row = torch.full((1, 1, 1, d), 1.0, device="cuda")
    if kind == "bf16":
        k[:] = 0.0
        k[:, :, 77] = 1.25
        v[:] = 1.0
        v[:, :, 77] = -1.0
    else:
        one = [torch.zeros(1, 1, T, d, device="cuda"), torch.ones(1, 1, T, d, device="cuda")]
        one[0][:, :, 77], one[1][:, :, 77] = 1.25 * row[0, 0], -row[0, 0]
        sd().sd_q8_append(one[0], one[1], k, v, kw["k_scale"], kw["v_scale"], torch.zeros(1, dtype=torch.int32, device="cuda"))
    for dt in (torch.float32, torch.bfloat16):
        run_and_check(q, k, v, qpos, kw, dt)


@pytest.mark.parametrize("kind", KINDS)
def test_large_and_tiny_queries(kind):
    q, k, v, qpos, kw = make(kind, 2, 1, 8, 2, 128, 200, [200, 150], seed=7)
    q[0, 0, 0] *= 100.0
    q[0, 0, 1] = 0.0
    q[0, 0, 2] *= 2.0 ** -90
    q[1, 0, 3, :7] *= 2.0 ** -20
    run_and_check(q, k, v, qpos, kw, torch.float32)


def test_equal_calls_give_equal_bits_and_leave_nothing_behind():
    x = make("e4m3", 3, 2, 8, 2, 128, 2000, [2000, 3, 900], seed=8)
    q, k, v, qpos, kw = x
    a, o1, l1 = sd().make_cache_attend_args(q, k, v, qpos, **kw)
    ws = sd().cache_attend_workspace(a)
    sd().sd_cache_attend(a)
    first = (o1.clone(), l1.clone())
    ws.fill_(255)     # whatever the workspace holds
    o1.fill_(7.0)
    sd().sd_cache_attend(a)
    torch.cuda.synchronize()
    assert torch.equal(o1, first[0]) and torch.equal(l1, first[1])


def test_a_stream_given_by_its_handle():
    x = make("int8", 3, 2, 8, 2, 128, 500, [500, 3, 400], seed=9)
    want = sd().cache_attend(*x[:4], **x[4])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sd().cache_attend(*x[:4], stream=s.cuda_stream, **x[4])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_capture_and_replay_with_growing_sequences():
    """append and attend captured once and replayed while the positions (device data) grow."""
    B, Hkv, Hq, d, T = 2, 2, 8, 128, 64
    g = torch.Generator("cuda").manual_seed(11)
    cache = sd().q8_cache(B, Hkv, T, d)
    q = torch.empty(B, 1, Hq, d, dtype=torch.bfloat16, device="cuda")
    new = [torch.empty(B, Hkv, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pos = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    a, out, lse = sd().make_cache_attend_args(q, cache[0], cache[1], pos, k_scale=cache[2], v_scale=cache[3])
    ws = sd().cache_attend_workspace(a)

    def step():
        sd().sd_q8_append(new[0], new[1], *cache, pos.view(-1))
        sd().sd_cache_attend(a)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        q.normal_(generator=g), new[0].normal_(generator=g), new[1].normal_(generator=g)
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    for t in range(40):
        q.normal_(generator=g), new[0].normal_(generator=g), new[1].normal_(generator=g)
        pos[0], pos[1] = t, t // 2
        graph.replay()
        torch.cuda.synchronize()
        r = ref.attend(q, cache[0], cache[1], pos, cache[2], cache[3])
        ref.check_attend(out, lse, r, True)
    del ws


def test_far_rows_of_a_cache_above_two_gigabytes():
    T, d = (1 << 24) + 700_001, 128
    g = torch.Generator("cuda").manual_seed(12)
    k, v, ks, vs = sd().q8_cache(1, 1, T, d)
    x = torch.randn(1, 1, 64, d, device="cuda", generator=g).bfloat16()
    sd().sd_q8_append(x, -x, k, v, ks, vs, torch.tensor([T - 64], dtype=torch.int32, device="cuda"))
    q = torch.randn(1, 1, 4, d, device="cuda", generator=g).bfloat16()
    qpos = torch.tensor([[T - 1]], dtype=torch.int32, device="cuda")
    idx = torch.arange(T - 64, T, dtype=torch.int32, device="cuda").view(1, 1, -1)
    out, lse = sd().cache_attend(q, k, v, qpos, k_scale=ks, v_scale=vs, idx=idx)
    kk, vv, s1, s2 = (t[:, :, T - 64:] for t in (k, v, ks, vs))
    r = ref.attend(q, kk, vv, torch.tensor([[63]]), s1, s2)
    ref.check_attend(out, lse, r, True)


def test_the_attended_values_are_those_of_the_tiered_call():
    """A cache of int8 rows attended here and by sd_gather_attend with every row in tier 2."""
    B, Hq, Hkv, d, T = 2, 8, 2, 128, 500
    q, k, v, qpos, kw = make("int8", B, 1, Hq, Hkv, d, T, [T, T], seed=13)
    full = torch.zeros(B, Hkv, T, d, dtype=torch.bfloat16, device="cuda")
    tier = torch.full((B, T), 2, dtype=torch.uint8, device="cuda")
    want, wl, _ = sd().gather_attend(q, full, full, None, T=T, tier=tier, k_int8=k, v_int8=v, k_scale=kw["k_scale"],
                                     v_scale=kw["v_scale"])
    out, lse = run_and_check(q, k, v, qpos, kw, torch.float32)
    # both within 2^-14 of the exact output (two-part weights, logits of size 10)
    assert float((out - want).abs().max()) <= 2.0 ** -13 and float((lse - wl).abs().max()) <= 2.0 ** -13


# ------------------------------------------------------------------ a shared prefix

PREFIX = [  # B, V, Hq, Hkv, d, T, lens, P
    (1, 1, 1, 1, 64, 1, [0], 1),                    # the prefix alone, one row
    (2, 1, 8, 2, 128, 5, [0, 5], 127),
    (3, 1, 28, 4, 128, 77, [77, 1, 0], 129),        # 7 query heads: row tiles of 126
    (2, 3, 9, 3, 64, 40, [40, 2], 1000),
    (40, 1, 8, 2, 128, 30, [i % 31 for i in range(40)], 700),     # 160 rows: two row tiles
    (70, 1, 16, 4, 64, 3, [i % 4 for i in range(70)], 300),       # 280 rows: three
    (5, 8, 32, 8, 128, 100, [100, 8, 9, 50, 3], 520),
    (3, 1, 32, 1, 128, 20, [0, 0, 0], 4000),        # long: split over the SMs
    (1, 32, 1, 1, 128, 64, [64], 260),
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", PREFIX, ids=lambda s: "-".join(map(str, s[:6])))
def test_shared_prefix(kind, shape, out_dtype):
    *own, P = shape
    x = make(kind, *own, seed=P)
    Hkv, d = shape[3], shape[4]
    g = torch.Generator("cuda").manual_seed(P)
    kp, vp = (torch.randn(Hkv, P, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    run_and_check_prefix(x, kp, vp, out_dtype)


EVEN = [  # prefixes whose key tiles are cut into equal runs over all heads (on 152 SMs)
    (2, 1, 320, 320, 64, 3, [3, 0], 200),           # runs shorter than three heads
    (3, 2, 160, 160, 128, 2, [2, 1, 0], 200),
    (33, 8, 80, 80, 64, 8, [8] * 33, 199),          # three row tiles: a pair and one alone
    (33, 8, 8, 8, 128, 8, [i % 9 for i in range(33)], 12743),
    (100, 8, 20, 20, 64, 8, [8] * 100, 5001),       # seven row tiles; more tiles a run than fp32 output folds at
]


@pytest.mark.parametrize("kind,out_dtype,shape",
                         [("int8", torch.float32, s) for s in EVEN[:3] + EVEN[4:]] +
                         [("bf16", torch.bfloat16, s) for s in EVEN[:4]])
def test_shared_prefix_in_equal_runs(kind, out_dtype, shape):
    *own, P = shape
    x = make(kind, *own, seed=P)
    Hkv, d = shape[3], shape[4]
    g = torch.Generator("cuda").manual_seed(P)
    kp, vp = (torch.randn(Hkv, P, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    kp *= torch.linspace(0.2, 2.0, P, device="cuda")[None, :, None].bfloat16()   # maxima that move along the prefix
    run_and_check_prefix(x, kp, vp, out_dtype)
    q, k, v, qpos, kw = x
    two = [sd().cache_attend(q, k, v, qpos, out_dtype=out_dtype, k_prefix=kp, v_prefix=vp, **kw) for _ in range(2)]
    assert torch.equal(two[0][0], two[1][0]) and torch.equal(two[0][1], two[1][1])


def run_and_check_prefix(x, kp, vp, out_dtype):
    # the prefix's weights are bf16 whatever the cache holds: held to the bf16 bound
    q, k, v, qpos, kw = x
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = sd().cache_attend(q, k, v, qpos, out_dtype=out_dtype, err_word=err, k_prefix=kp, v_prefix=vp, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    r = ref.attend(q, k, v, qpos, kw.get("k_scale"), kw.get("v_scale"), kp=kp, vp=vp)
    ref.check_attend(out, lse, r, f16=False)


@pytest.mark.parametrize("d", [64, 128])
def test_prefix_with_growing_logits(d):
    """Keys whose logits grow by many powers of two along the prefix (the output is rescaled over and over)
    and one query row for which they fall."""
    x = make("bf16", 2, 1, 8, 1, d, 4, [4, 0], seed=21)
    P = 1500
    g = torch.Generator("cuda").manual_seed(22)
    vp = torch.randn(1, P, d, device="cuda", generator=g).bfloat16()
    ramp = torch.linspace(0, 40, P, device="cuda")[None, :, None]
    kp = (ramp / math.sqrt(d) * torch.ones(1, 1, d, device="cuda")).bfloat16()
    x[0][:] = 1.0
    x[0][0, 0, 3] = -1.0
    run_and_check_prefix(x, kp, vp, torch.float32)


def test_prefix_rows_of_another_head_do_not_matter():
    """A prefix whose other KV head holds NaN right behind this head's last row."""
    x = make("int8", 2, 1, 8, 2, 128, 8, [8, 3], seed=23)
    g = torch.Generator("cuda").manual_seed(24)
    kp, vp = (torch.randn(2, 200, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
    clean = sd().cache_attend(*x[:4], k_prefix=kp, v_prefix=vp, **x[4])
    kp[1], vp[1] = math.nan, math.nan
    out, lse = sd().cache_attend(*x[:4], k_prefix=kp, v_prefix=vp, **x[4])
    assert torch.equal(out[:, :, :4], clean[0][:, :, :4]) and torch.equal(lse[:, :, :4], clean[1][:, :, :4])


def test_prefix_and_selection_together():
    B, V, Hq, Hkv, d, T = 3, 2, 8, 2, 128, 256
    q, k, v, qpos, kw = make("e4m3", B, V, Hq, Hkv, d, T, [256, 100, 2], seed=25)
    g = torch.Generator("cuda").manual_seed(26)
    kp, vp = (torch.randn(Hkv, 333, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    idx = torch.rand(B, Hkv, 16, device="cuda", generator=g).topk(5, -1).indices.to(torch.int32).contiguous()
    out, lse = sd().cache_attend(q, k, v, qpos, idx=idx, block=16, k_prefix=kp, v_prefix=vp, **kw)
    r = ref.attend(q, k, v, qpos, kw["k_scale"], kw["v_scale"], idx, 16, kp, vp)
    ref.check_attend(out, lse, r, f16=False)
