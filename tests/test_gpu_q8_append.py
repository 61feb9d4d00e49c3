"""sd_q8_append: new K/V rows quantised as they are written, codes and scales bit-equal to the
definition restated in 64 bits, every other cache row left as it was."""
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

CODES = [torch.int8, torch.float8_e4m3fn]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_sparse_decode_gqa_gb300 import build
    build.build()


def sd():
    from top_sparse_decode_gqa_gb300 import binding
    return binding


def check(k_new, v_new, cache, pos0, count, before):
    code = cache[0].dtype
    n, T = k_new.shape[2], cache[0].shape[2]
    for new, codes, scale, c0, s0 in ((k_new, cache[0], cache[2], before[0], before[2]),
                                      (v_new, cache[1], cache[3], before[1], before[3])):
        want_c, want_s = c0.float().cpu(), s0.cpu().clone()
        v, a = ref.quantise(new.cpu(), code)
        for b in range(new.shape[0]):
            for i in range(n if count is None else min(max(int(count[b]), 0), n)):
                t = int(pos0[b]) + i
                if 0 <= t < T:
                    want_c[b, :, t], want_s[b, :, t] = v[b, :, i].float(), a[b, :, i].float()
        # (some old e4m3 codes are NaNs: equal as such)
        assert torch.allclose(codes.float().cpu(), want_c, rtol=0, atol=0, equal_nan=True)
        assert torch.equal(scale.cpu(), want_s)


def old_cache(B, Hkv, T, d, code, g):
    """A cache that already holds something everywhere."""
    c = [torch.randint(-100, 100, (B, Hkv, T, d), device="cuda", generator=g, dtype=torch.int8).view(code)
         for _ in range(2)]
    return c + [torch.rand(B, Hkv, T, device="cuda", generator=g) for _ in range(2)]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("B,Hkv,n,d,T", [(1, 1, 1, 64, 1), (3, 2, 5, 128, 11), (13, 3, 37, 64, 101), (2, 8, 700, 128, 1000)])
def test_rows_match_the_definition(code, src, B, Hkv, n, d, T):
    g = torch.Generator("cuda").manual_seed(B * 100 + n)
    kv = (3 * torch.randn((B, n, 2 * Hkv, d), device="cuda", generator=g)).to(src)
    kv[:, : n // 2] *= 0.01
    k_new, v_new = kv[:, :, :Hkv].transpose(1, 2), kv[:, :, Hkv:].transpose(1, 2)
    cache = old_cache(B, Hkv, T, d, code, g)
    before = [x.clone() for x in cache]
    pos0 = torch.randint(0, T - n + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    count = torch.randint(0, n + 1, (B,), device="cuda", generator=g, dtype=torch.int32) if B > 1 else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sd().sd_q8_append(k_new, v_new, *cache, pos0, count=count, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(k_new, v_new, cache, pos0, count, before)


@pytest.mark.parametrize("code", CODES)
def test_hard_rows(code):
    """Zero rows, single spikes, the largest and smallest magnitudes, halfway points."""
    d = 128
    x = torch.zeros(1, 1, 9, d)
    x[0, 0, 1, 5] = -1.0
    x[0, 0, 2] = torch.arange(d) - 64.0
    x[0, 0, 3] = 3.0e38
    x[0, 0, 4] = 2.0 ** -101           # below the smallest kept
    x[0, 0, 5] = 2.0 ** -100
    x[0, 0, 6] = (torch.arange(d) - 63.5) * 2.0   # top 127 -> int8 codes at n + 0.5 steps
    x[0, 0, 7] = torch.logspace(-12, 0, d)        # through e4m3's subnormals
    x[0, 0, 8] = -torch.logspace(-3, 2, d)
    x = x.cuda()
    cache = list(sd().q8_cache(1, 1, 9, d, code))
    before = [c.clone() for c in cache]
    pos0 = torch.zeros(1, dtype=torch.int32, device="cuda")
    sd().sd_q8_append(x, -x, *cache, pos0)
    torch.cuda.synchronize()
    check(x, -x, cache, pos0, None, before)


def test_rows_outside_the_cache_are_skipped_and_reported():
    g = torch.Generator("cuda").manual_seed(3)
    B, Hkv, n, d, T = 4, 2, 6, 64, 10
    k, v = (torch.randn(B, Hkv, n, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    cache = old_cache(B, Hkv, T, d, torch.int8, g)
    before = [x.clone() for x in cache]
    pos0 = torch.tensor([-3, 7, 2147483647, 4], dtype=torch.int32, device="cuda")
    count = torch.tensor([6, 9, 6, -2], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sd().sd_q8_append(k, v, *cache, pos0, count=count, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == sd().SD_DEVERR_INDEX
    check(k, v, cache, pos0, count, before)


def test_same_codes_as_the_row_quantiser():
    """int8 codes and scales are those sd_quantize_rows_int8 gives the same rows."""
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(2, 3, 50, 128, device="cuda", generator=g).bfloat16()
    tier = torch.full((2, 50), 2, dtype=torch.uint8, device="cuda")
    codes, scales = sd().sd_quantize_rows_int8(x, tier)
    cache = sd().q8_cache(2, 3, 50, 128)
    sd().sd_q8_append(x, x, *cache, torch.zeros(2, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for c, s in ((cache[0], cache[2]), (cache[1], cache[3])):
        assert torch.equal(c, codes) and torch.equal(s, scales)


def test_far_rows_of_a_cache_above_two_gigabytes():
    B, Hkv, T, d = 1, 1, (1 << 24) + 3 + (1 << 20), 128   # codes of K reach past 2^31 bytes
    cache = sd().q8_cache(B, Hkv, T, d)
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(1, 1, 5, d, device="cuda", generator=g).bfloat16()
    pos0 = torch.tensor([T - 5], dtype=torch.int32, device="cuda")
    sd().sd_q8_append(x, x, *cache, pos0)
    torch.cuda.synchronize()
    v, a = ref.quantise(x.cpu(), torch.int8)
    assert torch.equal(cache[0][:, :, T - 5:].cpu().double(), v) and torch.equal(cache[2][:, :, T - 5:].cpu().double(), a)
    assert int(cache[0][:, :, : T - 5].any()) == 0
