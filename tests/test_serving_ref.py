"""The 64-bit restatements that the serving calls are tested against, pinned by something other
than themselves: hand-worked rows, torch's own casts and softmax, brute force."""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref


def test_int8_codes_by_hand():
    x = torch.zeros(1, 64)
    x[0, :5] = torch.tensor([-2.0, 1.0, 0.5, 2.0, 0.0078740157480315])  # scale 2/127, factor 63.5
    v, s = ref.quantise(x, torch.int8)
    # 1 * 63.5 and 0.5 * 63.5 = 31.75; ties go to the even code
    assert v[0, :5].tolist() == [-127.0, 64.0, 32.0, 127.0, 0.0]
    assert s[0].item() == float(torch.tensor(2.0) / torch.tensor(127.0))


def test_e4m3_codes_are_torchs_cast():
    x = torch.randn(500, 128) * torch.logspace(-6, 6, 500)[:, None]
    x[0] = 0
    v, s = ref.quantise(x, torch.float8_e4m3fn)
    a = x.abs().amax(-1, keepdim=True)
    a1 = torch.where(a == 0, torch.ones_like(a), a)
    y = (x * (torch.full_like(a1, 448.0) / a1)).clamp(-448, 448)
    assert torch.equal(v.float(), y.to(torch.float8_e4m3fn).float())
    assert torch.equal(s.float(), (a / torch.full_like(a, 448.0))[:, 0])


@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
def test_rows_below_the_smallest_are_zeros(code):
    v, s = ref.quantise(torch.tensor([[2.0 ** -101, 0.0], [2.0 ** -100, 0.0]]), code)
    assert v[0].tolist() == [0.0, 0.0] and s[0] == 0 and v[1, 0] > 0 and s[1] > 0


def test_attention_is_torchs_softmax():
    g = torch.Generator().manual_seed(1)
    B, V, Hq, Hkv, d, T, P = 2, 3, 6, 2, 64, 20, 7
    q = torch.randn(B, V, Hq, d, generator=g)
    k, v = (torch.randn(B, Hkv, T, d, generator=g) for _ in range(2))
    kp, vp = (torch.randn(Hkv, P, d, generator=g) for _ in range(2))
    qpos = torch.tensor([[4, 5, 6], [17, 30, -1]])
    out, lse, A, Z, n = ref.attend(q, k, v, qpos, kp=kp, vp=vp)
    for b in range(B):
        for t in range(V):
            for h in range(Hq):
                m = max(0, min(int(qpos[b, t]) + 1, T))
                K = torch.cat([k[b, h // 3, :m], kp[h // 3]]).double()
                W = torch.cat([v[b, h // 3, :m], vp[h // 3]]).double()
                z = K @ q[b, t, h].double() / math.sqrt(d)
                w = torch.softmax(z, 0)
                assert np.allclose(out[b, t, h], (w @ W).numpy(), rtol=1e-12, atol=1e-12)
                assert abs(lse[b, t, h] - torch.logsumexp(z, 0).item()) < 1e-12
                assert n[b, t, h] == m + P
                assert np.allclose(A[b, t, h], (w @ W.abs()).numpy(), rtol=1e-12)


def test_attention_over_a_selection_and_over_nothing():
    g = torch.Generator().manual_seed(2)
    q = torch.randn(1, 1, 2, 64, generator=g)
    k, v = (torch.randn(1, 1, 12, 64, generator=g) for _ in range(2))
    idx = torch.tensor([[[1, -1, 5, 1]]])      # blocks of 2: rows 2 3, none, 10 11, 2 3 again
    out, lse, *_ = ref.attend(q, k, v, torch.tensor([[10]]), idx=idx, block=2)
    rows = torch.tensor([2, 3, 10, 2, 3])      # row 11 is past the query
    z = k[0, 0, rows].double() @ q[0, 0, 0].double() / 8.0
    assert np.allclose(out[0, 0, 0], (torch.softmax(z, 0) @ v[0, 0, rows].double()).numpy(), rtol=1e-12)
    out, lse, *_ = ref.attend(q, k, v, torch.tensor([[-1]]))
    assert not out.any() and np.isneginf(lse).all()


def test_verification_by_hand():
    p = torch.tensor([[[0.5, 0.25, 0.25], [0.0, 0.5, 0.5], [1.0, 0.0, 0.0]]])
    q = torch.tensor([[[0.25, 0.5, 0.25], [0.5, 0.25, 0.25]]])
    # the first draft's ratio is 0.25 / 0.5, the second's 0 / 0.5
    t, a = ref.verify(p, q, torch.tensor([[1, 0]]), torch.tensor([[0.49, 0.0]]), torch.tensor([0.6]))
    assert a.tolist() == [1] and t.tolist() == [[1, 2, -1]]   # residual (0, 0.25, 0.25): 0.6 of it is in the last
    t, a = ref.verify(p, q, torch.tensor([[1, 0]]), torch.tensor([[0.5, 0.0]]), torch.tensor([0.6]))
    assert a.tolist() == [0] and t.tolist() == [[0, -1, -1]]  # residual (0.25, 0, 0)
    t, a = ref.verify(p, q, torch.tensor([[1, 2]]), torch.tensor([[0.1, 0.1]]), torch.tensor([0.9]))
    assert a.tolist() == [2] and t.tolist() == [[1, 2, 0]]
    t, a = ref.verify(p, q, torch.tensor([[1, 2]]), torch.tensor([[0.1, 0.1]]), torch.tensor([0.9]), torch.tensor([0]))
    assert a.tolist() == [0] and t.tolist() == [[2, -1, -1]]
    t, a = ref.verify(p, None, torch.tensor([[0, 1]]), torch.tensor([[0.49, 0.51]]), torch.tensor([0.2]))
    assert a.tolist() == [1] and t.tolist() == [[0, 2, -1]]   # 0.51 against 0.5, then token 1 left out


def test_the_bound_lets_no_wrong_weight_through():
    """check_attend refuses an output whose weights are off by more than its arithmetic allows."""
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, 1, 1, 64, generator=g)
    k, v = (torch.randn(1, 1, 50, 64, generator=g) for _ in range(2))
    r = ref.attend(q, k, v, torch.tensor([[49]]))
    out, lse = torch.from_numpy(r[0]).float(), torch.from_numpy(r[1]).float()
    ref.check_attend(out, lse, r, f16=True)
    for bad_out, bad_lse in ((out * (1 + 2e-3), lse), (out, lse + 1e-3), (out + 1e-3, lse)):
        with pytest.raises(AssertionError):
            ref.check_attend(bad_out, bad_lse, r, f16=True)
