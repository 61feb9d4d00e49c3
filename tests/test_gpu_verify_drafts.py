"""sd_verify_drafts: accepted drafts and the next token equal to the rule restated in 64 bits."""
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


def make(B, V, N, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    z = 2 * torch.randn(B, V + 1, N, device="cuda", generator=g)
    p = torch.softmax(z, -1).to(dtype)
    q = torch.softmax(z[:, :V] + 0.5 * torch.randn(B, V, N, device="cuda", generator=g), -1).to(dtype)
    race = torch.empty(B, V, N, device="cuda").exponential_(generator=g)
    draft = (q.float() / race).argmax(-1).to(torch.int32) if V else torch.empty(B, 0, dtype=torch.int32, device="cuda")
    u, un = torch.rand(B, V, device="cuda", generator=g), torch.rand(B, device="cuda", generator=g)
    return p, q, draft, u, un


def run(p, q, draft, u, un, count=None, err=None):
    t, a = sd().sd_verify_drafts(p, q, draft, u, un, count=count, err_word=err)
    torch.cuda.synchronize()
    return t.cpu().numpy(), a.cpu().numpy()


def same(got, want):
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,V,N", [(1, 1, 1), (1, 4, 7), (5, 3, 129), (3, 0, 50), (2, 8, 2048), (33, 5, 4099),
                                   (1, 2, 100003), (80, 2, 9000), (170, 1, 5000), (320, 1, 4100), (2, 40, 300)])
def test_matches_the_rule(dtype, B, V, N):
    x = make(B, V, N, dtype, B * 7 + N)
    same(run(*x), ref.verify(*x))
    count = torch.randint(-1, V + 2, (B,), dtype=torch.int32, device="cuda")
    same(run(*x, count=count), ref.verify(*x, count=count))


@pytest.mark.parametrize("N", [33, 5000, 16384])
def test_drafts_without_probabilities(N):
    p, _, _, u, un = make(9, 4, N, torch.float32, N)
    draft = p[:, :4].argmax(-1).to(torch.int32)
    same(run(p, None, draft, u, un), ref.verify(p, None, draft, u, un))


def test_borders():
    """Exact ties of the comparison and of the cumulative sum, equal rows, zero rows, u at its
    ends: dyadic probabilities, for which both sides are exact."""
    N = 1024
    p = torch.zeros(8, 2, N)
    q = torch.zeros(8, 1, N)
    draft = torch.zeros(8, 1, dtype=torch.int32)
    u, un = torch.zeros(8, 1), torch.zeros(8)
    p[:, :, [3, 700, 1000]] = torch.tensor([0.5, 0.25, 0.25])
    q[:, 0, 700] = 0.5
    q[:, 0, 3] = 0.5
    draft[:] = 700
    u[0], un[0] = 0.5, 0.5          # u q == p: not accepted; the residual is {1000: 0.25}
    u[1], un[1] = 0.25, 0.5         # accepted; 0.5 of the next row is not above 0.5: token 700
    u[2], un[2] = 0.25, 0.4999
    u[3], un[3] = 0.0, 0.0          # u = 0: accepted, then the first entry above zero
    u[4], un[4] = 0.9, 0.99999994
    q[5, 0] = p[5, 0]
    draft[5], un[5] = 5, 0.8        # p = q = 0 at the draft: rejected, no residual: the target itself
    p[6] = 0                        # zero rows: no token
    draft[7] = N                    # outside the vocabulary
    x = [t.cuda() for t in (p, q, draft, u, un)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(*x, err=err)
    same(got, ref.verify(*x))
    assert list(got[1][:4]) == [0, 1, 1, 1] and got[0][0, 0] == 1000 and got[0][1, 1] == 700 and got[0][2, 1] == 3
    assert got[0][6, 0] == -1 and int(err) == sd().SD_DEVERR_INDEX


def test_a_token_of_small_probability_is_found_where_it_is():
    """u_next aimed at the middle of single tokens' intervals of a long row (widths of 1e-6):
    sums in 32 bits would give the neighbours."""
    B, N = 64, 131072
    g = torch.Generator("cuda").manual_seed(8)
    p = torch.softmax(torch.randn(1, 1, N, device="cuda", generator=g), -1).expand(B, 1, N).contiguous()
    c = np.cumsum(p[0, 0].cpu().double().numpy())
    t = np.linspace(0, N - 1, B).astype(int)
    un = torch.from_numpy(((c[t] + np.concatenate([[0], c])[t]) / 2 / c[-1]).astype(np.float32)).cuda()
    empty = torch.empty(B, 0, dtype=torch.int32, device="cuda")
    got = run(p, torch.empty(B, 0, N, device="cuda"), empty, torch.empty(B, 0, device="cuda"), un)
    same(got, ref.verify(p, None, empty, torch.empty(B, 0), un))


def test_accepts_at_the_rate_of_the_rule():
    """Over many draws the accepted token's distribution is the target's (a sanity check of the rule
    itself): 4 tokens, the first output's frequencies within 5 standard deviations."""
    n = 60000
    g = torch.Generator("cuda").manual_seed(9)
    p0, q0 = torch.tensor([0.1, 0.2, 0.3, 0.4], device="cuda"), torch.tensor([0.4, 0.3, 0.2, 0.1], device="cuda")
    p = p0.expand(n, 2, 4).contiguous()
    q = q0.expand(n, 1, 4).contiguous()
    draft = torch.multinomial(q0, n, replacement=True, generator=g).to(torch.int32)[:, None]
    u, un = torch.rand(n, 1, device="cuda", generator=g), torch.rand(n, device="cuda", generator=g)
    t, _ = sd().sd_verify_drafts(p, q, draft, u, un)
    f = torch.bincount(t[:, 0].long(), minlength=4).double() / n
    sdv = (p0.double() * (1 - p0.double()) / n).sqrt()
    assert bool(((f - p0.double()).abs() <= 5 * sdv).all())
