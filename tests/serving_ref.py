"""Plain 64-bit restatements of the serving calls (8-bit append, cache attention, draft
verification) for their tests, and the error bounds the attention is held to."""
import math

import numpy as np
import torch

TINY = 2.0 ** -100


def quantise(x, code):
    """x [..., d] -> (code values fp64, scales fp32 as fp64): every fp32 step of the definition is
    rounded from its exact 64-bit value (a quotient or product of two fp32 numbers, rounded to
    fp64 and then to fp32, is the correctly rounded fp32 one)."""
    x = x.double()
    top = 127.0 if code == torch.int8 else 448.0
    a = x.abs().amax(-1, keepdim=True)
    live = a >= TINY
    safe = torch.where(live, a, torch.ones_like(a))
    inv = (top / safe).float().double()
    y = (x * inv).float().double() * live
    if code == torch.int8:
        v = torch.round(y).clamp(-127, 127)
    else:
        e = torch.frexp(y)[1].clamp(min=-5) - 1   # y = m 2^e, m in [1, 2); subnormals below 2^-6
        step = torch.exp2(e.double() - 3)
        v = (torch.round(y / step) * step).clamp(-448, 448)
    return v, torch.where(live, (a / top).float().double(), torch.zeros_like(a))[..., 0]


def values(codes, scale):
    """Cache rows in fp64 (scale None: a bf16 cache)."""
    if scale is None:
        return codes.double()
    return codes.float().double() * scale.double()[..., None]


def attend(q, k, v, qpos, ks=None, vs=None, idx=None, block=1, kp=None, vp=None):
    """(out, lse, A, Z, n): the attention in fp64, and what bounds its error: A = sum p |v| per
    output, Z = the largest scale * sum |q_j k_j| of each query row's attended rows, n = rows."""
    q, qpos = q.cpu().double(), qpos.cpu().numpy()
    B, V, Hq, d = q.shape
    Hkv, T = k.shape[1], k.shape[2]
    G, sc = Hq // Hkv, 1.0 / math.sqrt(d)
    out, A = np.zeros((B, V, Hq, d)), np.zeros((B, V, Hq, d))
    lse, Z, n = np.full((B, V, Hq), -np.inf), np.zeros((B, V, Hq)), np.zeros((B, V, Hq))
    for b in range(B):
        for h in range(Hkv):
            m = int(min(max(qpos[b].max(), -1), T - 1)) + 1
            kk = values(k[b, h, :m].cpu(), None if ks is None else ks[b, h, :m].cpu()).numpy()
            vv = values(v[b, h, :m].cpu(), None if vs is None else vs[b, h, :m].cpu()).numpy()
            if idx is None:
                rows = np.arange(m)
            else:
                e = idx[b, h].cpu().numpy().astype(np.int64)
                rows = (e[:, None] * block + np.arange(block)[None, :])[(e >= 0)].reshape(-1)
                rows = rows[rows < m]
            for t in range(V):
                mine = rows[rows <= qpos[b, t]]
                K, W = kk[mine], vv[mine]
                if kp is not None:
                    K = np.concatenate([K, kp[h].cpu().double().numpy()])
                    W = np.concatenate([W, vp[h].cpu().double().numpy()])
                if not len(K):
                    continue
                for g in range(G):
                    qq = q[b, t, h * G + g].numpy()
                    z = K @ qq * sc
                    top = z.max()
                    p = np.exp(z - top)
                    s = p.sum()
                    at = (b, t, h * G + g)
                    out[at], A[at] = p @ W / s, p @ np.abs(W) / s
                    lse[at], Z[at], n[at] = top + np.log(s), (np.abs(K) @ np.abs(qq)).max() * sc, len(K)
    return out, lse, A, Z, n


def check_attend(got, got_lse, ref, f16):
    """Holds an sd_cache_attend result to what its arithmetic allows.

    A logit is a fp32 sum of d products in at most d/16 + 2 tensor-core steps, each off by at
    most 2^-23 of the magnitudes added: 2^-19 Z for d <= 128 (10 steps, and the scale factors).
    A relative error r of a weight moves the output by at most r A, and the denominator's by
    another r A (|out| <= A).  Weights of fp32 output are sums of two 16-bit numbers (2^-17
    for bf16 parts, with the second part's own rounding 2^-16); of bf16 output single ones
    (half a step: 2^-8 for bf16 caches, 2^-11 for fp16 weights of 8-bit caches).  The sums over
    n rows take n/16 tensor-core steps and a few merges (64 allowed), 2^-23 each.  The output's
    own rounding: 2^-8 |out| for bf16, 2^-24 for fp32."""
    out, lse, A, Z, n = ref
    single = got.dtype == torch.bfloat16
    r = 2.0 ** -16 if not single else 2.0 ** (-11 if f16 else -8)
    steps = (n / 16 + 64) * 2.0 ** -23
    tol = (r + 2 * 2.0 ** -19 * Z + 2 * steps)[..., None] * A
    tol = tol + np.abs(out) * 2.0 ** (-8 if single else -24) + 1e-30
    g = got.cpu().double().numpy()
    bad = ~(np.abs(g - out) <= tol)
    assert not bad.any(), (f"out: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(g - out) / tol):.2f} of the "
                           f"bound, first at {np.argwhere(bad)[0]}: {g[bad][0]} for {out[bad][0]}")
    gl = got_lse.cpu().double().numpy()
    fin = np.isfinite(lse)
    assert np.array_equal(np.isfinite(gl), fin) and np.array_equal(gl[~fin], lse[~fin]), "lse: infinities differ"
    ltol = 2.0 ** -19 * Z + steps + 2.0 ** -22 * (1 + np.abs(np.where(fin, lse, 0)))
    lbad = fin & ~(np.abs(np.where(fin, gl, 0) - np.where(fin, lse, 0)) <= ltol)
    assert not lbad.any(), f"lse: {np.argwhere(lbad)[0]}: {gl[lbad][0]} for {lse[lbad][0]}"


def verify(p, q, draft, u, un, count=None):
    """(tokens, accepted) in fp64."""
    p, draft = p.cpu().double().numpy(), draft.cpu().numpy()
    q = None if q is None else q.cpu().double().numpy()
    u, un = u.cpu().double().numpy(), un.cpu().double().numpy()
    B, V1, N = p.shape
    tokens, accepted = np.full((B, V1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n = V1 - 1 if count is None else min(max(int(count[b]), 0), V1 - 1)
        a = 0
        while a < n:
            x = draft[b, a]
            if not (0 <= x < N and u[b, a] * (1.0 if q is None else q[b, a, x]) < p[b, a, x]):
                break
            tokens[b, a] = x
            a += 1
        r = p[b, a].copy()
        if a < n:
            if q is not None:
                r = np.maximum(r - q[b, a], 0)
            elif 0 <= draft[b, a] < N:
                r[draft[b, a]] = 0
            if not r.any():
                r = p[b, a]
        c = np.cumsum(r)
        tokens[b, a] = -1 if c[-1] == 0 else np.searchsorted(c, un[b] * c[-1], side="right")
        accepted[b] = a
    return tokens, accepted
