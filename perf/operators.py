"""Cases for the serving operators around an 8-bit K/V cache and a speculative verify step.

Three operators, as a decode loop runs them:

* append: ``sd_q8_append`` quantises new tokens' K/V rows as they are written into an 8-bit
  cache (int8 or e4m3 codes, one fp32 scale a row).
* attend: ``sd_cache_attend`` attends the V query tokens of every sequence to its own cache
  (8-bit or bf16, all rows up to each query's position or selected blocks) and, where the
  batch shares a prefix, to that prefix, which is read once for all sequences.
* verify: ``sd_verify_drafts`` accepts drafted tokens against the target's probabilities and
  samples the next token, from given random numbers.

With ``own`` false ``run`` computes the same in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "int8": torch.int8,
       "e4m3": torch.float8_e4m3fn}
_TOP = {"int8": 127.0, "e4m3": 448.0}
_TINY = 2.0 ** -100  # a row whose largest magnitude is below this is stored as zeros


# ------------------------------------------------------------------------------- cases

def _append(name, B, Hkv, n, d, T, src, code, ragged):
    return {"name": name, "op": "append", "B": B, "Hkv": Hkv, "n": n, "d": d, "T": T, "src": src, "code": code,
            "ragged": ragged}


def _attend(name, B, V, Hq, Hkv, d, T, cache, fill, P=0, out="f32", n_idx=0, block=1):
    return {"name": name, "op": "attend", "B": B, "V": V, "Hq": Hq, "Hkv": Hkv, "d": d, "T": T, "cache": cache,
            "fill": fill, "P": P, "out": out, "n_idx": n_idx, "block": block}


def _verify(name, B, V, N, p, ragged):
    return {"name": name, "op": "verify", "B": B, "V": V, "N": N, "p": p, "ragged": ragged}


def listed():
    return [
        # one decode step's new token of 8 sequences: latency alone
        _append("append_decode", 8, 8, 1, 128, 1024, "bf16", "int8", False),
        # a padded batch of draft windows of different lengths, fp32 projections, d = 64
        _append("append_ragged", 13, 4, 37, 64, 1001, "f32", "int8", True),
        # a prompt's K/V written at once
        _append("append_prompt", 4, 8, 8192, 128, 8192, "bf16", "e4m3", False),
        # a single short chat
        _attend("q8_decode_short", 1, 1, 32, 8, 128, 1000, "int8", 1.0, out="bf16"),
        # a serving batch of sequences of different lengths
        _attend("q8_decode_ragged", 8, 1, 32, 8, 128, 32768, "e4m3", 0.25, out="bf16"),
        # the verify step of 8 drafted tokens over long contexts
        _attend("q8_verify_long", 4, 8, 32, 8, 128, 131072, "int8", 1.0),
        # the top 64 blocks of 64 tokens of each KV head
        _attend("q8_select_blocks", 4, 1, 32, 8, 128, 131072, "int8", 1.0, n_idx=64, block=64),
        # three requests over a short system prompt, 7 query heads a KV head
        _attend("prefix_short", 3, 1, 28, 4, 128, 77, "bf16", 0.0, P=1500),
        # a batch over one long shared document, each with its own turn
        _attend("prefix_decode", 64, 1, 32, 8, 128, 512, "bf16", 0.1, P=32768, out="bf16"),
        # the same with drafted tokens to verify and the own turns kept in 8 bits
        _attend("prefix_verify", 32, 8, 32, 8, 128, 1024, "e4m3", 0.2, P=32768, out="bf16"),
        # one sequence's drafts
        _verify("verify_one", 1, 4, 32768, "f32", False),
        # a batch's drafts against a large vocabulary
        _verify("verify_batch", 64, 8, 131072, "f32", True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads = [(32, 8), (28, 4), (4, 1), (8, 8), (16, 1), (12, 3)]
    while True:
        op = rng.choice(["append", "attend", "attend", "prefix", "prefix", "verify"])
        if op == "append":
            n = _log(rng, 1, 8192)
            c = _append("", _log(rng, 1, 64), rng.choice([1, 3, 4, 8]), n, rng.choice([64, 128, 128]),
                        n + _log(rng, 1, 2048), rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice(["int8", "e4m3"]),
                        rng.random() < 0.5)
            ok = c["B"] * c["Hkv"] * n * c["d"] <= 4 * 8 * 8192 * 128 and c["B"] * c["Hkv"] * c["T"] * c["d"] <= 1 << 27
        elif op in ("attend", "prefix"):
            Hq, Hkv = rng.choice(heads)
            G = Hq // Hkv
            V = rng.randint(1, max(1, 32 // G)) if rng.random() < 0.5 else 1
            d = rng.choice([64, 128, 128])
            out = rng.choice(["f32", "bf16"])
            fill = round(rng.random(), 2)
            if op == "attend":
                T = _log(rng, 1, 131072)
                cache = rng.choice(["int8", "e4m3", "int8", "e4m3", "bf16"])
                c = _attend("", _log(rng, 1, 64), V, Hq, Hkv, d, T, cache, fill, out=out)
                if rng.random() < 0.4:
                    c["block"] = block = rng.choice([1, 4, 16, 64, 5])
                    c["T"] = T = max(1, T // block) * block
                    c["n_idx"] = _log(rng, 1, max(1, min(T // block, 8192 // block)))
            else:
                c = _attend("", _log(rng, 1, 128), V, Hq, Hkv, d, _log(rng, 1, 2048), rng.choice(["bf16", "int8", "e4m3"]),
                            fill, P=_log(rng, 1, 65536), out=out)
            rows = c["B"] * V * Hq
            ok = rows * (c["T"] + c["P"]) <= 32 * 8 * 32 * (32768 + 1024) and c["B"] * Hkv * c["T"] <= 4 * 8 * 131072
        else:
            c = _verify("", _log(rng, 1, 64), rng.randint(1, 12), _log(rng, 1, 131072), rng.choice(["f32", "f32", "bf16"]),
                        rng.random() < 0.5)
            ok = c["B"] * (c["V"] + 1) * c["N"] <= 64 * 9 * 131072
        if ok:
            del c["name"]
            return c


def _lens(c):
    """The sequences' own lengths: from fill * T to T, at least V (the drafted tokens), at most T."""
    B, T, lo = c["B"], c["T"], c["fill"]
    f = np.linspace(lo, 1.0, B) if B > 1 else np.array([1.0])
    return np.clip(np.round(f * T).astype(np.int64), min(T, c["V"]), T)


def _counts(c, most):
    """How many of `most` tokens each sequence of a padded batch has: all of them, or 0 to all."""
    B = c["B"]
    if not c["ragged"]:
        return np.full(B, most, dtype=np.int64)
    return np.round(np.linspace(0, most, B) if B > 1 else np.array([most])).astype(np.int64)


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _quantise(x, code):
    """Codes and scales of rows x [..., d] in 32 bits: a = max |x|, codes of x * (top / a), scale a / top."""
    x = x.float()
    top = _TOP[code]
    a = x.abs().amax(-1, keepdim=True)
    zero = a < _TINY
    a1 = torch.where(zero, torch.ones_like(a), a)
    y = x * (torch.full_like(a1, top) / a1)
    y = torch.where(zero, torch.zeros_like(y), y)
    scale = torch.where(zero, torch.zeros_like(a), a / torch.full_like(a, top))
    if code == "int8":
        return torch.round(y).clamp(-127, 127).to(torch.int8), scale[..., 0]
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale[..., 0]


def _cache(shape, kind, g):
    """A cache of N(0, 1) rows [B, Hkv, T, d] of this kind, with its scales (None for bf16)."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for b in range(shape[0]):
        x[b].normal_(generator=g)
    if kind == "bf16":
        return x, None
    codes = torch.empty(shape, dtype=_DT[kind], device="cuda")
    scales = torch.empty(shape[:-1], dtype=torch.float32, device="cuda")
    for b in range(shape[0]):
        codes[b], scales[b] = _quantise(x[b], kind)
    return codes, scales


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    rng = np.random.default_rng(int(seed))
    s = {"case": c}
    if c["op"] == "append":
        B, Hkv, n, d, T = c["B"], c["Hkv"], c["n"], c["d"], c["T"]
        # the projections' output [B, n, (K heads, V heads), d], seen head-major without a copy
        kv = torch.randn((B, n, 2 * Hkv, d), device="cuda", generator=g).to(_DT[c["src"]])
        s["k_new"], s["v_new"] = (kv[:, :, h:h + Hkv].transpose(1, 2) for h in (0, Hkv))
        for name in ("k", "v"):
            s[name + "_codes"] = torch.zeros((B, Hkv, T, d), dtype=torch.int8, device="cuda").view(_DT[c["code"]])
            s[name + "_scale"] = torch.zeros((B, Hkv, T), dtype=torch.float32, device="cuda")
        s["pos0"] = torch.from_numpy(rng.integers(0, T - n + 1, B).astype(np.int32)).cuda()
        s["count"] = torch.from_numpy(rng.permutation(_counts(c, n)).astype(np.int32)).cuda()
    elif c["op"] == "attend":
        B, V, Hq, Hkv, d, T, P = (c[x] for x in ("B", "V", "Hq", "Hkv", "d", "T", "P"))
        s["q"] = torch.randn((B, V, Hq, d), device="cuda", generator=g).to(torch.bfloat16)
        s["k"], s["ks"] = _cache((B, Hkv, T, d), c["cache"], g)
        s["v"], s["vs"] = _cache((B, Hkv, T, d), c["cache"], g)
        lens = rng.permutation(_lens(c))
        # the V query tokens are the last ones of their sequence
        s["qpos"] = torch.from_numpy((lens[:, None] - V + np.arange(V)[None, :]).astype(np.int32)).cuda()
        s["idx"] = None
        if c["n_idx"]:
            key = torch.rand((B, Hkv, T // c["block"]), device="cuda", generator=g)
            s["idx"] = key.topk(c["n_idx"], -1).indices.sort(-1).values.to(torch.int32)
        s["kp"] = s["vp"] = None
        if P:
            s["kp"], s["vp"] = (torch.randn((Hkv, P, d), device="cuda", generator=g).to(torch.bfloat16) for _ in "kv")
    else:
        B, V, N = c["B"], c["V"], c["N"]
        p = torch.empty((B, V + 1, N), dtype=_DT[c["p"]], device="cuda")
        q = torch.empty((B, V, N), dtype=_DT[c["p"]], device="cuda")
        draft = torch.empty((B, V), dtype=torch.int32, device="cuda")
        for b in range(B):  # a draft model that follows the target at some distance
            z = 2.0 * torch.randn((V + 1, N), device="cuda", generator=g)
            p[b] = torch.softmax(z, -1)
            q[b] = torch.softmax(z[:V] + 0.5 * torch.randn((V, N), device="cuda", generator=g), -1)
            race = torch.empty((V, N), device="cuda").exponential_(generator=g)
            draft[b] = (q[b].float() / race).argmax(-1)
        s["p"], s["q"], s["draft"] = p, q, draft
        s["u"] = torch.rand((B, V), device="cuda", generator=g)
        s["u_next"] = torch.rand((B,), device="cuda", generator=g)
        s["count"] = torch.from_numpy(rng.permutation(_counts(c, V)).astype(np.int32)).cuda()
    if own:  # the buffers and the marshalled call that a decode loop keeps between its steps
        _plan(s)
    return s


def _plan(s):
    from top_sparse_decode_gqa_gb300 import binding as sd
    c = s["case"]
    if c["op"] == "append":
        s["call"] = sd.prepare_q8_append(s["k_new"], s["v_new"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"],
                                         s["pos0"], count=s["count"])
    elif c["op"] == "attend":
        a, s["out"], s["lse"] = sd.make_cache_attend_args(
            s["q"], s["k"], s["v"], s["qpos"], k_scale=s["ks"], v_scale=s["vs"], idx=s["idx"], block=c["block"],
            k_prefix=s["kp"], v_prefix=s["vp"], out_dtype=_DT[c["out"]])
        s["ws"] = sd.cache_attend_workspace(a)
        s["call"] = sd.prepare_cache_attend(a)
    else:
        B, V = s["draft"].shape
        s["tokens"] = torch.empty((B, V + 1), dtype=torch.int32, device="cuda")
        s["accepted"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        s["call"] = sd.prepare_verify_drafts(s["p"], s["q"], s["draft"], s["u"], s["u_next"], s["tokens"], s["accepted"],
                                             count=s["count"])


# ------------------------------------------------------------------------------- passes

def _append_plain(s):
    T, code = s["case"]["T"], s["case"]["code"]
    pos0, count = s["pos0"].long(), s["count"].long()
    src = torch.arange(T, device="cuda")[None, :] - pos0[:, None]          # [B, T]: the new token for cache row t
    hit = ((src >= 0) & (src < count[:, None]))[:, None, :, None]
    src = src.clamp(0, s["case"]["n"] - 1)[:, None, :, None]
    for x, codes, scales in ((s["k_new"], s["k_codes"], s["k_scale"]), (s["v_new"], s["v_codes"], s["v_scale"])):
        y, a = _quantise(x, code)
        y, old = y.view(torch.int8), codes.view(torch.int8)
        old.copy_(torch.where(hit, y.gather(2, src.expand(old.shape)), old))
        scales.copy_(torch.where(hit[..., 0], a.gather(2, src[..., 0].expand(scales.shape)), scales))
    return {"k": s["k_codes"], "v": s["v_codes"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _attend_plain(s):
    c = s["case"]
    B, V, Hq, Hkv, d, T = (c[x] for x in ("B", "V", "Hq", "Hkv", "d", "T"))
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d)
    q = s["q"].float().reshape(B, V, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, V * G, d)
    k, v, ks, vs = s["k"], s["v"], s["ks"], s["vs"]
    rows = torch.arange(T, device="cuda").expand(B, Hkv, T)
    if s["idx"] is not None:
        blk = c["block"]
        rows = (s["idx"].long()[..., None] * blk + torch.arange(blk, device="cuda")).reshape(B, Hkv, -1)
        at = rows[..., None].expand(B, Hkv, rows.shape[-1], d)
        k, v = (x.view(torch.int8).gather(2, at).view(x.dtype) if x.dtype != torch.bfloat16 else x.gather(2, at)
                for x in (k, v))
        if ks is not None:
            ks, vs = ks.gather(2, rows), vs.gather(2, rows)
    k, v = k.float(), v.float()
    if ks is not None:
        k, v = k * ks[..., None], v * vs[..., None]
    z = torch.matmul(q, k.transpose(-1, -2)) * scale                         # [B, Hkv, V*G, rows]
    limit = s["qpos"].long().repeat_interleave(G, dim=1)[:, None, :, None]   # [B, 1, V*G, 1]
    z = torch.where(rows[:, :, None, :] <= limit, z, torch.full_like(z[:1, :1, :1, :1], -math.inf))
    m = z.amax(-1, keepdim=True)
    if c["P"]:
        zp = torch.matmul(q, s["kp"].float().transpose(-1, -2)) * scale      # [B, Hkv, V*G, P]
        m = torch.maximum(m, zp.amax(-1, keepdim=True))
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(z - m0)
    l, o = e.sum(-1, keepdim=True), torch.matmul(e, v)
    if c["P"]:
        e = torch.exp(zp - m0)
        l, o = l + e.sum(-1, keepdim=True), o + torch.matmul(e, s["vp"].float())
    out = o / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m0 + torch.log(l))[..., 0]
    out = out.reshape(B, Hkv, V, G, d).permute(0, 2, 1, 3, 4).reshape(B, V, Hq, d).to(_DT[c["out"]])
    return {"out": out, "lse": lse.reshape(B, Hkv, V, G).permute(0, 2, 1, 3).reshape(B, V, Hq)}


def _verify_plain(s):
    p, q, x, count = s["p"], s["q"], s["draft"].long(), s["count"].long()
    B, V = x.shape
    px = p[:, :V].gather(2, x[..., None])[..., 0].double()
    qx = q.gather(2, x[..., None])[..., 0].double()
    ok = (s["u"].double() * qx < px) & (torch.arange(V, device="cuda") < count[:, None])
    a = ok.to(torch.int32).cumprod(1).sum(1)                                 # accepted drafts
    at = torch.arange(B, device="cuda")
    pa = p[at, a].double()
    r = pa - q[at, a.clamp(max=V - 1)].double() * (a < count)[:, None]
    r = r.clamp(min=0.0)
    cum = r.cumsum(1)
    total = cum[:, -1:]
    whole = pa.cumsum(1)
    cum = torch.where(total > 0, cum, whole)                                 # no residual: the target itself
    nxt = (cum <= s["u_next"].double()[:, None] * cum[:, -1:]).sum(1)
    i = torch.arange(V + 1, device="cuda")[None, :]
    xs = torch.cat([x, torch.full_like(x[:, :1], -1)], 1)
    tokens = torch.where(i < a[:, None], xs, torch.where(i == a[:, None], nxt[:, None], torch.full_like(xs, -1)))
    return {"tokens": tokens.to(torch.int32), "accepted": a.to(torch.int32)}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        s["call"]()
        if op == "append":
            return {"k": s["k_codes"], "v": s["v_codes"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        if op == "attend":
            return {"out": s["out"], "lse": s["lse"]}
        return {"tokens": s["tokens"], "accepted": s["accepted"]}
    return {"append": _append_plain, "attend": _attend_plain, "verify": _verify_plain}[op](s)


# ------------------------------------------------------------------------------- work

def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4, "int8": 1, "e4m3": 1}
    if c["op"] == "append":
        rows = 2 * c["Hkv"] * int(_counts(c, c["n"]).sum())
        return {"bytes": rows * (c["d"] * (size[c["src"]] + 1) + 4), "flops": 3 * rows * c["d"]}
    if c["op"] == "attend":
        B, V, Hq, Hkv, d = (c[x] for x in ("B", "V", "Hq", "Hkv", "d"))
        lens = _lens(c)
        # selected rows past a sequence's length take no part: about their share of the list
        own_rows = float(lens.sum()) if not c["n_idx"] else c["n_idx"] * c["block"] * float((lens / c["T"]).sum())
        row = 2 * d * size[c["cache"]] + (0 if c["cache"] == "bf16" else 8)
        data = Hkv * own_rows * row + 2 * Hkv * c["P"] * d * 2 + B * V * Hq * (d * (2 + size[c["out"]]) + 4)
        return {"bytes": data + 4 * B * Hkv * c["n_idx"], "flops": 4.0 * d * V * Hq * (own_rows + B * c["P"])}
    # one row of p and of q (the first rejected draft's), and the drafts' own entries
    B, V = c["B"], c["V"]
    return {"bytes": B * (2 * c["N"] * size[c["p"]] + V * (2 * size[c["p"]] + 12)), "flops": 3.0 * B * c["N"]}


# ------------------------------------------------------------------------------- definition in 64 bits

def _exact_codes(x, code):
    """[..., d] fp64 values of the input -> (code values, scales), every fp32 step of the definition rounded from 64 bits."""
    top = _TOP[code]
    a = x.abs().max(-1).values
    live = a >= _TINY
    inv = (top / a.where(live, torch.ones_like(a))).float().double()
    y = (x * inv[..., None]).float().double() * live[..., None]
    if code == "int8":
        v = y.round().clamp(-127, 127).to(torch.int8)
    else:
        _, e = torch.frexp(y)
        quantum = torch.exp2((e - 1).clamp(min=-6).double() - 3)
        v = (y / quantum).round() * quantum
        v = v.clamp(-448, 448)
    return v, torch.where(live, a / top, torch.zeros_like(a))


def _exact_append(c, s):
    got = {}
    pos0, count = s["pos0"].tolist(), s["count"].tolist()
    for name in ("k", "v"):
        new, shape = s[name + "_new"], s[name + "_codes"].shape
        codes = torch.zeros(shape, dtype=torch.int8 if c["code"] == "int8" else torch.float32, device="cuda")
        scales = torch.zeros(shape[:-1], dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            v, a = _exact_codes(new[b, :, :count[b]].double(), c["code"])
            codes[b, :, pos0[b]:pos0[b] + count[b]] = v.to(codes.dtype)
            scales[b, :, pos0[b]:pos0[b] + count[b]] = a
        got[name], got[name + "_scale"] = codes, scales
    return got


def _exact_attend(c, s):
    B, V, Hq, Hkv, d, T, P = (c[x] for x in ("B", "V", "Hq", "Hkv", "d", "T", "P"))
    G = Hq // Hkv
    out = torch.zeros((B, V, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, V, Hq), -math.inf, dtype=torch.float64, device="cuda")
    qpos = s["qpos"].cpu().numpy()
    for h in range(Hkv):
        heads = slice(h * G, (h + 1) * G)
        if P:
            q = s["q"][:, :, heads].double().reshape(-1, d)
            zp = (q @ s["kp"][h].double().T).mul_(d ** -0.5)
            lp = torch.logsumexp(zp, 1)
            op = (zp.sub_(lp[:, None]).exp_() @ s["vp"][h].double()).reshape(B, V, G, d)
            lp = lp.reshape(B, V, G)
            del zp
        for b in range(B):
            n = int(qpos[b].max()) + 1
            if s["idx"] is None:
                rows = torch.arange(n, device="cuda")
            else:
                rows = torch.cat([torch.arange(i * c["block"], (i + 1) * c["block"]) for i in s["idx"][b, h].tolist()]).cuda()
                rows = rows[rows < n]
            k, v = (s[x][b, h].view(torch.int8)[rows].view(s[x].dtype).double() if s[x].dtype != torch.bfloat16
                    else s[x][b, h][rows].double() for x in ("k", "v"))
            if s["ks"] is not None:
                k, v = k * s["ks"][b, h][rows].double()[:, None], v * s["vs"][b, h][rows].double()[:, None]
            z = torch.einsum("vgd,td->vgt", s["q"][b, :, heads].double(), k) * d ** -0.5
            seen = rows[None, None, :] <= torch.from_numpy(qpos[b].astype(np.int64)).cuda()[:, None, None]
            z = z.masked_fill(~seen, -math.inf)
            if rows.numel():
                ls = torch.logsumexp(z, -1)
                o = torch.einsum("vgt,td->vgd", torch.exp(z - ls.masked_fill(ls == -math.inf, 0.0)[..., None]), v)
            else:
                ls = torch.full((V, G), -math.inf, dtype=torch.float64, device="cuda")
                o = torch.zeros((V, G, d), dtype=torch.float64, device="cuda")
            if P:
                both = torch.logaddexp(ls, lp[b])
                o = o * torch.exp(ls - both)[..., None] + op[b] * torch.exp(lp[b] - both)[..., None]
                ls = both
            out[b, :, heads], lse[b, :, heads] = o, ls
    return {"out": out, "lse": lse}


def _exact_verify(c, s):
    B, V = c["B"], c["V"]
    tokens, accepted = np.full((B, V + 1), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    draft, u = s["draft"].cpu().numpy(), s["u"].cpu().double().numpy()
    un, count = s["u_next"].cpu().double().numpy(), s["count"].cpu().numpy()
    for b in range(B):
        p, q = s["p"][b].double().cpu().numpy(), s["q"][b].double().cpu().numpy()
        a = 0
        while a < count[b] and u[b, a] * q[a, draft[b, a]] < p[a, draft[b, a]]:
            tokens[b, a] = draft[b, a]
            a += 1
        r = np.maximum(p[a] - q[a], 0.0) if a < count[b] else p[a]
        if not r.any():
            r = p[a]
        cum = np.cumsum(r)
        tokens[b, a] = np.searchsorted(cum, un[b] * cum[-1], side="right")
        accepted[b] = a
    return {"tokens": tokens, "accepted": accepted}


def exact(case, seed):
    global own
    was, own = own, False  # the inputs alone
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](case, s)
