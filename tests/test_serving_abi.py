"""Argument checks of the serving calls (8-bit append, cache attention, draft verification): what
they refuse, before anything is launched.  No GPU needed: no call here reaches a kernel."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def sd():
    from top_sparse_decode_gqa_gb300 import binding, build
    build.build()
    binding.lib()
    return binding


def append_args(sd, **kw):
    a = sd.sd_q8_append_args()
    a.k_new = a.v_new = a.k_codes = a.v_codes = a.k_scale = a.v_scale = a.pos0 = 4096
    a.dtype, a.code_dtype = sd.SD_BF16, sd.SD_I8
    a.B, a.Hkv, a.n, a.d, a.T = 2, 4, 3, 128, 100
    a.k_stride_b = a.v_stride_b = 3 * 4 * 128
    a.k_stride_h = a.v_stride_h = 128
    a.k_stride_n = a.v_stride_n = 4 * 128
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=3), INVALID), (dict(code_dtype=1), INVALID), (dict(code_dtype=9), INVALID),
    (dict(B=-1), INVALID), (dict(n=-1), INVALID), (dict(Hkv=0), INVALID), (dict(Hkv=65536), INVALID), (dict(T=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(B=1 << 20, n=1 << 10), INVALID),
    (dict(k_new=None), INVALID), (dict(v_codes=None), INVALID), (dict(k_scale=None), INVALID), (dict(pos0=None), INVALID),
    (dict(k_new=4098), INVALID), (dict(v_codes=4104), INVALID),
    (dict(k_stride_n=4), INVALID), (dict(v_stride_h=-128), INVALID), (dict(k_stride_b=130), INVALID),
    (dict(dtype=0, k_stride_n=2), INVALID),
])
def test_append_refuses(sd, bad, status):
    assert sd.lib().sd_q8_append(ctypes.byref(append_args(sd, **bad)), None) == status
    assert b"sd_q8_append" in sd.lib().sd_last_error_message()


def test_append_of_nothing(sd):
    for kw in (dict(B=0), dict(n=0)):
        assert sd.lib().sd_q8_append(ctypes.byref(append_args(sd, k_new=None, **kw)), None) == 0
    assert sd.lib().sd_q8_append(None, None) == INVALID


def attend_args(sd, **kw):
    a = sd.sd_cache_attend_args()
    a.q = a.k_cache = a.v_cache = a.k_scale = a.v_scale = a.qpos = a.out = a.lse = a.workspace = 4096
    a.cache_dtype, a.out_dtype = sd.SD_I8, sd.SD_F32
    a.B, a.V, a.Hq, a.Hkv, a.d, a.T, a.block = 2, 1, 8, 2, 128, 100, 1
    a.scale = 0.1
    a.workspace_bytes = 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,status", [
    (dict(cache_dtype=0), INVALID), (dict(cache_dtype=2), INVALID), (dict(out_dtype=2), INVALID),
    (dict(B=-1), INVALID), (dict(V=0), INVALID), (dict(Hq=7), INVALID), (dict(Hkv=0), INVALID), (dict(T=0), INVALID),
    (dict(P=-1), INVALID), (dict(B=65536), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(idx=4096, n_idx=-1), INVALID), (dict(idx=4096, n_idx=1, block=0), INVALID),
    (dict(idx=4096, n_idx=1 << 20, block=1 << 12), INVALID), (dict(idx=4096, n_idx=(1 << 20) + 1, block=1 << 10), INVALID),
    (dict(T=(1 << 30) + 1), INVALID), (dict(P=(1 << 30) + 1, k_prefix=4096, v_prefix=4096), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(V=9), UNSUPPORTED), (dict(Hq=66), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k_scale=None), INVALID), (dict(qpos=None), INVALID), (dict(out=None), INVALID),
    (dict(P=5), INVALID), (dict(q=4100), INVALID), (dict(out=4100), INVALID), (dict(P=5, k_prefix=4104, v_prefix=4096), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace_bytes=100), INVALID), (dict(workspace=4096 + 64), INVALID),
    (dict(B=65535, Hkv=1024, Hq=1024, T=1 << 30), INVALID),
    (dict(Hkv=64, Hq=64, P=1 << 30, k_prefix=4096, v_prefix=4096), INVALID),
])
def test_attend_refuses(sd, bad, status):
    assert sd.lib().sd_cache_attend(ctypes.byref(attend_args(sd, **bad)), None) == status
    assert b"sd_cache_attend" in sd.lib().sd_last_error_message()


def test_attend_of_nothing_and_workspace_sizes(sd):
    L = sd.lib()
    assert L.sd_cache_attend(ctypes.byref(attend_args(sd, B=0, q=None)), None) == 0
    assert L.sd_cache_attend_workspace_bytes(ctypes.byref(attend_args(sd, B=0))) == 0
    assert L.sd_cache_attend_workspace_bytes(ctypes.byref(attend_args(sd, d=96))) == 0
    one = L.sd_cache_attend_workspace_bytes(ctypes.byref(attend_args(sd)))
    more = L.sd_cache_attend_workspace_bytes(ctypes.byref(attend_args(sd, P=100000)))
    assert 0 < one < more
    # a pure computation over the sizes: pointers do not matter
    assert L.sd_cache_attend_workspace_bytes(ctypes.byref(attend_args(sd, q=None, out=None))) == one
    # one byte less is refused
    assert L.sd_cache_attend(ctypes.byref(attend_args(sd, workspace_bytes=one - 1)), None) == INVALID


def verify_status(sd, p=4096, q=4096, dtype=0, draft=4096, u=4096, u_next=4096, B=2, V=3, N=100, tokens=4096, accepted=4096):
    P = ctypes.c_void_p
    return sd.lib().sd_verify_drafts(P(p), P(q), dtype, P(draft), P(u), P(u_next), None, B, V, N, P(tokens), P(accepted),
                                     None, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(B=-1), dict(V=-1), dict(V=1025), dict(N=0), dict(N=(1 << 24) + 1), dict(p=None),
    dict(draft=None), dict(u=None), dict(u_next=None), dict(tokens=None), dict(accepted=None), dict(p=4100), dict(q=4104),
    dict(B=1 << 29),
])
def test_verify_refuses(sd, bad):
    assert verify_status(sd, **bad) == INVALID
    assert b"sd_verify_drafts" in sd.lib().sd_last_error_message()


def test_verify_of_nothing(sd):
    assert verify_status(sd, B=0, p=None) == 0


def test_the_binding_refuses_tensors_that_do_not_fit(sd):
    """Host tensors, wrong types and shapes, before any pointer is passed on."""
    k = torch.zeros(1, 1, 4, 128, dtype=torch.int8)
    s = torch.zeros(1, 1, 4)
    q = torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16)
    pos = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sd.make_cache_attend_args(q, k, k, pos, k_scale=s, v_scale=s)   # on the host
    with pytest.raises(ValueError):
        sd.make_cache_attend_args(q, k, k, pos)                         # no scales
    with pytest.raises(TypeError):
        sd.make_cache_attend_args(q, k.float(), k.float(), pos)
    with pytest.raises(ValueError):
        sd.make_cache_attend_args(q, q, q, pos, k_prefix=q[0])          # half a prefix
    with pytest.raises(TypeError):
        sd.q8_cache(1, 1, 4, 128, torch.float16, device="cpu")
    with pytest.raises(ValueError):
        sd.make_q8_append_args(q, q, k, k, s, s, pos[0])
    with pytest.raises(ValueError):
        sd.sd_verify_drafts(torch.zeros(1, 2, 8), torch.zeros(1, 1, 8), pos, torch.zeros(1, 1), torch.zeros(1))


def test_an_empty_cache_for_the_host_side(sd):
    k, v, ks, vs = sd.q8_cache(2, 3, 5, 64, torch.float8_e4m3fn, device="cpu")
    assert k.shape == v.shape == (2, 3, 5, 64) and k.dtype == torch.float8_e4m3fn
    assert ks.shape == vs.shape == (2, 3, 5) and not bool(ks.any())


def test_a_workspace_of_the_host_is_refused(sd):
    a = sd.sd_cache_attend_args()
    with pytest.raises(ValueError, match="workspace must be a contiguous CUDA tensor"):
        sd.prepare_cache_attend(a, workspace=torch.empty(4096, dtype=torch.uint8))
    assert not a.workspace and a.workspace_bytes == 0
