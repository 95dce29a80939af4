"""Refusals of the rotary, shared-prefix, scoring and eviction calls, and the plans (no GPU)."""
import ctypes
import math

import pytest
import torch

from head_dim_flash_gb300 import _ffi, api
from tests.test_abi import lib  # noqa: F401

FAKE = 1 << 20  # never read: every call below is refused before a launch
V = dict(sb=4 * 100 * 512, sh=100 * 512, sn=512)


def view(ptr=FAKE, sb=V["sb"], sh=V["sh"], sn=V["sn"]):
    return _ffi.View(ptr, sb, sh, sn)


NULL, ODD, SHIFTED = view(ptr=0), view(sn=12), view(ptr=FAKE + 8)


def rope(lib, dt=0, q=None, k=None, qo=None, ko=None, turns=FAKE, rot=512, m=1.0, start=FAKE, pos=None, B=2, Hq=4,
         Hkv=2, N=100, D=512, packed=False, cu=FAKE):
    plan = _ffi.RopePlan(turns, rot, 0, m)
    q, k, qo, ko = (view() if x is None else x for x in (q, k, qo, ko))
    if packed:
        return lib.ffpa_varlen_rope(dt, q.data, k.data, qo.data, ko.data, plan, cu, start, pos, B, N, Hq, Hkv, D, 0,
                                    None)
    return lib.ffpa_rope(dt, q, k, qo, ko, plan, start, pos, B, Hq, Hkv, N, D, 0, None)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kw,status,msg", [
    (dict(dt=7), 2, "dtype"), (dict(D=48), 2, "head dim"), (dict(D=1056), 2, "head dim"), (dict(rot=8), 2, "rot_dim"),
    (dict(rot=24), 2, "rot_dim"), (dict(rot=528), 2, "rot_dim"), (dict(rot=0), 2, "rot_dim"),
    (dict(m=math.nan), 1, "mscale"), (dict(B=-1), 1, "negative"), (dict(N=-1), 1, "negative"),
    (dict(Hkv=-1), 1, "negative"), (dict(turns=0), 1, "turns"), (dict(turns=FAKE + 4), 1, "turns"),
    (dict(start=FAKE + 2), 1, "4-byte"), (dict(pos=FAKE), 1, "not both"), (dict(q=NULL), 1, "q"),
    (dict(ko=NULL), 1, "k_out"), (dict(qo=SHIFTED), 1, "q_out"), (dict(Hq=1 << 30), 2, "heads")])
def test_rope_refusals(lib, packed, kw, status, msg):  # noqa: F811
    assert rope(lib, packed=packed, **kw) == status
    assert msg in lib.ffpa_last_error().decode()


def test_rope_refusals_of_one_form(lib):  # noqa: F811
    assert rope(lib, q=ODD) == 1 and "stride_n" in lib.ffpa_last_error().decode()
    assert rope(lib, packed=True, cu=None) == 1 and "cu_seqlens" in lib.ffpa_last_error().decode()
    assert rope(lib, packed=True, cu=FAKE + 1) == 1
    assert rope(lib, B=1 << 16, N=1 << 16) == 2 and "tokens" in lib.ffpa_last_error().decode()
    for kw in (dict(B=0), dict(N=0), dict(Hq=0, Hkv=0)):
        assert rope(lib, q=NULL, k=NULL, qo=NULL, ko=NULL, turns=None, start=None, **kw) == 0


def shared(lib, dt=0, q=None, kp=None, vp=None, k=None, v=None, lens=FAKE, o=None, lse=FAKE, ws=FAKE, nbytes=1 << 40,
           B=2, Hq=4, Hkv=2, Nq=1, Np=100, N=100, D=512, scale=0.1):
    q, kp, vp, k, v, o = (view() if x is None else x for x in (q, kp, vp, k, v, o))
    return lib.ffpa_decode_fwd_shared(dt, q, kp, vp, k, v, lens, o, lse, ws, nbytes, B, Hq, Hkv, Nq, Np, N, D, 0, scale,
                                      None)


def weigh(lib, dt=0, q=None, k=None, v=None, lens=FAKE, w=FAKE, wo=FAKE, o=None, lse=FAKE, ws=FAKE, nbytes=1 << 40, B=2,
          Hq=4, Hkv=2, Nq=1, N=100, D=512, scale=0.1):
    q, k, v, o = (view() if x is None else x for x in (q, k, v, o))
    return lib.ffpa_decode_fwd_weights(dt, q, k, v, lens, w, wo, o, lse, ws, nbytes, B, Hq, Hkv, Nq, N, D, 0, scale, None)


@pytest.mark.parametrize("fn", [shared, weigh])
@pytest.mark.parametrize("kw,status,msg", [
    (dict(dt=3), 2, "dtype"), (dict(D=96), 2, "64"), (dict(D=1088), 2, "head dim"), (dict(Hq=3), 1, "multiple"),
    (dict(Hkv=0), 1, "multiple"), (dict(scale=math.inf), 1, "scale"), (dict(N=-1), 1, "negative"),
    (dict(q=NULL), 1, "q"), (dict(k=ODD), 1, "k"), (dict(v=NULL), 1, "v"), (dict(o=SHIFTED), 1, "o"),
    (dict(lse=0), 1, "lse"), (dict(lens=FAKE + 2), 1, "lens"), (dict(nbytes=10), 1, "workspace"),
    (dict(ws=0), 1, "workspace"), (dict(ws=FAKE + 16), 1, "256"),
    (dict(B=1 << 16, Hq=1 << 9, Hkv=1 << 9, N=1 << 20), 2, "units")])
def test_decode_refusals(lib, fn, kw, status, msg):  # noqa: F811
    assert fn(lib, **kw) == status
    assert msg in lib.ffpa_last_error().decode()


def test_decode_refusals_of_one_form(lib):  # noqa: F811
    assert shared(lib, kp=NULL) == 1 and "k_prefix" in lib.ffpa_last_error().decode()
    assert shared(lib, vp=ODD) == 1 and "v_prefix" in lib.ffpa_last_error().decode()
    assert shared(lib, Np=-1) == 1
    assert shared(lib, Np=2 ** 31 - 50) == 2
    assert weigh(lib, w=0) == 1 and "weights" in lib.ffpa_last_error().decode()
    assert weigh(lib, wo=FAKE + 4) == 1 and "weights_out" in lib.ffpa_last_error().decode()
    for kw in (dict(B=0), dict(Nq=0), dict(Hq=0, Hkv=0)):
        assert shared(lib, q=NULL, kp=NULL, k=NULL, v=NULL, o=NULL, lse=0, ws=0, nbytes=0, **kw) == 0
        assert weigh(lib, q=NULL, k=NULL, v=NULL, o=NULL, lse=0, ws=0, nbytes=0, w=0, wo=0, **kw) == 0


def test_workspace_queries(lib):  # noqa: F811
    for D in range(64, 1025, 64):
        for Nq in (1, 3, 40):
            assert lib.ffpa_decode_shared_workspace_bytes(0, 3, 8, 2, Nq, 1000, 100, D) > 0
            # a score per row and token
            assert lib.ffpa_decode_weights_workspace_bytes(1, 3, 8, 2, Nq, 1000, D) >= 3 * 8 * Nq * 1000 * 4
    for bad in ((2, 1, 4, 2, 1, 64), (0, 0, 4, 2, 1, 64), (0, 1, 3, 2, 1, 64), (0, 1, 4, 0, 1, 64), (0, 1, 4, 2, 0, 64),
                (0, 1, 4, 2, 1, 96), (0, 1, 4, 2, 1, 1088), (0, 1, 4, 2, 1, 0)):
        assert lib.ffpa_decode_shared_workspace_bytes(*bad[:5], 100, 100, bad[5]) == 0
        assert lib.ffpa_decode_weights_workspace_bytes(*bad[:5], 100, bad[5]) == 0
    assert lib.ffpa_decode_weights_workspace_bytes(0, 1, 4, 2, 1, -1, 64) == 0
    assert lib.ffpa_decode_shared_workspace_bytes(0, 1, 4, 2, 1, -1, 1, 64) == 0


def evict(lib, dt=0, k=None, v=None, w=FAKE, lens=FAKE, ko=None, vo=None, wo=2 * FAKE, lo=FAKE, kept=FAKE, B=2, Hkv=2,
          N=100, Nout=100, D=512, keep=50, recent=5):
    k, v = view() if k is None else k, view(ptr=4 * FAKE) if v is None else v
    ko, vo = view(ptr=2 * FAKE) if ko is None else ko, view(ptr=3 * FAKE) if vo is None else vo
    return lib.ffpa_kv_evict(dt, k, v, w, lens, ko, vo, wo, lo, kept, B, Hkv, N, Nout, D, keep, recent, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(dt=3), 2, "dtype"), (dict(D=40), 2, "head dim"), (dict(N=-1), 1, "negative"), (dict(keep=0), 1, "keep"),
    (dict(recent=-1), 1, "recent"), (dict(recent=51), 1, "recent"), (dict(Nout=49), 1, "N_out"),
    (dict(k=NULL), 1, "k"), (dict(vo=ODD), 1, "v_out"), (dict(w=0), 1, "weights"), (dict(wo=FAKE + 4), 1, "weights_out"),
    (dict(lens=0), 1, "lens"), (dict(lo=0), 1, "lens_out"), (dict(kept=FAKE + 1), 1, "kept"),
    (dict(B=1 << 20, Hkv=1 << 12), 2, "B*Hkv"),
    # in place is all of it in place
    (dict(ko=view()), 1, "in place"), (dict(vo=view(ptr=4 * FAKE)), 1, "in place"), (dict(wo=FAKE), 1, "in place"),
    (dict(vo=view()), 1, "in place"),
    (dict(ko=view(sn=1024), vo=view(ptr=4 * FAKE), wo=FAKE), 1, "views"),
    (dict(ko=view(), vo=view(ptr=4 * FAKE), wo=FAKE, Nout=90), 1, "views")])
def test_evict_refusals(lib, kw, status, msg):  # noqa: F811
    assert evict(lib, **kw) == status
    assert msg in lib.ffpa_last_error().decode()


def test_evict_nothing(lib):  # noqa: F811
    assert evict(lib, B=0, k=NULL, v=NULL, ko=NULL, vo=NULL, w=0, wo=0, lens=0, lo=0, kept=0) == 0


def test_plans():
    p = api.rope_plan(64, device="cpu")
    assert p.rot_dim == 64 and p.mscale == 1.0 and not p.interleaved
    t = [x % 2 ** 64 for x in p.turns.tolist()]
    for i, x in enumerate(t):  # 64-bit arithmetic: 2^-52 of the value
        assert abs(x / 2 ** 64 - 10000 ** (-2 * i / 64) / (2 * math.pi)) <= 2.0 ** -52
    # whole turns fall away, turning back is the complement
    two = api.rope_plan(16, inv_freq=[2 * math.pi * 2.25, -math.pi / 2] + [0.0] * 6, device="cpu").turns.tolist()
    assert two[0] == 2 ** 62 and two[1] == -(2 ** 62) and two[2:] == [0] * 6
    assert api.rope_plan(16, scaling="yarn", factor=4.0, original_len=100, device="cpu").mscale == 0.1 * math.log(4) + 1
    assert api.rope_plan(16, scaling="yarn", factor=4.0, original_len=100, mscale=2.0, device="cpu").mscale == 2.0
    for kw in (dict(scaling="other"), dict(base=0.0), dict(factor=-1.0), dict(scaling="yarn", factor=2.0),
               dict(inv_freq=[1.0]), dict(inv_freq=[math.inf] * 8), dict(mscale=math.nan)):
        with pytest.raises(ValueError):
            api.rope_plan(16, device="cpu", **kw)
    for rot in (0, 8, 20):
        with pytest.raises(NotImplementedError):
            api.rope_plan(rot, device="cpu")


def test_tensors_off_the_gpu_are_refused():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    w = torch.zeros(1, 2, 4)
    plan = api.rope_plan(64, device="cpu")
    for call in (lambda: api.rope(x, x, plan), lambda: api.varlen_rope(x[0], x[0], plan, torch.zeros(2).int()),
                 lambda: api.decode_fwd_shared(x, x, x, x, x), lambda: api.decode_fwd_weights(x, x, x, w),
                 lambda: api.kv_evict(x, x, w, torch.zeros(1).int(), 2)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_structures_match_the_header():
    assert ctypes.sizeof(_ffi.RopePlan) == 24
