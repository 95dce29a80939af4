"""Rotary positions, decode over a shared prefix, decode that scores its cache and eviction, against their
definitions in 64 bits.

Tolerances: a rounding to the output's type is off by at most eps / 2 of the value. O takes one for P and one for
itself; scores are fp32 sums of D products, off by at most D 2^-23 of the sum of magnitudes (`delta`), which
moves a softmax weight by at most twice that of itself; P in fp16 has steps of 2^-24 below 2^-14 of its row's
largest. The other fp32 steps (exp2, sums, divisions) are within 2^-18."""
import math

import pytest
import torch

import head_dim_flash_gb300 as ffpa
from head_dim_flash_gb300 import api

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def within(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol) & ~(got.double() == ref)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}, worst " \
        f"{float(((got.double() - ref).abs() - tol).nan_to_num(1e9)[bad].max()):.3e} over its bound"


# ----------------------------------------------------------------- rotary positions
def thetas(rot, base=10000.0):
    return base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)


def turned(x, pos, theta, interleaved, m=1.0, sign=1.0):
    """x [..., D] in 64 bits, positions broadcast against x's leading dims."""
    rot = 2 * theta.numel()
    y = x.double().clone()
    a = pos.double()[..., None] * theta * sign
    c, s = torch.cos(a) * m, torch.sin(a) * m
    i = torch.arange(rot // 2, device=x.device)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    u, v = x.double()[..., i], x.double()[..., j]
    y[..., i], y[..., j] = u * c - v * s, u * s + v * c
    return y


def check_turned(got, x, pos, theta, interleaved, m=1.0, sign=1.0, what="rope"):
    ref = turned(x, pos, theta, interleaved, m, sign)
    eps = torch.finfo(x.dtype).eps
    # two fp32 products of values off by 2^-21 (cos, sin) each, then the rounding
    big = x.double().abs().amax(-1, keepdim=True)
    within(got, ref, eps / 2 * ref.abs() + 2.0 ** -19 * max(1, m) * big + 2.0 ** -25, what)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,N,D,rot", [
    (1, 1, 1, 1, 64, 64), (2, 4, 2, 5, 64, 16), (3, 5, 1, 17, 96, 96), (2, 8, 2, 33, 320, 128),
    (1, 32, 8, 70, 512, 512), (2, 3, 3, 9, 992, 976), (1, 2, 1, 130, 1024, 1024), (32, 32, 8, 1, 512, 256)])
def test_rope(dt, interleaved, B, Hq, Hkv, N, D, rot):
    g = gen(1)
    theta = thetas(rot)
    plan = ffpa.rope_plan(rot, interleaved=interleaved)
    q, k = randn(g, B, Hq, N, D, dtype=DT[dt]), randn(g, B, Hkv, N, D, dtype=DT[dt])
    start = torch.randint(0, 100000, (B,), generator=g, device="cuda", dtype=torch.int32)
    pos = start[:, None] + torch.arange(N, device="cuda")
    yq, yk = ffpa.rope(q, k, plan, start=start)
    api.get_status()
    check_turned(yq, q, pos[:, None], theta, interleaved, what="q")
    check_turned(yk, k, pos[:, None], theta, interleaved, what="k")
    # no start; a projection's layout; one tensor
    y, none = ffpa.rope(q.transpose(1, 2).contiguous().transpose(1, 2), None, plan)
    assert none is None
    check_turned(y, q, torch.arange(N, device="cuda"), theta, interleaved, what="from 0")
    # every position given, in place
    any_pos = torch.randint(-(2 ** 31), 2 ** 31 - 1, (B, N), generator=g, device="cuda", dtype=torch.int64).int()
    q2, k2 = q.clone(), k.clone()
    y, z = ffpa.rope(q2, k2, plan, positions=any_pos, q_out=q2, k_out=k2)
    assert y is q2 and z is k2
    # at 2^31 the definition's own angles carry 2^-53 of 2^31 radians: 2^-22
    check_turned(q2, q, any_pos[:, None], theta, interleaved, what="in place q")
    check_turned(k2, k, any_pos[:, None], theta, interleaved, what="in place k")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,D,rot,Hq,Hkv", [
    ((1,), 64, 64, 1, 1), ((0, 5, 0, 0, 31, 1, 0), 320, 64, 4, 2), ((700, 3, 64), 512, 512, 8, 2),
    (tuple(range(40)), 128, 32, 3, 1)])
def test_varlen_rope(dt, lens, D, rot, Hq, Hkv):
    g = gen(2)
    T = sum(lens)
    behind = 7  # rows of no sequence
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    q, k = randn(g, T + behind, Hq, D, dtype=DT[dt]), randn(g, T + behind, Hkv, D, dtype=DT[dt])
    plan = ffpa.rope_plan(rot, interleaved=True, scaling="linear", factor=4.0)
    start = torch.randint(0, 1 << 20, (len(lens),), generator=g, device="cuda", dtype=torch.int32)
    b = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
    local = torch.arange(T, device="cuda") - cu.long()[b]
    yq, yk = torch.full_like(q, 3.0), torch.full_like(k, 3.0)
    out = ffpa.varlen_rope(q, k, plan, cu, start=start, q_out=yq, k_out=yk)
    assert out[0] is yq and out[1] is yk
    pos = (local + start[b])[:, None]
    check_turned(yq[:T], q[:T], pos, thetas(rot) / 4, True)
    check_turned(yk[:T], k[:T], pos, thetas(rot) / 4, True)
    assert bool((yq[T:] == 3).all()) and bool((yk[T:] == 3).all())
    given = torch.randint(0, 1000, (T + behind,), generator=g, device="cuda", dtype=torch.int32)
    yq, yk = ffpa.varlen_rope(q, None, plan, cu, positions=given)
    check_turned(yq[:T], q[:T], given[:T, None], thetas(rot) / 4, True)


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 8.0), ("ntk", 8.0), ("yarn", 16.0)])
def test_scaled_frequencies(scaling, factor):
    rot, original = 128, 4096
    theta, m = thetas(rot), 1.0
    if scaling == "linear":
        theta = theta / factor
    elif scaling == "ntk":
        theta = thetas(rot, 10000.0 * factor ** (rot / (rot - 2)))
    elif scaling == "yarn":
        out, m = theta.clone(), 0.1 * math.log(factor) + 1
        for i, t in enumerate(theta.tolist()):
            r = original * t / (2 * math.pi)
            w = min(1.0, max(0.0, (r - 1) / 31))
            out[i] = t / factor * (1 - w) + t * w
        theta = out
    plan = ffpa.rope_plan(rot, scaling=scaling, factor=factor, original_len=original)
    q = randn(gen(3), 1, 2, 300, 256, dtype=torch.bfloat16)
    start = ints(130000)
    y, _ = ffpa.rope(q, None, plan, start=start)
    check_turned(y, q, torch.arange(300, device="cuda") + 130000, theta, False, m)
    y2, _ = ffpa.rope(q, None, ffpa.rope_plan(rot, inv_freq=theta, mscale=m), start=start)
    check_turned(y2, q, torch.arange(300, device="cuda") + 130000, theta, False, m)


@pytest.mark.parametrize("packed", [False, True])
def test_rope_gradient(packed):
    """<dy, R x> differentiated by the formula (R^T dy) and by a difference along a direction."""
    g = gen(4)
    D, rot = 320, 96
    plan = ffpa.rope_plan(rot, interleaved=packed, mscale=1.25)
    theta = thetas(rot)
    if packed:
        cu = ints(0, 9, 9, 30)
        q, k = (randn(g, 33, h, D, dtype=torch.float16).requires_grad_() for h in (4, 2))
        pos = torch.cat((torch.arange(9), torch.arange(21))).cuda()[:, None]
        yq, yk = ffpa.varlen_rope(q, k, plan, cu)
        rows = slice(0, 30)
    else:
        q, k = (randn(g, 2, h, 30, D, dtype=torch.float16).requires_grad_() for h in (4, 2))
        pos = torch.arange(30, device="cuda")
        yq, yk = ffpa.rope(q, k, plan)
        rows = slice(None)
    dy = [randn(g, *y.shape, dtype=torch.float16) for y in (yq, yk)]
    dq, dk = torch.autograd.grad((yq, yk), (q, k), dy)
    check_turned(dq[rows], dy[0][rows], pos, theta, packed, 1.25, -1.0, "dq")
    check_turned(dk[rows], dy[1][rows], pos, theta, packed, 1.25, -1.0, "dk")
    if packed:
        assert bool((dq[30:] == 0).all()) and bool((dk[30:] == 0).all())
    # the operator is linear: f(x + h) - f(x) = <dy, R h>, exact in 64 bits, against <grad, h>
    h = randn(g, *q.shape, dtype=torch.float16)
    lhs = (dy[0][rows].double() * turned(h[rows], pos, theta, packed, 1.25)).sum()
    rhs = (dq[rows].double() * h[rows].double()).sum()
    slack = (torch.finfo(torch.float16).eps / 2 * dq[rows].double().abs() + 2.0 ** -17) * h[rows].double().abs()
    assert abs(float(lhs - rhs)) <= float(slack.sum())
    # only one output used, a gradient that is broadcast
    y = (ffpa.varlen_rope(q, k, plan, ints(0, 33)) if packed else ffpa.rope(q, k, plan))[1]
    y.sum().backward()
    assert q.grad is None or bool((q.grad == 0).all())
    p2 = torch.arange(33, device="cuda")[:, None] if packed else pos
    check_turned(k.grad, torch.ones_like(k), p2, theta, packed, 1.25, -1.0, "broadcast")


@pytest.mark.parametrize("Nq,Nkv", [(40, 40), (3, 40), (40, 25)])
def test_attention_takes_a_plan(Nq, Nkv):
    g = gen(5)
    plan = ffpa.rope_plan(64)
    q = randn(g, 2, 4, Nq, 128, dtype=torch.bfloat16).requires_grad_()
    k, v = (randn(g, 2, 2, Nkv, 128, dtype=torch.bfloat16).requires_grad_() for _ in range(2))
    o = ffpa.attention(q, k, v, causal=True, rope=plan)
    pq = (torch.arange(Nq, device="cuda") + Nkv - Nq).int().expand(2, Nq).contiguous()
    q2, _ = ffpa.rope(q, None, plan, positions=pq)
    k2, _ = ffpa.rope(k, None, plan)
    o2 = ffpa.attention(q2, k2, v, causal=True)
    assert torch.equal(o, o2)
    do = randn(g, *o.shape, dtype=torch.bfloat16)
    for x, y in zip(torch.autograd.grad(o, (q, k, v), do), torch.autograd.grad(o2, (q, k, v), do)):
        assert torch.equal(x, y)


def test_varlen_attention_takes_a_plan():
    g = gen(6)
    plan = ffpa.rope_plan(64, interleaved=True)
    cq, ck = ints(0, 10, 25), ints(0, 30, 37)
    q = randn(g, 25, 4, 128, dtype=torch.float16)
    k, v = (randn(g, 37, 2, 128, dtype=torch.float16) for _ in range(2))
    o = ffpa.varlen_attention(q, k, v, cq, ck, causal=True, rope=plan)
    for b in range(2):
        one = [x[c[b]:c[b + 1]].transpose(0, 1)[None] for x, c in ((q, cq), (k, ck), (v, ck))]
        ref = ffpa.attention(*one, causal=True, rope=plan)[0].transpose(0, 1)
        assert float((o[cq[b]:cq[b + 1]].float() - ref.float()).abs().max()) <= 2e-2
    s = ffpa.varlen_attention(k, k, v, ck, causal=True, rope=plan)
    t = ffpa.varlen_attention(*ffpa.varlen_rope(k, k, plan, ck), v, ck, causal=True)
    assert torch.equal(s, t)


def test_rope_gradient_of_one_input():
    g = gen(7)
    plan = ffpa.rope_plan(64)
    q = randn(g, 2, 4, 9, 64, dtype=torch.bfloat16)
    k = randn(g, 2, 2, 9, 64, dtype=torch.bfloat16).requires_grad_()
    pos = torch.arange(9, device="cuda")
    yq, yk = ffpa.rope(q, k, plan)
    dy = randn(g, *yk.shape, dtype=torch.bfloat16)
    (dk,) = torch.autograd.grad((yq, yk), (k,), (torch.ones_like(yq), dy), retain_graph=True)
    check_turned(dk, dy, pos, thetas(64), False, sign=-1.0)
    (dk,) = torch.autograd.grad(yk, (k,), dy)
    check_turned(dk, dy, pos, thetas(64), False, sign=-1.0)
    x = q.clone().requires_grad_()
    (g1,) = torch.autograd.grad(ffpa.rope(x, None, plan)[0].float().pow(2).sum(), (x,), create_graph=True)
    with pytest.raises(RuntimeError):  # not silently without its second derivative
        g1.sum().backward()


# ----------------------------------------------------------------- decode
def reference(q, k, v, end, kp=None, vp=None):
    """Rows of one sequence in 64 bits: q [Hq, Nq, D], k, v [Hkv, n, D], end [Nq]: first key not seen.
    Returns o, lse, the weights per kv head and key of k, sum w |v| and delta."""
    Hq, Nq, D = q.shape
    H = k.shape[0]
    if kp is not None:
        k, v = torch.cat((kp, k), 1), torch.cat((vp, v), 1)
    qd = q.double().reshape(H, -1, D) / math.sqrt(D)
    s = qd @ k.double().transpose(1, 2)
    big = (qd.abs() @ k.double().abs().transpose(1, 2)).amax() if k.shape[1] else torch.zeros((), device=q.device)
    e = end.repeat(Hq // H)[None, :, None]
    s = torch.where(torch.arange(k.shape[1], device=q.device) < e, s, -math.inf)
    z = torch.logsumexp(s, -1) if k.shape[1] else torch.full(s.shape[:2], -math.inf, device=q.device).double()
    p = torch.where(torch.isinf(z)[..., None], 0.0, torch.exp(s - z[..., None]))
    o = p @ v.double()
    return (o.view(Hq, Nq, D), z.view(Hq, Nq), p.sum(1), (p @ v.double().abs()).view(Hq, Nq, D),
            float(big) * D * 2.0 ** -23, v.double().abs().sum(1)[:, None].expand(H, Hq // H * Nq, D).reshape(Hq, Nq, D))


def check_decode(o, lse, ref, what):
    ro, rl, _, mag, delta, steps = ref
    eps = torch.finfo(o.dtype).eps
    tol = mag * (eps / 2 + 2 * delta + 2.0 ** -18) + eps / 2 * ro.abs() + 2.0 ** -25 * steps + 2.0 ** -25
    within(o, ro, tol, what + " o")
    assert torch.equal(torch.isinf(lse), torch.isinf(rl)), what
    fin = ~torch.isinf(rl)
    within(lse[fin], rl[fin], delta + 2.0 ** -20 * (1 + rl[fin].abs()), what + " lse")
    assert bool((o[~fin] == 0).all()) and bool((lse[~fin] == -math.inf).all()), what


def row_ends(n, Nq, causal):
    return n - Nq + 1 + torch.arange(Nq, device="cuda") if causal else torch.full((Nq,), n, device="cuda")


def caches(g, B, H, N, D, dtype, lens, behind=math.nan):
    k, v = randn(g, B, H, N, D, dtype=dtype), randn(g, B, H, N, D, dtype=dtype)
    for b, n in enumerate(lens):
        k[b, :, n:] = behind
        v[b, :, n:] = behind
    return k, v


WEIGH = [  # Hkv, G, Nq, D, N, lens
    (1, 1, 1, 64, 1, (1,)),
    (2, 1, 1, 64, 40, (40, 0, 7)),
    (1, 4, 4, 128, 300, (300, 3, 129, 0, 31)),
    (2, 3, 2, 192, 257, (257, 255, 1)),
    (3, 16, 2, 256, 100, (99, 33)),
    (2, 4, 1, 320, 2001, (2001, 16, 17, 1000)),
    (8, 4, 1, 512, 777, (777,)),
    (1, 16, 4, 512, 300, (300, 150)),
    (2, 8, 3, 448, 130, (5, 130)),
    (1, 7, 3, 832, 333, (333, 64, 2)),
    (2, 2, 1, 1024, 97, (97, 96)),
    (4, 2, 1, 64, 5000, (5000, 4999)),
    (2, 3, 3, 384, 700, (700, 13, 350)),
    (2, 8, 3, 64, 400, (400, 399)),
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,G,Nq,D,N,lens", WEIGH)
def test_decode_weights(dt, causal, H, G, Nq, D, N, lens):
    g = gen(10)
    B = len(lens)
    q = randn(g, B, Nq, H * G, D, dtype=DT[dt]).transpose(1, 2)
    k, v = caches(g, B, H, N, D, DT[dt], lens)
    w0 = torch.rand((B, H, N), generator=g, device="cuda")
    w = torch.full_like(w0, -1.0)
    o, lse, w2 = ffpa.decode_fwd_weights(q, k, v, w0, ints(*lens), causal=causal, weights_out=w)
    api.get_status()
    assert w2 is w
    for b, n in enumerate(lens):
        ref = reference(q[b], k[b, :, :n], v[b, :, :n], row_ends(n, Nq, causal))
        check_decode(o[b], lse[b], ref, f"sequence {b}")
        exact = w0[b, :, :n].double() + ref[2]
        within(w[b, :, :n], exact, (2 * ref[4] + 2.0 ** -18) * ref[2] + 2.0 ** -23 * exact, f"weights {b}")
        assert bool((w[b, :, n:] == -1).all())
    # in place, and the same bits again
    again = w0.clone()
    o2, lse2, w3 = ffpa.decode_fwd_weights(q, k, v, again, ints(*lens), causal=causal)
    assert w3 is again and torch.equal(o, o2) and torch.equal(lse, lse2)
    for b, n in enumerate(lens):
        assert torch.equal(again[b, :, :n], w[b, :, :n]) and torch.equal(again[b, :, n:], w0[b, :, n:])


def test_decode_weights_of_a_long_batch():
    """More sequences than lengths are staged for, most of them empty; no lengths at all."""
    g = gen(11)
    B, H, N, D = 1500, 1, 9, 64
    lens = [(i * 7) % 10 if i % 3 else 0 for i in range(B)]
    q = randn(g, B, 2, 1, D, dtype=torch.bfloat16)
    k, v = caches(g, B, H, N, D, torch.bfloat16, lens)
    w = torch.zeros((B, H, N), device="cuda")
    o, lse, _ = ffpa.decode_fwd_weights(q, k, v, w, ints(*lens))
    api.get_status()
    for b in list(range(0, B, 97)) + [B - 1]:
        ref = reference(q[b], k[b, :, :lens[b]], v[b, :, :lens[b]], row_ends(lens[b], 1, False))
        check_decode(o[b], lse[b], ref, f"sequence {b}")
    k, v = randn(g, 3, 2, 50, D, dtype=torch.float16), randn(g, 3, 2, 50, D, dtype=torch.float16)
    q = randn(g, 3, 4, 2, D, dtype=torch.float16)
    w = torch.zeros((3, 2, 50), device="cuda")
    o, lse, _ = ffpa.decode_fwd_weights(q, k, v, w, causal=True)
    for b in range(3):
        check_decode(o[b], lse[b], reference(q[b], k[b], v[b], row_ends(50, 2, True)), f"whole {b}")
    assert abs(float(w.sum()) - 3 * 4 * 2) < 1e-3


SHARED = [  # B, Hkv, G, Nq, D, Np, N, lens
    (1, 1, 1, 1, 64, 1, 1, (1,)),
    (2, 2, 1, 1, 64, 33, 5, (0, 5)),
    (4, 2, 4, 1, 512, 500, 90, (90, 1, 0, 33)),
    (3, 1, 2, 4, 320, 3, 4, (0, 1, 4)),
    (9, 1, 4, 2, 320, 700, 40, (40, 0, 39, 1, 2, 3, 32, 33, 31)),
    (33, 2, 4, 1, 256, 300, 9, tuple(range(9)) * 3 + (9,) * 6),
    (5, 2, 16, 3, 512, 1000, 20, (20, 3, 0, 7, 19)),
    (40, 1, 8, 1, 640, 400, 3, (3,) * 39 + (0,)),
    (3, 2, 3, 1, 1024, 130, 17, (17, 16, 0)),
    (17, 1, 7, 3, 832, 257, 3, (3,) * 17),
    (70, 1, 4, 1, 512, 5000, 2, (2,) * 70),
    (20, 2, 4, 1, 128, 4000, 60, (60,) * 20),
    (3, 2, 4, 1, 192, 0, 60, (60, 0, 7)),
    (6, 1, 8, 2, 384, 900, 0, (0,) * 6),
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,H,G,Nq,D,Np,N,lens", SHARED)
def test_decode_shared(dt, causal, B, H, G, Nq, D, Np, N, lens):
    g = gen(12)
    q = randn(g, B, Nq, H * G, D, dtype=DT[dt]).transpose(1, 2)
    k, v = caches(g, B, H, N, D, DT[dt], lens)
    # the prefix as [Np, H, D]
    kp, vp = (randn(g, 1, Np, H, D, dtype=DT[dt]).transpose(1, 2) for _ in range(2))
    o, lse = ffpa.decode_fwd_shared(q, kp, vp, k, v, ints(*lens), causal=causal)
    api.get_status()
    for b, n in enumerate(lens):
        ref = reference(q[b], k[b, :, :n], v[b, :, :n], row_ends(Np + n, Nq, causal), kp[0], vp[0])
        check_decode(o[b], lse[b], ref, f"sequence {b}")
    ws = ffpa.decode_shared_workspace(q, kp, k)
    ws.fill_(255)  # whatever it holds
    o2, lse2 = ffpa.decode_fwd_shared(q, kp, vp, k, v, ints(*lens), causal=causal, workspace=ws, out=q)
    assert o2 is q and torch.equal(o, o2) and torch.equal(lse, lse2)


# ----------------------------------------------------------------- eviction
def kept_rows(w, n, keep, recent):
    """Indices that stay, of the first n scores of a list."""
    if n <= keep:
        return list(range(n))
    early = n - recent
    key = [-math.inf if x != x else x for x in w[:early]]
    nan = [x != x for x in w[:early]]
    order = sorted(range(early), key=lambda j: (nan[j], -key[j], j))
    return sorted(order[:keep - recent]) + list(range(early, n))


def scores(g, B, H, N, kind):
    w = torch.exp(2 * randn(g, B, H, N))
    if kind == "ties":
        w = (w * 2).round() / 2
    elif kind == "equal":
        w.fill_(0.25)
    elif kind == "odd":
        w = randn(g, B, H, N)
        w[..., ::7] = math.nan
        w[..., 1::7] = -0.0
        w[..., 2::7] = 0.0
        w[..., 3::11] = math.inf
        w[..., 4::11] = -math.inf
        w[..., 5::13] = 1e-42
    return w


EVICT = [  # Hkv, N, D, lens, keep, recent
    (1, 1, 64, (1,), 1, 0), (2, 40, 64, (40, 0, 39, 20), 20, 0), (1, 300, 320, (300, 299, 128), 128, 128),
    (3, 513, 96, (513, 1, 512), 511, 7), (2, 5000, 512, (5000, 4096, 2049), 2048, 100),
    (1, 9000, 64, (9000, 8999), 8998, 0), (2, 130, 1024, (130, 77), 1, 0), (2, 130, 1024, (130, 77), 1, 1),
    (1, 20000, 128, (20000,), 333, 32), (2, 50, 128, (50, 3), 64, 10),
    # many kv heads: in place, CTAs of 128 and of 256 head dims
    (8, 700, 160, tuple(700 - 41 * i for i in range(16)), 300, 20),
    (8, 700, 320, tuple(700 - 41 * i for i in range(16)), 300, 20)]


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("H,N,D,lens,keep,recent", EVICT)
def test_evict(kind, in_place, H, N, D, lens, keep, recent):
    g = gen(20)
    B = len(lens)
    dt = torch.bfloat16 if in_place else torch.float16
    # stored as [B, N, H, D]
    k, v = (randn(g, B, N, H, D, dtype=dt).transpose(1, 2) for _ in range(2))
    w = scores(g, B, H, N, kind)
    k0, v0, w0 = k.clone(), v.clone(), w.clone()
    n = ints(*lens)
    if in_place:
        ko, vo, wo, no, kept = ffpa.kv_evict(k, v, w, n, keep, recent)
        assert ko is k and vo is v and wo is w and no is n
        before = (k0, v0, w0)
    else:
        m = min(keep, N) + 3
        ko, vo = (torch.full((B, H, m, D), 5.0, dtype=dt, device="cuda") for _ in range(2))
        wo = torch.full((B, H, m), 5.0, device="cuda")
        before = tuple(x.clone() for x in (ko, vo, wo))
        r = ffpa.kv_evict(k, v, w, n, keep, recent, k_out=ko, v_out=vo, weights_out=wo)
        assert r[0] is ko and r[1] is vo and r[2] is wo
        no, kept = r[3:]
        assert n.tolist() == list(lens)
    api.get_status()
    assert no.tolist() == [min(x, keep) for x in lens]
    host = w0.cpu()
    for b in range(B):
        for h in range(H):
            rows = kept_rows(host[b, h].tolist(), lens[b], keep, recent)
            m = len(rows)
            assert kept[b, h, :m].tolist() == rows and bool((kept[b, h, m:] == -1).all())
            j = torch.tensor(rows, dtype=torch.long, device="cuda")
            for got, old, src in ((ko, before[0], k0), (vo, before[1], v0), (wo, before[2], w0)):
                assert torch.equal(got[b, h, :m].nan_to_num(-7), src[b, h, j].nan_to_num(-7))
                assert torch.equal(got[b, h, m:].nan_to_num(-7), old[b, h, m:].nan_to_num(-7))


# ----------------------------------------------------------------- together, and around
def test_a_serving_loop():
    """Tokens get their positions, enter the cache, attend and score it; it is cut when it is full."""
    g = gen(30)
    B, H, G, D, N, keep, recent = 3, 2, 4, 320, 48, 24, 8
    dt = torch.bfloat16
    plan = ffpa.rope_plan(128)
    k, v = (torch.zeros((B, H, N, D), dtype=dt, device="cuda") for _ in range(2))
    w = torch.zeros((B, H, N), device="cuda")
    lens, seen = torch.zeros(B, dtype=torch.int32, device="cuda"), ints(0, 5, 9)
    prefix = [randn(g, 1, H, 100, D, dtype=dt) for _ in range(2)]
    rk, rv, rw = ([[[] for _ in range(H)] for _ in range(B)] for _ in range(3))  # keys, values, scores
    n = 0
    for step in range(70):
        q = randn(g, B, H * G, 1, D, dtype=dt)
        kn, vn = randn(g, B, H, 1, D, dtype=dt), randn(g, B, H, 1, D, dtype=dt)
        q, kn = ffpa.rope(q, kn, plan, start=seen)
        at = lens.long()[:, None, None, None].expand(B, H, 1, D)
        k.scatter_(2, at, kn)
        v.scatter_(2, at, vn)
        w.scatter_(2, at[..., 0], 0.0)
        lens += 1
        seen += 1
        n += 1
        o, lse, _ = ffpa.decode_fwd_weights(q, k, v, w, lens)
        o2, _ = ffpa.decode_fwd_shared(q, *prefix, k, v, lens)
        for b in range(B):
            for h in range(H):
                rk[b][h].append(kn[b, h, 0])
                rv[b][h].append(vn[b, h, 0])
                rw[b][h].append(0.0)
            tk, tv = (torch.stack([torch.stack(x) for x in y[b]]) for y in (rk, rv))
            ref = reference(q[b], tk, tv, row_ends(n, 1, False))
            check_decode(o[b], lse[b], ref, f"step {step}")
            both = reference(q[b], tk, tv, row_ends(100 + n, 1, False), prefix[0][0], prefix[1][0])
            assert float((o2[b].double() - both[0]).abs().max()) < 2e-2
            for h in range(H):
                rw[b][h] = [x + float(y) for x, y in zip(rw[b][h], ref[2][h])]
        if n == N:
            scores_now = w.cpu()
            *_, kept = ffpa.kv_evict(k, v, w, lens, keep, recent)
            for b in range(B):
                for h in range(H):
                    rows = kept_rows(scores_now[b, h].tolist(), n, keep, recent)
                    assert kept[b, h].tolist() == rows
                    for x in (rk, rv, rw):
                        x[b][h] = [x[b][h][j] for j in rows]
            n = keep
            assert lens.tolist() == [keep] * B
        for b in range(B):
            for h in range(H):
                assert torch.allclose(w[b, h, :n].double().cpu(), torch.tensor(rw[b][h]).double(), atol=1e-4)
    api.get_status()


def test_a_captured_step():
    """A step on device lengths is captured once and replayed on new ones, on another stream than the default."""
    g = gen(31)
    B, H, G, D, N = 4, 2, 4, 512, 600
    dt = torch.float16
    plan = ffpa.rope_plan(D)
    k, v = (randn(g, B, H, N, D, dtype=dt) for _ in range(2))
    kp, vp = (randn(g, 1, H, 900, D, dtype=dt) for _ in range(2))
    q0, kn = randn(g, B, H * G, 1, D, dtype=dt), randn(g, B, H, 1, D, dtype=dt)
    lens = ints(1, 2, 3, 4)
    w = torch.zeros((B, H, N), device="cuda")

    def step():
        q, _ = ffpa.rope(q0, kn, plan, start=lens)
        return ffpa.decode_fwd_weights(q, k, v, w, lens, weights_out=w2), ffpa.decode_fwd_shared(q, kp, vp, k, v, lens), \
            ffpa.kv_evict(k, v, w2, lens, 100, 10, k_out=ko, v_out=vo, weights_out=wo, lens_out=no)

    w2 = torch.zeros_like(w)
    ko, vo = (torch.zeros((B, H, 100, D), dtype=dt, device="cuda") for _ in range(2))
    wo, no = torch.zeros((B, H, 100), device="cuda"), ints(0, 0, 0, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = step()
    torch.cuda.current_stream().wait_stream(s)
    for lengths in ((600, 0, 33, 599), (5, 101, 100, 300)):
        lens.copy_(ints(*lengths))
        for x in (w2, ko, vo, wo):
            x.zero_()
        graph.replay()
        flat = [x.clone() for y in outs for x in y] + [no.clone()]
        for x in (w2, ko, vo, wo):
            x.zero_()
        want = step()
        for x, y in zip(flat, [x for y in want for x in y] + [no]):
            assert torch.equal(x, y)
    api.get_status()


def test_two_calls_at_once():
    g = gen(32)
    B, H, G, D, N = 8, 4, 4, 320, 2000
    lens = ints(*[(i * 331) % 2000 for i in range(B)])
    sets = []
    for i in range(2):
        q = randn(g, B, H * G, 1, D, dtype=torch.bfloat16)
        k, v = (randn(g, B, H, N, D, dtype=torch.bfloat16) for _ in range(2))
        w = torch.rand((B, H, N), generator=g, device="cuda")
        want = ffpa.decode_fwd_weights(q, k, v, w, lens, weights_out=torch.zeros_like(w))
        sets.append((q, k, v, w, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for q, k, v, w, want, s in sets:
            with torch.cuda.stream(s):
                got.append((ffpa.decode_fwd_weights(q, k, v, w, lens, weights_out=torch.zeros_like(w)), want))
    torch.cuda.synchronize()
    for x, y in got:
        assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_caches_beyond_32_bits():
    """The second sequence begins more than 2^31 elements behind the first."""
    g = gen(34)
    N, D, lens = 17_000_000, 128, (7, 300)
    k, v = (torch.empty((2, 1, N, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.stride(0) > 2 ** 31
    for b, n in enumerate(lens):
        k[b, :, :n], v[b, :, :n] = randn(g, 1, n, D), randn(g, 1, n, D)
        k[b, :, n:n + 64], v[b, :, n:n + 64] = math.nan, math.nan
    q = randn(g, 2, 4, 1, D, dtype=torch.bfloat16)
    w = torch.zeros((2, 1, N), device="cuda")
    n = ints(*lens)
    o, lse, _ = ffpa.decode_fwd_weights(q, k, v, w, n)
    o2, lse2 = ffpa.decode_fwd_shared(q, k[1:, :, :50], v[1:, :, :50], k, v, n)
    api.get_status()
    for b, m in enumerate(lens):
        ref = reference(q[b], k[b, :, :m], v[b, :, :m], row_ends(m, 1, False))
        check_decode(o[b], lse[b], ref, f"sequence {b}")
        within(w[b, :, :m], ref[2], (2 * ref[4] + 2.0 ** -18) * ref[2] + 2.0 ** -23, "weights")
        ref = reference(q[b], k[b, :, :m], v[b, :, :m], row_ends(50 + m, 1, False), k[1, :, :50], v[1, :, :50])
        check_decode(o2[b], lse2[b], ref, f"behind a prefix {b}")
    assert float(w.sum()) == pytest.approx(8, abs=1e-4)
    last, row = k[1, 0, 299].clone(), kept_rows(w[1, 0, :300].cpu().tolist(), 300, 100, 10)
    before = k[1, 0, :300].clone()
    *_, kept = ffpa.kv_evict(k, v, w, n, 100, 10)
    api.get_status()
    assert kept[1, 0].tolist() == row and n.tolist() == [7, 100]
    assert torch.equal(k[1, 0, :100], before[row]) and torch.equal(k[1, 0, 99], last)
    x = k[:, :, -5:]  # rows at the far end of the storage
    x.copy_(randn(g, 2, 1, 5, D))
    y, _ = ffpa.rope(x, None, ffpa.rope_plan(D), start=ints(3, 1 << 30))
    check_turned(y, x, torch.tensor([[3], [1 << 30]], device="cuda")[:, None] + torch.arange(5, device="cuda"), thetas(D), False)


def test_calls_follow_the_current_stream():
    """On a side stream, behind work that makes their inputs there."""
    g = gen(35)
    plan = ffpa.rope_plan(128)
    q, k, v = (randn(g, 4, h, 2000, 128, dtype=torch.bfloat16) for h in (8, 2, 2))
    lens = ints(2000, 100, 0, 1999)
    w = torch.rand((4, 2, 2000), generator=g, device="cuda")
    s = torch.cuda.Stream()

    def calls(q, k, v, w, lens):
        rq, rk = ffpa.rope(q, k, plan)
        o = ffpa.decode_fwd_weights(rq[:, :, :1], rk, v, w, lens, weights_out=torch.zeros_like(w))
        p = ffpa.decode_fwd_shared(rq[:, :, :3], rk[:1], v[:1], rk, v, lens, causal=True)
        e = ffpa.kv_evict(rk, v, o[2], lens, 64, 8, k_out=torch.zeros_like(k), v_out=torch.zeros_like(v),
                          weights_out=torch.zeros_like(w))
        return [rq, rk, *o, *p, *e]

    want = calls(q, k, v, w, lens)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        late = [torch.zeros_like(x) for x in (q, k, v, w, lens)]
        for _ in range(20):  # the inputs arrive late
            for x, y in zip(late, (q, k, v, w, lens)):
                x.copy_(y)
        got = calls(*late)
    s.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bad", [-1, 51])
def test_a_length_outside_its_cache_is_reported(bad):
    g = gen(33)
    q = randn(g, 2, 4, 1, 64, dtype=torch.bfloat16)
    k, v = (randn(g, 2, 2, 50, 64, dtype=torch.bfloat16) for _ in range(2))
    w = torch.zeros((2, 2, 50), device="cuda")
    for call in (lambda n: ffpa.decode_fwd_weights(q, k, v, w, n),
                 lambda n: ffpa.decode_fwd_shared(q, k[:1], v[:1], k, v, n),
                 lambda n: ffpa.kv_evict(k, v, w, n, 10)):
        call(ints(bad, 50))
        with pytest.raises(ValueError, match="length of sequence 0"):
            api.get_status()
        call(ints(9, 50))
        api.get_status()
