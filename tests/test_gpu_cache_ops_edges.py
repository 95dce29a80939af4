"""The cache operators at their edges: the prefix on the tensor cores in each of its forms, scales below zero, rows that
are not numbers, packed batches with rows of no sequence, forward-mode differentiation, narrow eviction in place.
References and tolerances are those of test_gpu_cache_ops."""
import math

import pytest
import torch
from torch.autograd import forward_ad

import head_dim_flash_gb300 as ffpa
from head_dim_flash_gb300 import api
from tests.test_gpu_cache_ops import DT, caches, check_decode, gen, ints, kept_rows, randn, reference, row_ends, within

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- the prefix on the tensor cores
SPLIT = [  # B, Hkv, G, Nq, D, Np, N, lens
    # one CTA per row tile
    (40, 2, 2, 1, 64, 4225, 5, (0, 5, 1, 2) * 10),
    (30, 2, 2, 3, 128, 1665, 9, (0, 1, 2, 3, 9) * 6),
    (1, 1, 1, 1500, 192, 1100, 0, (0,)),
    # clusters of two, whole and unequal slabs, 128 rows and fewer of them
    (20, 2, 4, 4, 320, 1025, 6, (0, 1, 2, 3, 4) * 4),
    (3, 1, 2, 300, 320, 1153, 40, (0, 40, 7)),
    (1, 1, 2, 1300, 320, 1200, 3, (3,)),
    (9, 4, 4, 2, 448, 1985, 3, (0, 1, 3) * 3),
    (8, 4, 4, 4, 512, 1281, 5, (0, 1, 2, 3, 5, 4, 0, 1)),
    (5, 8, 4, 1, 512, 3000, 30, (0, 30, 1, 16, 17)),
    # pairs
    (11, 2, 4, 3, 512, 2177, 4, (0, 1, 2, 4, 3, 0, 1, 2, 4, 3, 0)),
    (26, 2, 4, 3, 512, 1281, 2, (0, 1) * 13),
    (1, 1, 2, 1300, 512, 1200, 3, (3,)),
    # clusters of three and four
    (12, 2, 4, 3, 576, 2177, 4, (0, 1, 2, 4) * 3),
    (17, 2, 4, 3, 640, 1537, 3, (3,) + (0, 1, 2, 3) * 4),
    (17, 2, 4, 3, 768, 1537, 3, (3,) + (0, 1, 2, 3) * 4),
    (1, 1, 1, 700, 768, 1025, 0, (0,)),
    (12, 2, 4, 3, 832, 2177, 4, (0, 1, 2, 4) * 3),
    (12, 2, 4, 3, 1024, 2177, 4, (0, 1, 2, 4) * 3),
    (1, 1, 1, 700, 1024, 1025, 2, (2,)),
]


def split_taken(B, H, G, Nq, D, Np, N):
    """The scratch of a prefix in the line does not depend on its length; the tensor cores' parts need their own."""
    from head_dim_flash_gb300 import _ffi

    return _ffi.load().ffpa_decode_shared_workspace_bytes(0, B, H * G, H, Nq, Np, N, D) != \
        _ffi.load().ffpa_decode_shared_workspace_bytes(0, B, H * G, H, Nq, 1, N, D)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,H,G,Nq,D,Np,N,lens", SPLIT)
def test_shared_prefix_on_the_tensor_cores(dt, causal, B, H, G, Nq, D, Np, N, lens):
    """Causal limits inside the prefix, on both sides of a tile's border, before whole splits, at no key at all."""
    assert split_taken(B, H, G, Nq, D, Np, N) and len(lens) == B
    g = gen(40)
    q = randn(g, B, Nq, H * G, D, dtype=DT[dt]).transpose(1, 2)
    k, v = caches(g, B, H, N, D, DT[dt], lens)
    kp, vp = (randn(g, 1, Np, H, D, dtype=DT[dt]).transpose(1, 2) for _ in range(2))
    o, lse = ffpa.decode_fwd_shared(q, kp, vp, k, v, ints(*lens), causal=causal)
    api.get_status()
    for b, n in enumerate(lens):
        ref = reference(q[b], k[b, :, :n], v[b, :, :n], row_ends(Np + n, Nq, causal), kp[0], vp[0])
        check_decode(o[b], lse[b], ref, f"sequence {b}")
    again = ffpa.decode_fwd_shared(q, kp, vp, k, v, ints(*lens), causal=causal, out=q)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


# ----------------------------------------------------------------- scales below zero
# softmax(-s q k) is softmax(s (-q) k); products, sums and roundings are the same but for their signs
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,H,G,Nq,D,Np,N,lens", [
    (3, 1, 2, 2, 320, 700, 9, (9, 0, 1)), (30, 2, 2, 3, 128, 1665, 9, (0, 1, 2, 3, 9) * 6),
    (20, 2, 4, 4, 320, 1025, 6, (0, 1, 2, 3, 4) * 4), (8, 4, 4, 4, 512, 1281, 5, (0, 1, 2, 3, 5, 4, 0, 1)),
    (11, 2, 4, 3, 512, 2177, 4, (0, 1, 2, 4, 3, 0, 1, 2, 4, 3, 0)), (12, 2, 4, 3, 1024, 2177, 4, (0, 1, 2, 4) * 3)])
def test_shared_with_a_negative_scale(dt, causal, B, H, G, Nq, D, Np, N, lens):
    g = gen(41)
    q = randn(g, B, H * G, Nq, D, dtype=DT[dt]) * 3  # scores far from each other
    k, v = caches(g, B, H, N, D, DT[dt], lens)
    kp, vp = (randn(g, 1, H, Np, D, dtype=DT[dt]) for _ in range(2))
    s = 1 / math.sqrt(D)
    o, lse = ffpa.decode_fwd_shared(q, kp, vp, k, v, ints(*lens), causal=causal, scale=-s)
    api.get_status()
    for b, n in enumerate(lens):
        ref = reference(-q[b], k[b, :, :n], v[b, :, :n], row_ends(Np + n, Nq, causal), kp[0], vp[0])
        check_decode(o[b], lse[b], ref, f"sequence {b}")
    o2, lse2 = ffpa.decode_fwd_shared(-q, kp, vp, k, v, ints(*lens), causal=causal, scale=s)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_weights_with_a_negative_scale(dt):
    g = gen(42)
    lens = (2001, 16, 0, 1000)
    q = randn(g, 4, 8, 2, 320, dtype=DT[dt])
    k, v = caches(g, 4, 2, 2001, 320, DT[dt], lens)
    w = [torch.zeros((4, 2, 2001), device="cuda") for _ in range(2)]
    a = ffpa.decode_fwd_weights(q, k, v, w[0], ints(*lens), causal=True, scale=-0.07)
    b = ffpa.decode_fwd_weights(-q, k, v, w[1], ints(*lens), causal=True, scale=0.07)
    api.get_status()
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and float(w[0].sum()) == pytest.approx(3 * 16, abs=1e-3)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,H,G,Nq,Nkv,D", [
    (1, 2, 2, 300, 300, 64), (1, 2, 1, 130, 257, 320), (1, 1, 2, 200, 70, 512), (2, 1, 1, 257, 390, 640),
    (1, 1, 1, 140, 129, 992), (1, 2, 1, 260, 700, 1024), (2, 2, 4, 3, 500, 512)])
def test_attention_with_a_negative_scale(dt, causal, B, H, G, Nq, Nkv, D):
    g = gen(43)
    q = (randn(g, B, H * G, Nq, D, dtype=DT[dt]) * 3).requires_grad_()
    k, v = (randn(g, B, H, Nkv, D, dtype=DT[dt]).requires_grad_() for _ in range(2))
    do = randn(g, *q.shape, dtype=DT[dt])
    s = 1 / math.sqrt(D)
    out = []
    for x, scale in ((q, -s), (-q, s)):
        o, lse = ffpa.attention(x, k, v, causal=causal, scale=scale, return_lse=True)
        out.append((o, lse, *torch.autograd.grad(o, (q, k, v), do)))
    api.get_status()
    for b in range(B):
        ref = reference(-q.detach()[b], k.detach()[b], v.detach()[b], row_ends(Nkv, Nq, causal))
        check_decode(out[0][0][b], out[0][1][b], ref, f"entry {b}")
    for x, y, what in zip(*out, ("o", "lse", "dq", "dk", "dv")):
        assert torch.equal(x, y), what


def test_varlen_attention_with_a_negative_scale():
    g = gen(44)
    cu = ints(0, 10, 300, 700)
    q = randn(g, 700, 4, 320, dtype=torch.float16) * 3
    k, v = (randn(g, 700, 2, 320, dtype=torch.float16) for _ in range(2))
    a = ffpa.varlen_attention(q, k, v, cu, causal=True, scale=-0.05, return_lse=True)
    b = ffpa.varlen_attention(-q, k, v, cu, causal=True, scale=0.05, return_lse=True)
    api.get_status()
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and bool(torch.isfinite(a[1]).all())


@pytest.mark.parametrize("D", [128, 512])
def test_fp8_with_a_negative_scale(D):
    g = gen(45)
    q = randn(g, 1, 2, 300, D, dtype=torch.bfloat16) * 3
    k, v = (randn(g, 1, 2, 390, D, dtype=torch.bfloat16) for _ in range(2))
    a, b = (ffpa.fwd_fp8(x, k, v, False, s)[:2] for x, s in ((q, -0.05), (-q, 0.05)))
    api.get_status()
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and bool(torch.isfinite(a[1]).all())


# ----------------------------------------------------------------- rows that are not numbers
def is_nan(x):
    return bool(torch.isnan(x).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("B,H,G,Nq,D,Np,N", [
    (2, 2, 4, 1, 512, 0, 60),       # whole units
    (2, 2, 4, 1, 512, 40, 5000),    # units that ranges cut
    (2, 1, 8, 4, 320, 40, 5000),
    (1, 1, 4, 1, 512, 40000, 5),    # more pieces of a row than a warp has lanes
    (5, 8, 4, 1, 512, 3000, 30),    # the tensor cores: one CTA per slab
    (11, 2, 4, 3, 512, 2177, 4),    # pairs
    (30, 2, 2, 3, 128, 1665, 9)])
def test_shared_rows_that_are_not_numbers(bad, B, H, G, Nq, D, Np, N):
    """A query that is not a number, then one key of the prefix or of a cache."""
    g = gen(46)
    q = randn(g, B, H * G, Nq, D, dtype=torch.bfloat16)
    k, v = (randn(g, B, H, N, D, dtype=torch.bfloat16) for _ in range(2))
    kp, vp = (randn(g, 1, H, Np, D, dtype=torch.bfloat16) for _ in range(2))
    q0 = q.clone()
    q0[B - 1, 1, 0, 5] = bad
    if math.isinf(bad):  # +inf against keys of both signs: some scores are +inf
        q0[B - 1, 1, 0, 5:7] = bad
    o, lse = ffpa.decode_fwd_shared(q0, kp, vp, k, v)
    api.get_status()
    assert is_nan(o[B - 1, 1, 0]) and is_nan(lse[B - 1, 1, 0])
    ref = [reference(q[b], k[b], v[b], row_ends(Np + N, Nq, False), kp[0], vp[0]) for b in range(B)]

    def others(o, lse, there):
        for b in range(B):
            at = there[b]
            x = [y.clone() for y in (o[b], lse[b])]
            for y, z in zip(x, ref[b]):
                y[at] = z[at].to(y.dtype)  # (not compared)
            check_decode(*x, ref[b], f"sequence {b}")

    hit = torch.zeros((B, H * G, Nq), dtype=torch.bool, device="cuda")
    hit[B - 1, 1, 0] = True
    others(o, lse, hit)
    # one key of the prefix: every row of its head; one of a sequence's own: its rows
    for own in (False, True):
        if not own and Np == 0:
            continue
        k1, kp1 = k.clone(), kp.clone()
        hit = torch.zeros((B, H * G, Nq), dtype=torch.bool, device="cuda")
        if own:
            k1[0, H - 1, N // 2, 9] = math.nan
            hit[0, (H - 1) * G:] = True
        else:
            kp1[0, H - 1, Np // 2, 9] = math.nan
            hit[:, (H - 1) * G:] = True
        o, lse = ffpa.decode_fwd_shared(q, kp1, vp, k1, v)
        api.get_status()
        assert is_nan(o[hit]) and is_nan(lse[hit])
        others(o, lse, hit)


@pytest.mark.parametrize("G,Nq,D,N", [(4, 1, 512, 60), (4, 1, 512, 9000), (8, 3, 320, 60), (8, 3, 320, 9000),
                                      (4, 4, 64, 9000)])
def test_weights_of_rows_that_are_not_numbers(G, Nq, D, N):
    g = gen(47)
    q = randn(g, 2, 2 * G, Nq, D, dtype=torch.float16)
    k, v = (randn(g, 2, 2, N, D, dtype=torch.float16) for _ in range(2))
    for what in ("query", "key"):
        q0, k0 = q.clone(), k.clone()
        if what == "query":
            q0[1, 0, 0, 3] = math.nan
        else:
            k0[1, 0, N - 2, 3] = math.nan
        w = torch.zeros((2, 2, N), device="cuda")
        o, lse, _ = ffpa.decode_fwd_weights(q0, k0, v, w)
        api.get_status()
        hit = torch.zeros((2, 2 * G, Nq), dtype=torch.bool, device="cuda")
        if what == "query":
            hit[1, 0, 0] = True
        else:
            hit[1, :G] = True
        assert is_nan(o[hit]) and is_nan(lse[hit]) and is_nan(w[1, 0])
        assert not bool(torch.isnan(o[~hit]).any()) and bool(torch.isfinite(lse[~hit]).all())
        for b, h in ((0, 0), (0, 1), (1, 1)):
            ref = reference(q[b, h * G:(h + 1) * G], k[b, h:h + 1], v[b, h:h + 1], row_ends(N, Nq, False))
            check_decode(o[b, h * G:(h + 1) * G], lse[b, h * G:(h + 1) * G], ref, f"{what} {b} {h}")
            within(w[b, h], ref[2][0], (2 * ref[4] + 2.0 ** -18) * ref[2][0] + 2.0 ** -23 * ref[2][0], f"weights {b} {h}")


# ----------------------------------------------------------------- rotary positions
def left_behind(shape, dtype):
    """The allocator's next block of this size holds NaN."""
    for _ in range(4):
        torch.full(shape, math.nan, dtype=dtype, device="cuda")


@pytest.mark.parametrize("rot", [64, 128])
def test_new_packed_outputs_have_no_rows_left_as_they_were(rot):
    g = gen(48)
    plan = ffpa.rope_plan(rot)
    T, D = 900, 128
    q, k = randn(g, T, 4, D, dtype=torch.bfloat16), randn(g, T, 2, D, dtype=torch.bfloat16)
    for cu, there in ((ints(0, 300, 700), range(0, 700)), (ints(100, 300), range(100, 300)), (ints(0), range(0, 0)),
                      (ints(0, 0, 0), range(0, 0))):
        left_behind(q.shape, q.dtype)
        left_behind(k.shape, k.dtype)
        yq, yk = ffpa.varlen_rope(q, k, plan, cu)
        api.get_status()
        rows = torch.zeros(T, dtype=torch.bool, device="cuda")
        rows[there.start:there.stop] = True
        for x, y in ((q, yq), (k, yk)):
            assert bool((y[~rows] == 0).all()) and not bool(torch.isnan(y).any())
            given = torch.full_like(x, 3.0)
            r, _ = ffpa.varlen_rope(x, None, plan, cu, q_out=given)
            assert torch.equal(r[rows], y[rows]) and bool((r[~rows] == 3).all())
    # the gradient, too
    x = q.clone().requires_grad_()
    y, _ = ffpa.varlen_rope(x, None, plan, ints(0, 300, 700))
    left_behind(q.shape, q.dtype)
    (dx,) = torch.autograd.grad(y, x, torch.ones_like(y))
    assert bool((dx[700:] == 0).all()) and not bool(torch.isnan(dx).any())


@pytest.mark.parametrize("D", [64, 320, 512])
def test_packed_attention_with_a_plan_and_padding(D):
    """Rows behind the last sequence reach none of its results or gradients."""
    g = gen(49)
    plan = ffpa.rope_plan(64)
    T, pad = 437, 90
    cu = ints(0, 130, T)
    q, k, v = (randn(g, T + pad, h, D, dtype=torch.bfloat16) for h in (4, 2, 2))
    do = randn(g, T + pad, 4, D, dtype=torch.bfloat16)
    out = []
    for n in (T, T + pad):
        x = [t[:n].clone().requires_grad_() for t in (q, k, v)]
        for t in x:
            left_behind(t.shape, t.dtype)
        o = ffpa.varlen_attention(*x, cu, causal=True, rope=plan)
        out.append([t[:T] for t in (o, *torch.autograd.grad(o, x, do[:n]))])
    api.get_status()
    for x, y, what in zip(*out, ("o", "dq", "dk", "dv")):
        assert bool(torch.isfinite(y).all()) and torch.equal(x, y), what


def test_forward_mode_is_refused():
    g = gen(50)
    plan = ffpa.rope_plan(64)
    q, k = randn(g, 1, 4, 9, 64, dtype=torch.bfloat16), randn(g, 1, 2, 9, 64, dtype=torch.bfloat16)
    plain = ffpa.rope(q, k, plan)
    with forward_ad.dual_level():
        dual = [forward_ad.make_dual(x, torch.ones_like(x)) for x in (q, k)]
        for call in (lambda: ffpa.rope(dual[0], k, plan), lambda: ffpa.rope(q, dual[1], plan),
                     lambda: ffpa.rope(dual[0], None, plan), lambda: ffpa.attention(dual[0], k, k, rope=plan),
                     lambda: ffpa.varlen_rope(q[0], dual[1][0], plan, ints(0, 4)),
                     lambda: ffpa.varlen_attention(dual[0][0], dual[1][0], k[0], ints(0, 4), rope=plan)):
            with pytest.raises(RuntimeError):
                call()
        y = ffpa.rope(q, k, plan)  # tensors without a tangent
    assert all(torch.equal(a, b) for a, b in zip(y, plain))


# ----------------------------------------------------------------- eviction
@pytest.mark.parametrize("D", [64, 96])
def test_evict_in_place_of_narrow_heads(D):
    """More kv heads than SMs: slices of 64 head dims, 256 rows a batch and several batches."""
    g = gen(51)
    B, H, N, keep, recent = 16, 8, 1500, 701, 30
    lens = [1500 - 53 * i for i in range(B)]
    k, v = (randn(g, B, N, H, D, dtype=torch.bfloat16).transpose(1, 2) for _ in range(2))
    w = torch.rand((B, H, N), generator=g, device="cuda")
    k0, v0, w0 = k.clone(), v.clone(), w.cpu()
    n = ints(*lens)
    *_, kept = ffpa.kv_evict(k, v, w, n, keep, recent)
    api.get_status()
    assert n.tolist() == [min(x, keep) for x in lens]
    for b in range(B):
        for h in range(H):
            rows = kept_rows(w0[b, h].tolist(), lens[b], keep, recent)
            assert kept[b, h].tolist() == rows
            for x, x0 in ((k, k0), (v, v0)):
                assert torch.equal(x[b, h, :keep], x0[b, h, rows]) and torch.equal(x[b, h, keep:], x0[b, h, keep:])
