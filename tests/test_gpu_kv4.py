"""GPU tests of the 4-bit K/V cache: writing, reading back, and decode attention over it.

References: oracle/kv4.py (format and layout, bit for bit) and the fp64
attention oracle on the cached values, which are exact in bf16 and fp16.

Tolerances of the attention, derived and not tuned:
* O. The products run on exact operands (cached values; Q scaled by a power of
  two), so the errors are: P rounded to fp16 (half a step: 2^-11 relative; 2^-25
  absolute where P, scaled so that the row's largest is at least 2^6, is
  subnormal: under 2^-17 of the largest |V| for the lengths here), fp32
  accumulation (at most one rounding of 2^-23 per 16 keys and per join), and
  the rounding of the output to its type (eps / 2). With A = sum_j P_j |V_j| / l
  (the oracle's attention with |V|) and n keys:
    |dO| <= eps/2 |O| + (2^-11 + (n / 16 + 64) 2^-23) A + 2^-17 max|V|
* Scores in fp32: D / 16 accumulation steps of 2^-23 of M = scale max sum |q k|,
  which enters P and the sum alike: another 2 e_S A on O and e_S on the LSE, with
  e_S = (D / 16 + 8) 2^-23 M.
* LSE: e_S plus 2^-20 (the approximate exponential and logarithm, 2^-22 each),
  the sum's rounding (n / 16 + 64) 2^-23, and eight roundings of itself.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from head_dim_flash_gb300 import api
from oracle import kv4

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_dim_flash_gb300 import build

    build.build()
    oracle.build()


def block_tables(lens, page, rng, spare=2):
    """Shuffled pages for sequences of these lengths: (int32 table with -1 past each sequence, pages)."""
    blocks = [-(-n // page) for n in lens]
    order = rng.permutation(sum(blocks) + spare)
    table = np.full((len(lens), max(1, max(blocks))), -1, np.int32)
    used = 0
    for b, k in enumerate(blocks):
        table[b, :k] = order[used:used + k]
        used += k
    return table, len(order)


def random_cache(pages, page, H, D, rng):
    """Bytes as earlier tokens of ordinary size left them."""
    c = rng.integers(0, 256, (pages, 2, H, page // 16, D // 64, 576), dtype=np.uint8)
    c[..., 512:] = rng.integers(0x60, 0x78, c[..., 512:].shape, dtype=np.uint8)
    return c


def f64(x):
    return x.double().cpu().numpy()


def dev(x, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dt is None else t.to(dt)


# ------------------------------------------------------------------- writing
@pytest.mark.parametrize("dt,D,page,H,lo,new,transposed", [
    (BF16, 512, 64, 2, (0, 0, 0), (16, 64, 33), False),
    (FP16, 512, 64, 2, (5, 63, 100), (1, 1, 1), True),
    (BF16, 64, 16, 3, (0, 7, 15), (0, 17, 40), True),
    (FP16, 320, 48, 1, (47, 1, 16), (3, 95, 31), False),
    (BF16, 1024, 32, 1, (9, 0, 30), (20, 1, 5), True),
])
def test_write_matches_the_reference_byte_for_byte(dt, D, page, H, lo, new, transposed):
    rng = np.random.default_rng(D + page)
    table, pages = block_tables([a + n for a, n in zip(lo, new)], page, rng)
    ref = random_cache(pages, page, H, D, rng)
    cache = dev(ref)
    B, N = len(lo), max(new)
    x = [torch.from_numpy(rng.standard_normal((B, N, H, D)) * 3).to(dt).cuda() for _ in range(2)]
    k, v = (t.transpose(1, 2) if transposed else t.transpose(1, 2).contiguous() for t in x)
    api.kv4_write(cache, dev(table), k, v, start=dev(np.array(lo, np.int32)), count=dev(np.array(new, np.int32)))
    api.get_status()
    for b in range(B):
        kv4.write(ref, table[b], lo[b], f64(x[0][b, :new[b]]), f64(x[1][b, :new[b]]))
    assert np.array_equal(cache.cpu().numpy(), ref)  # the written cells, and every other byte as it was


@pytest.mark.parametrize("first,pitch", [(8, 208), (0, 200), (8, 200), (16, 224)])
def test_rows_on_sixteen_and_on_thirty_two_bytes(first, pitch):
    # rows that begin on an odd multiple of 16 bytes, every row or every other one, against rows on 32
    rng = np.random.default_rng(first + pitch)
    B, N, H, D, page = 2, 37, 2, 192, 32
    table, pages = block_tables([N, N + 3], page, rng)
    ref = random_cache(pages, page, H, D, rng)
    cache, t = dev(ref), dev(table)
    wide = [torch.from_numpy(rng.standard_normal((B, N, H, pitch))).to(BF16).cuda() for _ in range(2)]
    k, v = (w[..., first:first + D].transpose(1, 2) for w in wide)
    start, count = (dev(np.array(x, np.int32)) for x in ((0, 3), (N, N)))
    api.kv4_write(cache, t, k, v, start=start)
    out = [torch.full_like(w, -7.0) for w in wide]
    api.kv4_read(cache, t, count, start=start, k_out=out[0][..., first:first + D].transpose(1, 2),
                 v_out=out[1][..., first:first + D].transpose(1, 2))
    api.get_status()
    for b in range(B):
        lo = int(start[b])
        kv4.write(ref, table[b], lo, f64(k[b].transpose(0, 1)), f64(v[b].transpose(0, 1)))
        for got, want in zip(out, kv4.read(ref, table[b], lo, N)):
            assert np.array_equal(f64(got[b, ..., first:first + D]), want)
            assert (got[b, ..., :first] == -7).all() and (got[b, ..., first + D:] == -7).all()
    assert np.array_equal(cache.cpu().numpy(), ref)


@pytest.mark.parametrize("off", [1, 4, 8])
def test_inputs_that_do_not_begin_on_sixteen_bytes_are_copied(off):
    def at(shape):  # contiguous, 2 `off` bytes into an allocation
        n = math.prod(shape)
        return torch.randn(n + off, device="cuda").to(BF16)[off:].view(shape)

    Hkv, D, page, lens = 2, 128, 16, [20, 3]
    cu = torch.tensor([0, 20, 23], dtype=torch.int32, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    k, v, q = at((23, Hkv, D)), at((23, Hkv, D)), at((2, 4, 1, D))
    kd, vd = at((2, Hkv, 20, D)), at((2, Hkv, 20, D))
    calls = [lambda c, k, v: api.varlen_kv4_write(c, table, k, v, cu, 20), lambda c, k, v: api.kv4_write(c, table, k, v)]
    for call, x, y in zip(calls, (k, kd), (v, vd)):
        got, want = (api.kv4_cache(4, page, Hkv, D) for _ in range(2))
        call(got, x, y)
        call(want, x.clone(), y.clone())
        api.get_status()
        assert torch.equal(got, want)
    o, lse = api.decode_fwd_kv4(q, got, table, ln)
    want, want_l = api.decode_fwd_kv4(q.clone(), got, table, ln)
    api.get_status()
    assert torch.equal(o, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("start", [None, (3, 0, 50, 17)])
def test_packed_write_matches_the_reference(start):
    rng = np.random.default_rng(5)
    new, H, D, page = (19, 0, 70, 1), 2, 192, 32
    lo = start or (0, 0, 0, 0)
    table, pages = block_tables([a + n for a, n in zip(lo, new)], page, rng)
    ref = random_cache(pages, page, H, D, rng)
    cache = dev(ref)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = (torch.from_numpy(rng.standard_normal((cu[-1], H, D))).to(BF16).cuda() for _ in range(2))
    api.varlen_kv4_write(cache, dev(table), k, v, dev(cu), max(new),
                         start=None if start is None else dev(np.array(lo, np.int32)))
    api.get_status()
    for b in range(len(new)):
        kv4.write(ref, table[b], lo[b], f64(k[cu[b]:cu[b + 1]]), f64(v[cu[b]:cu[b + 1]]))
    assert np.array_equal(cache.cpu().numpy(), ref)


def test_every_finite_magnitude_as_a_group_scale():
    # one group per magnitude, beside random smaller values: all scale roundings of both types
    for dt in (FP16, BF16):
        bits = torch.arange(0, 0x7C00 if dt == FP16 else 0x7F80, dtype=torch.int32).to(torch.int16)
        amax = bits.view(dt).double().numpy()
        n = -(-len(amax) // 4)
        amax = np.resize(amax, (n, 1, 4, 1))
        rng = np.random.default_rng(1)
        x = amax * rng.choice([1, 1, .5, .25, 1 / 6, 5 / 6, 5 / 12, 7 / 12, 1 / 8, 1 / 24, -1, -.75, 0], (n, 1, 4, 16))
        x[..., 0] = amax[..., 0]
        with np.errstate(over="ignore"):
            k = torch.from_numpy(x.reshape(n, 1, 64)).to(dt).cuda()
        v = k.flip(-1).contiguous()
        cache = api.kv4_cache(1, -(-n // 16) * 16, 1, 64)
        table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        api.varlen_kv4_write(cache, table, k, v, cu, n)
        rk, rv = api.varlen_kv4_read(cache, table, cu, n, total=n, dtype=dt)
        api.get_status()
        for src, got in ((k, rk), (v, rv)):
            code, sc = kv4.quantize(f64(src))
            assert np.array_equal(f64(got), kv4.dequantize(code, sc))


def test_infinities_saturate_and_nan_is_zero():
    x = torch.randn(1, 2, 3, 128, dtype=torch.float32)
    x[0, 0, 0, 3], x[0, 0, 1, 20], x[0, 1, 2, 100] = math.inf, -math.inf, math.nan
    x[0, 1, 0, 64:80] = math.nan
    x = x.to(BF16).cuda()
    cache = api.kv4_cache(1, 16, 2, 128)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    api.kv4_write(cache, table, x, x)
    count = torch.tensor([3], dtype=torch.int32, device="cuda")
    k, v = api.kv4_read(cache, table, count, max_count=3)
    api.get_status()
    code, sc = kv4.quantize(f64(x))
    want = kv4.dequantize(code, sc)
    assert np.isfinite(want).all() and want[0, 0, 0, 3] == 61440 and want[0, 0, 1, 20] == -61440
    assert np.array_equal(f64(k), want) and np.array_equal(f64(v), want)


# ------------------------------------------------------------------- reading
@pytest.mark.parametrize("dt,D,page,H,start,count", [
    (BF16, 512, 64, 2, None, (100, 0, 64)),
    (FP16, 64, 16, 3, (1, 15, 16), (16, 1, 40)),
    (FP16, 640, 32, 1, (0, 31, 33), (5, 33, 2)),
])
def test_read_matches_the_reference_and_leaves_other_rows(dt, D, page, H, start, count):
    rng = np.random.default_rng(D)
    lo = start or (0,) * len(count)
    table, pages = block_tables([a + n for a, n in zip(lo, count)], page, rng)
    ref = random_cache(pages, page, H, D, rng)
    cache = dev(ref)
    B, N = len(count), max(count) + 3
    st = None if start is None else dev(np.array(lo, np.int32))
    wide = [torch.full((B, N, H, D + 64), -7.0, dtype=dt, device="cuda") for _ in range(2)]
    k, v = (w[..., :D].transpose(1, 2) for w in wide)
    api.kv4_read(cache, dev(table), dev(np.array(count, np.int32)), start=st, k_out=k, v_out=v)
    api.get_status()
    for b in range(B):
        for got, want in zip(wide, kv4.read(ref, table[b], lo[b], count[b])):
            assert np.array_equal(f64(got[b, :count[b], :, :D]), want)
            assert (got[b, count[b]:] == -7).all() and (got[..., D:] == -7).all()
    cu = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    pk, pv = api.varlen_kv4_read(cache, dev(table), dev(cu), max(count), total=int(cu[-1]) + 2, dtype=dt, start=st)
    api.get_status()
    for b in range(B):
        assert torch.equal(pk[cu[b]:cu[b + 1]], wide[0][b, :count[b], :, :D])
        assert torch.equal(pv[cu[b]:cu[b + 1]], wide[1][b, :count[b], :, :D])
    assert (pk[cu[-1]:] == 0).all() and (pv[cu[-1]:] == 0).all()
    assert np.array_equal(cache.cpu().numpy(), ref)


def test_cells_past_four_gigabytes():
    D, H, page = 512, 8, 64
    pages = (5 << 30) // (2 * H * 4 * 8 * 576)
    cache = torch.empty(pages, 2, H, 4, 8, 576, dtype=torch.uint8, device="cuda")
    cache[-3:] = 0
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(1, H, 100, D, device="cuda").to(BF16) for _ in range(2))
    api.kv4_write(cache, table, k, v)
    n = torch.tensor([100], dtype=torch.int32, device="cuda")
    rk, rv = api.kv4_read(cache, table, n, max_count=100)
    q = torch.randn(1, 8, 1, D, device="cuda").to(BF16)
    o, lse = api.decode_fwd_kv4(q, cache, table, n)
    api.get_status()
    for x, y in ((k, rk), (v, rv)):
        code, sc = kv4.quantize(f64(x))
        assert np.array_equal(f64(y), kv4.dequantize(code, sc))
    check_attention(q, rk, rv, [100], False, None, o, lse)


# ----------------------------------------------------------------- attention
def check_attention(q, k, v, lens, causal, scale, o, lse):
    """o, lse against the oracle on the cached values k, v [B, Hkv, >= len, D], per sequence."""
    B, Hq, Nq, D = q.shape
    Hkv = k.shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    o, lse = f64(o), f64(lse)
    assert np.isfinite(o).all()
    for b in range(B):
        n = lens[b]
        if n == 0:
            assert (o[b] == 0).all() and np.isneginf(lse[b]).all()
            continue
        qb, kb, vb = (t.cpu() for t in (q[b:b + 1], k[b:b + 1, :, :n], v[b:b + 1, :, :n]))
        o_ref, l_ref = oracle.attention_fwd(qb, kb, vb, causal, scale)
        mean, _ = oracle.attention_fwd(qb, kb, vb.abs(), causal, scale)
        qa = np.abs(f64(qb[0])).reshape(Hkv, -1, D)
        m = abs(scale) * np.einsum("hrd,hjd->hrj", qa, np.abs(f64(kb[0]))).max(-1).reshape(1, Hq, Nq)
        e_s = (D / 16 + 8) * 2.0 ** -23 * m
        tol = torch.finfo(q.dtype).eps / 2 * np.abs(o_ref) + 2.0 ** -17 * float(vb.abs().max()) + \
            (2.0 ** -11 + (n / 16 + 64) * 2.0 ** -23 + 2 * e_s[..., None]) * mean
        assert np.all(np.abs(o[b:b + 1] - o_ref) <= tol), float((np.abs(o[b:b + 1] - o_ref) / tol).max())
        none = np.isneginf(l_ref)
        assert np.array_equal(none, np.isneginf(lse[b:b + 1])) and (o[b:b + 1][none] == 0).all()
        with np.errstate(invalid="ignore"):
            lt = e_s + 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -23 + 8 * 2.0 ** -24 * np.abs(l_ref)
            ok = none | (np.abs(lse[b:b + 1] - l_ref) <= lt)
        assert ok.all(), float(np.abs(lse[b:b + 1] - l_ref)[~none].max())


def decode_case(lens, Hkv, G, Nq, D, page, causal, dt, seed=0, scale=None, q_amp=1.0, k_amp=1.0, width=0):
    rng = np.random.default_rng(seed)
    table, pages = block_tables(lens, page, rng)
    if width:
        table = np.concatenate([table, np.full((len(lens), width), -1, np.int32)], 1)
    B, n = len(lens), max(1, max(lens))
    cache = torch.full((pages, 2, Hkv, page // 16, D // 64, 576), 255, dtype=torch.uint8, device="cuda")
    k, v = (torch.from_numpy(rng.standard_normal((B, Hkv, n, D)) * a).to(dt).cuda() for a in (k_amp, 1.0))
    q = torch.from_numpy(rng.standard_normal((B, Hkv * G, Nq, D)) * q_amp).to(dt).cuda()
    t, ln = dev(table), dev(np.array(lens, np.int32))
    api.kv4_write(cache, t, k, v, count=ln)   # every other cell holds bytes that stand for NaN
    rk, rv = api.kv4_read(cache, t, ln, max_count=n, dtype=dt)
    o, lse = api.decode_fwd_kv4(q, cache, t, ln, causal, scale)
    api.get_status()
    check_attention(q, rk, rv, lens, causal, scale, o, lse)
    return q, cache, t, ln, o, lse


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 1000])
def test_decode_lengths(n):
    decode_case([n, 40], 2, 4, 1, 512, 64, False, BF16, seed=n)


@pytest.mark.parametrize("D", [64, 128, 192, 256, 320, 384, 448, 512, 576, 640, 704, 832, 1024])
def test_decode_head_dims(D):
    decode_case([300, 77], 2, 4, 1, D, 32, False, FP16, seed=D)
    decode_case([129], 1, 3, 4, D, 16, True, BF16, seed=D + 1)


@pytest.mark.parametrize("D", [768, 960])
def test_decode_head_dims_of_twelve_and_fifteen_chunks(D):
    # eight and sixteen rows, across parts and pages
    decode_case([300, 77], 2, 4, 1, D, 32, False, FP16, seed=D)
    decode_case([129], 1, 3, 4, D, 16, True, BF16, seed=D + 1)
    decode_case([1500, 17, 0, 790], 2, 8, 1, D, 48, False, BF16, seed=D + 2)
    decode_case([1500, 17, 0, 790], 1, 5, 3, D, 112, True, FP16, seed=D + 3)


@pytest.mark.parametrize("G,Nq", [(1, 1), (3, 1), (8, 1), (16, 1), (32, 1), (4, 2), (4, 4), (5, 7), (1, 40), (16, 4)])
@pytest.mark.parametrize("causal", [False, True])
def test_decode_groups_and_rows(G, Nq, causal):
    decode_case([5, 200, 1, 131], 2, G, Nq, 320, 16, causal, BF16, seed=G * Nq)


@pytest.mark.parametrize("page", [16, 48, 64, 256, 4096])
def test_decode_pages_and_ragged_lengths(page):
    decode_case([1, 0, 700, 16, 0, 4095, 333], 1, 4, 1, 256, page, False, FP16, seed=page, width=3)


@pytest.mark.parametrize("D", [64, 128, 320, 512, 896, 1024])
@pytest.mark.parametrize("page", [16, 48, 112, 2048])
def test_decode_steps_over_pages(D, page):
    # steps that begin and end anywhere in a page, and span many; short and long groups, eight and sixteen rows
    lens = [1500, 17, 0, 790]
    decode_case(lens, 2, 2, 1, D, page, False, BF16, seed=D + page)
    decode_case(lens, 1, 5, 3, D, page, True, FP16, seed=2 * D + page)


def test_decode_up_to_the_last_token_an_int_can_count():
    """2^31 - 1 tokens on two pages: every block is the first, the last block the second, whose own last token
    (position 2^31 - 1, one past the sequence) would outweigh all others.

    The oracle is the softmax with every key counted as often as it occurs. 16 groups on each of more than 140 SMs
    share 2^27 strips: below 2^16 per group, and one addition per strip to a lane's sum (2^-24 each) and to a product
    (2^-23): at most 2^-8 of the sum and 2^-7 of A; P's rounding is 2^-11 of A, the output's 2^-9 of itself."""
    D, page, n = 64, 1 << 20, (1 << 31) - 1
    blocks = 1 << 11
    cache = api.kv4_cache(2, page, 1, D)
    q = torch.randn(1, 4, 1, D, device="cuda").to(BF16)
    k, v = (torch.randn(1, 1, page, D, device="cuda").to(BF16) for _ in range(2))
    both = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    k2 = k.clone()
    k2[0, 0, -1] = 40 * q.sum(1)[0, 0]
    for p, kk in ((0, k), (1, k2)):
        api.kv4_write(cache, both[p:p + 1], kk, v)
    table = torch.zeros(1, blocks, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    o, lse = api.decode_fwd_kv4(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    rk, rv = api.kv4_read(cache, both[:1], torch.tensor([page], dtype=torch.int32, device="cuda"), max_count=page)
    api.get_status()
    s = q[0, :, 0].double() @ rk[0, 0].double().T / 8
    w = torch.full((page,), float(blocks), dtype=torch.float64, device="cuda")
    w[-1] -= 1
    e = (s - s.amax(1, keepdim=True)).exp() * w
    l = e.sum(1, keepdim=True)
    want, mean = e @ rv[0, 0].double() / l, e @ rv[0, 0].double().abs() / l
    m = (q[0, :, 0].double().abs() @ rk[0, 0].double().abs().T).amax(1, keepdim=True) / 8
    e_s = (D / 16 + 8) * 2.0 ** -23 * m
    assert ((o[0, :, 0].double() - want).abs() <= 2.0 ** -9 * want.abs() + (2.0 ** -7 + 2.0 ** -8 + 2.0 ** -11 + 2 * e_s) * mean +
            2.0 ** -17 * rv.abs().max().double()).all()
    assert ((lse[0, :, 0:1].double() - (l.log() + s.amax(1, keepdim=True))).abs() <= 2.0 ** -8 + 2.0 ** -20 + e_s +
            2.0 ** -19).all()


def test_decode_long_context_on_few_heads():
    decode_case([40000], 1, 2, 1, 128, 64, False, BF16, seed=1)
    decode_case([9000], 1, 16, 2, 1024, 128, True, FP16, seed=2)


def test_decode_many_short_sequences():
    rng = np.random.default_rng(0)
    decode_case([int(x) for x in rng.integers(0, 70, 300)], 3, 2, 1, 64, 16, False, BF16, seed=3)


def test_decode_rows_without_keys():
    # causal with fewer cached tokens than query rows
    q, *_, o, lse = decode_case([3, 8, 1], 1, 2, 8, 512, 16, True, BF16)
    assert torch.isneginf(lse[0, :, :5]).all() and (o[0, :, :5] == 0).all()


@pytest.mark.parametrize("scale,q_amp,k_amp", [(None, 8.0, 4.0), (0.0, 1, 1), (-0.05, 1, 1), (3.0, 1, 1)])
def test_decode_large_and_odd_scores(scale, q_amp, k_amp):
    decode_case([500, 90], 2, 4, 2, 192, 32, True, BF16, seed=9, scale=scale, q_amp=q_amp, k_amp=k_amp)


@pytest.mark.parametrize("q_amp,k_amp", [(2.0 ** 60, 2.0 ** -8), (2.0 ** -60, 2.0 ** 10), (2.0 ** -100, 1.0)])
def test_decode_queries_outside_the_range_of_fp16(q_amp, k_amp):
    s = 1 / (math.sqrt(128) * q_amp * k_amp)
    decode_case([200], 1, 4, 1, 128, 32, False, BF16, seed=11, scale=s, q_amp=q_amp, k_amp=k_amp)


def test_decode_growing_scores():
    # the row maximum grows with every key, far past where a kept reference would overflow
    D, n = 64, 600
    k = torch.zeros(1, 1, n, D)
    k[0, 0, :, 0] = torch.arange(n) // 4 * 0.5
    k = k.to(BF16).cuda()
    v = torch.randn(1, 1, n, D).to(BF16).cuda()
    q = torch.zeros(1, 4, 1, D, dtype=BF16, device="cuda")
    q[0, :, 0, 0] = torch.tensor([1.0, 4.0, -4.0, 16.0])
    cache = api.kv4_cache(n // 16 + 1, 16, 1, D)
    t = torch.arange(n // 16 + 1, dtype=torch.int32, device="cuda").view(1, -1)
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    api.kv4_write(cache, t, k, v)
    rk, rv = api.kv4_read(cache, t, ln, max_count=n)
    o, lse = api.decode_fwd_kv4(q, cache, t, ln, False, 1.0)
    api.get_status()
    check_attention(q, rk, rv, [n], False, 1.0, o, lse)


def test_decode_a_row_that_is_not_finite_stays_alone():
    q, cache, t, ln, o, lse = decode_case([100, 50], 2, 4, 2, 128, 16, True, BF16, seed=4)
    q[0, 3, 1, 17], q[1, 0, 0, 5] = math.nan, math.inf
    o2, lse2 = api.decode_fwd_kv4(q, cache, t, ln, True)
    api.get_status()
    same = torch.ones(2, 8, 2, dtype=torch.bool)
    same[0, 3, 1] = same[1, 0, 0] = False
    assert torch.equal(o2[same.cuda()], o[same.cuda()]) and torch.equal(lse2[same.cuda()], lse[same.cuda()])
    assert torch.isnan(o2[0, 3, 1]).all() and not torch.isfinite(o2[1, 0, 0]).any()


@pytest.mark.parametrize("G,Nq", [(1, 1), (3, 1), (4, 1), (2, 2)])
@pytest.mark.parametrize("D,n", [(64, 32), (128, 47), (320, 64), (512, 32), (1024, 34)])
def test_decode_of_up_to_four_rows_in_fp16_rounds_its_output_alone(G, Nq, D, n):
    """P in 22 bits, where values cancel: |O| is far below A = sum P |V| / l, so 11 bits of P would show.

    P is fp16 and an fp16 remainder: 2^-22 of itself, or 2^-25 where the remainder is subnormal, next to a largest P
    of at least 2^6 (n 2^-31 max|V|). The rest is as at the top of this file."""
    rng = np.random.default_rng(D + n + G)
    page, Hkv, B = 16, 2, 2
    lens = [n, n]
    table, pages = block_tables(lens, page, rng)
    signs = np.where(np.arange(n) % 2, 1.0, -1.0)
    v = np.stack([rng.permutation(signs) for _ in range(B * Hkv * D)]).reshape(B, Hkv, D, n).transpose(0, 1, 3, 2)
    k, v = dev(rng.standard_normal((B, Hkv, n, D)), FP16), dev(v, FP16)
    q = dev(0.1 * rng.standard_normal((B, Hkv * G, Nq, D)), FP16)
    cache, t, ln = api.kv4_cache(pages, page, Hkv, D), dev(table), dev(np.array(lens, np.int32))
    api.kv4_write(cache, t, k, v)
    rk, rv = api.kv4_read(cache, t, ln, max_count=n, dtype=FP16)
    o, lse = api.decode_fwd_kv4(q, cache, t, ln)
    api.get_status()
    check_attention(q, rk, rv, lens, False, None, o, lse)
    want, _ = oracle.attention_fwd(q.cpu(), rk.cpu(), rv.cpu(), False, 1 / math.sqrt(D))
    mean, _ = oracle.attention_fwd(q.cpu(), rk.cpu(), rv.abs().cpu(), False, 1 / math.sqrt(D))
    qa = np.abs(f64(q)).reshape(B, Hkv, G * Nq, D)
    m = np.einsum("bhrd,bhjd->bhrj", qa, np.abs(f64(rk))).max(-1).reshape(B, Hkv * G, Nq, 1) / math.sqrt(D)
    e_s = (D / 16 + 8) * 2.0 ** -23 * m
    tol = torch.finfo(FP16).eps / 2 * np.abs(want) + n * 2.0 ** -31 * float(rv.abs().max()) + \
        (2.0 ** -22 + (n / 16 + 64) * 2.0 ** -23 + 2 * e_s) * mean
    off = np.abs(f64(o) - want) / tol
    assert off.max() <= 1, off.max()


def test_decode_strided_views_and_shared_pages():
    rng = np.random.default_rng(2)
    B, Hkv, G, Nq, D, page = 3, 2, 4, 2, 256, 32
    cache = dev(random_cache(6, page, Hkv, D, rng))
    big = dev(np.array([[4, 1, 3, -1, 9], [4, 1, 0, 5, 9], [4, 2, -1, -1, 9], [9] * 5], np.int32))
    table = big[:3, :4]   # rows of a wider table; all sequences share page 4
    lens = [70, 128, 40]
    ln = dev(np.array(lens, np.int32))
    q = torch.randn(B, Nq, Hkv * G, D, device="cuda").to(FP16).transpose(1, 2)
    wide = torch.full((B, Nq, Hkv * G, D + 64), float("nan"), dtype=FP16, device="cuda")
    o, lse = api.decode_fwd_kv4(q, cache, table, ln, True, out=wide[..., :D].transpose(1, 2))
    k, v = api.kv4_read(cache, table, ln, max_count=128, dtype=FP16)
    api.get_status()
    assert torch.isnan(wide[..., D:]).all()
    check_attention(q, k, v, lens, True, None, o, lse)


def test_decode_is_deterministic_and_takes_any_workspace_contents():
    q, cache, t, ln, o, lse = decode_case([3000, 17, 900, 0], 2, 4, 1, 512, 64, False, BF16, seed=6)
    from head_dim_flash_gb300 import _ffi

    n = int(_ffi.ffpa_decode_kv4_workspace_bytes(_ffi.BF16, 4, 8, 2, 1, 512))
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        o2, lse2 = api.decode_fwd_kv4(q, cache, t, ln, workspace=ws)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
    api.get_status()


# ------------------------------------------------------------ used together
def test_prompt_then_decoding_steps():
    """A ragged prompt enters the cache and attends over it through the packed kernels; then tokens one by one."""
    lens, Hkv, G, D, page, steps = [37, 130, 1], 2, 2, 320, 16, 5
    rng = np.random.default_rng(8)
    table, pages = block_tables([n + steps for n in lens], page, rng)
    t = dev(table)
    cache = api.kv4_cache(pages, page, Hkv, D)
    cu = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    T = sum(lens)
    k, v = (torch.randn(T, Hkv, D, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn(T, Hkv * G, D, device="cuda").to(BF16)
    api.varlen_kv4_write(cache, t, k, v, cu, max(lens))
    ck, cv = api.varlen_kv4_read(cache, t, cu, max(lens), total=T)
    o, _ = api.varlen_attention(q, ck, cv, cu, causal=True, return_lse=True)
    api.get_status()
    ref, _ = oracle.varlen_fwd(q.cpu(), ck.cpu(), cv.cpu(), cu.cpu(), causal=True)
    assert np.abs(f64(o) - ref).max() <= 2e-2
    now = dev(np.array(lens, np.int32))
    for s in range(steps):
        k1, v1 = (torch.randn(3, Hkv, 1, D, device="cuda").to(BF16) for _ in range(2))
        q1 = torch.randn(3, Hkv * G, 1, D, device="cuda").to(BF16)
        api.kv4_write(cache, t, k1, v1, start=now)
        now = now + 1
        o, lse = api.decode_fwd_kv4(q1, cache, t, now, causal=True)
        full = [n + s + 1 for n in lens]
        rk, rv = api.kv4_read(cache, t, now, max_count=max(full))
        api.get_status()
        check_attention(q1, rk, rv, full, True, None, o, lse)
        for b in range(3):   # the prompt's tokens are still what they were
            m = min(lens[b], 20)
            assert torch.equal(rk[b, :, :m].transpose(0, 1), ck[int(cu[b]):int(cu[b]) + m])


def test_steps_captured_into_graphs_and_replayed():
    """Two captured steps (write, decode) that share nothing but the cache; lengths move between replays."""
    Hkv, G, D, page, B = 2, 4, 128, 16, 2
    cache = api.kv4_cache(20, page, Hkv, D)
    t = torch.arange(20, dtype=torch.int32, device="cuda").view(B, 10)
    start = torch.tensor([5, 0], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(B, Hkv, 1, D, device="cuda").to(FP16) for _ in range(2))
    q = torch.randn(B, Hkv * G, 1, D, device="cuda").to(FP16)
    api.kv4_write(cache, t, *(torch.randn(B, Hkv, 5, D, device="cuda").to(FP16) for _ in range(2)))
    outs, graphs = [], []
    side = torch.cuda.Stream()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            api.kv4_write(cache, t, k, v, start=start)
            outs.append(api.decode_fwd_kv4(q, cache, t, start + 1))
        graphs.append(g)
    for step in range(40):
        for x in (k, v, q):
            x.copy_(torch.randn_like(x))
        graphs[step % 2].replay()
        start += 1
        if step % 13 == 0:
            lens = start.tolist()
            rk, rv = api.kv4_read(cache, t, start, max_count=max(lens), dtype=FP16)
            api.get_status()
            check_attention(q, rk, rv, lens, False, None, *outs[step % 2])


def test_another_stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        decode_case([300, 20], 1, 4, 1, 128, 32, False, BF16, seed=21)
    torch.cuda.current_stream().wait_stream(s)


def test_calls_at_once_on_two_streams():
    """Decodes with their own workspaces, and writes to other pages of the same cache, at the same time."""
    rng = np.random.default_rng(30)
    Hkv, G, D, page = 2, 4, 320, 32
    lens = [[900, 3, 411], [64, 2000, 5]]
    table, pages = block_tables(lens[0] + lens[1], page, rng)
    cache = dev(random_cache(pages + 1, page, Hkv, D, rng))
    spare = torch.full((1, 1), pages, dtype=torch.int32, device="cuda")
    x = torch.randn(1, Hkv, page, D, device="cuda").to(BF16)
    q = torch.randn(3, Hkv * G, 2, D, device="cuda").to(BF16)
    tables = [dev(table[:3]), dev(table[3:])]
    ln = [dev(np.array(n, np.int32)) for n in lens]
    want = [api.decode_fwd_kv4(q, cache, tables[i], ln[i], True) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(api.decode_fwd_kv4(q, cache, tables[i], ln[i], True))
                if i:
                    api.kv4_write(cache, spare, x, x)
    torch.cuda.synchronize()
    api.get_status()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_calls_read_what_the_kernels_before_them_write():
    """A chain whose every call reads the outputs of the one before it, against the same calls one at a time: the
    forward's kernels let the next one start before they end."""
    torch.manual_seed(5)
    B, H, N, D, page = 1, 4, 1000, 256, 64
    x = [torch.randn(B, H, N, D, device="cuda").to(BF16) for _ in range(3)]
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(1, 16)
    n = torch.tensor([N], dtype=torch.int32, device="cuda")

    def chain(wait):
        cache = api.kv4_cache(16, page, H, D)
        q, k, v = x
        for _ in range(4):
            k, _ = api.fwd(q, k, v, True)
            wait()
            api.kv4_write(cache, table, k, k)
            wait()
            o, lse = api.decode_fwd_kv4(k[:, :, -2:], cache, table, n, True)
            wait()
            api.kv4_write(cache, table, o, o, start=n - 2)
            wait()
            k, v = api.kv4_read(cache, table, n, max_count=N)
            wait()
            v, _ = api.fwd(v, k, v)
            wait()
        return cache, k, v, o, lse

    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        got = chain(lambda: None)
        api.get_status()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_results_take_the_place_of_their_inputs():
    # the rows of a unit are read before any of them is written
    q, cache, t, ln, o, lse = decode_case([3000, 17, 900, 0], 2, 8, 2, 256, 64, True, BF16, seed=31)
    api.decode_fwd_kv4(q, cache, t, ln, True, out=q, lse=lse)
    api.get_status()
    assert torch.equal(q, o)


# ----------------------------------------------------------------- refusals
def test_a_cache_without_pages_holds_no_tokens():
    cache = api.kv4_cache(0, 16, 1, 128)
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    ln = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, 1, 128, device="cuda").to(BF16)
    x = torch.randn(2, 1, 3, 128, device="cuda").to(BF16)
    for call in (lambda: api.decode_fwd_kv4(q, cache, table, ln), lambda: api.kv4_read(cache, table, ln, max_count=3),
                 lambda: api.kv4_write(cache, table, x, x, count=ln)):
        out = call()
        with pytest.raises(ValueError, match="sequence 0"):
            api.get_status()
        if out is not None:
            assert (out[0][1] == 0).all()


def test_workspace_refusals():
    cache = api.kv4_cache(4, 16, 2, 128)
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    ln = torch.tensor([3, 3], dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 4, 1, 128, dtype=BF16, device="cuda")
    ws = api.decode_kv4_workspace(q, cache)
    big = torch.empty(2 * ws.numel(), dtype=torch.uint8, device="cuda")
    for bad in (ws.cpu(), big[::2], ws[:-1], big[8:]):   # elsewhere, strided, too small, not aligned
        with pytest.raises(ValueError, match="workspace"):
            api.decode_fwd_kv4(q, cache, table, ln, workspace=bad)
    api.decode_fwd_kv4(q, cache, table, ln, workspace=ws)
    api.get_status()


@pytest.mark.parametrize("bad", ["page", "negative page", "length", "negative length"])
def test_a_sequence_outside_its_cache_is_an_error_and_others_are_not(bad):
    rng = np.random.default_rng(12)
    cache = dev(random_cache(8, 16, 1, 128, rng))
    table = torch.tensor([[0, 1, 2, 3], [4, 5, 6, 7], [3, 2, 1, 0]], dtype=torch.int32, device="cuda")
    ln = torch.tensor([50, 64, 33], dtype=torch.int32, device="cuda")
    q = torch.randn(3, 4, 1, 128, device="cuda").to(BF16)
    good, good_l = api.decode_fwd_kv4(q, cache, table, ln)
    rk, rv = api.kv4_read(cache, table, ln, max_count=64)
    api.get_status()
    before = cache.clone()
    if "page" in bad:
        table[1, 2] = 8 if bad == "page" else -1
    else:
        ln[1] = 65 if bad == "length" else -2
    x = torch.randn(3, 1, 64, 128, device="cuda").to(BF16)
    for call in (lambda: api.decode_fwd_kv4(q, cache, table, ln), lambda: api.kv4_read(cache, table, ln, max_count=64),
                 lambda: api.kv4_write(cache, table, x, x, count=ln)):
        out = call()
        with pytest.raises(ValueError, match="sequence 1"):
            api.get_status()
        api.get_status()  # cleared
        if out is not None and out[0].dim() == 4 and out[0].shape == good.shape:
            assert torch.equal(out[0][::2], good[::2]) and torch.equal(out[1][::2], good_l[::2])
        elif out is not None:
            assert torch.equal(out[0][::2], rk[::2]) and torch.equal(out[1][::2], rv[::2])
    if "length" in bad:  # nothing of the refused sequence was written
        assert torch.equal(cache[4:], before[4:])


def test_python_refusals():
    cache = api.kv4_cache(4, 16, 2, 128)
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    ln = torch.tensor([3, 3], dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 4, 1, 128, dtype=BF16, device="cuda")
    k = torch.zeros(2, 2, 4, 128, dtype=BF16, device="cuda")
    cases = [
        (ValueError, lambda: api.kv4_cache(4, 24, 2, 128)),
        (NotImplementedError, lambda: api.kv4_cache(4, 16, 2, 96)),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache.float(), table, ln)),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache[:, :, :1], table, ln)),      # not contiguous
        (ValueError, lambda: api.decode_fwd_kv4(q, cache, table.long(), ln)),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache, table[:1], ln)),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache, table.cpu(), ln)),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache, table.t(), ln)),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache, table, ln.long())),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache, table, ln[:1])),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache, table, ln.cpu())),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache, table, None)),
        (ValueError, lambda: api.decode_fwd_kv4(q[..., :64], cache, table, ln)),
        (ValueError, lambda: api.decode_fwd_kv4(q[:, :3], cache, table, ln)),         # 3 heads over 2
        (NotImplementedError, lambda: api.decode_fwd_kv4(q.float(), cache, table, ln)),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache, table, ln, scale=math.nan)),
        (ValueError, lambda: api.decode_fwd_kv4(q, cache, table, ln, out=q[:1])),
        (ValueError, lambda: api.kv4_write(cache, table, k[:, :1], k[:, :1])),
        (ValueError, lambda: api.kv4_write(cache, table, k, k[:, :, :2])),
        (ValueError, lambda: api.kv4_write(cache, table, k, k.half())),
        (ValueError, lambda: api.kv4_write(cache, table, k.cpu(), k.cpu())),
        (NotImplementedError, lambda: api.kv4_write(cache, table, k.float(), k.float())),
        (ValueError, lambda: api.kv4_write(cache, table, k, k, start=ln.long())),
        (ValueError, lambda: api.kv4_read(cache, table, ln)),
        (ValueError, lambda: api.kv4_read(cache, table, ln, max_count=4, k_out=k, v_out=k.clone())),
        (ValueError, lambda: api.kv4_read(cache, table, None, max_count=4)),
        (ValueError, lambda: api.varlen_kv4_read(cache, table, ln, 4, k_out=k[0].transpose(0, 1))),
    ]
    for error, call in cases:
        with pytest.raises(error):
            call()
    api.get_status()


def test_nothing_to_do():
    cache = api.kv4_cache(4, 16, 2, 128)
    z = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    o, lse = api.decode_fwd_kv4(torch.zeros(0, 4, 1, 128, dtype=BF16, device="cuda"), cache, z, e)
    assert o.numel() == 0 and lse.numel() == 0
    api.kv4_write(cache, z, *(torch.zeros(0, 2, 3, 128, dtype=BF16, device="cuda") for _ in range(2)), start=e)
    t = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv4_write(cache, t, *(torch.zeros(1, 2, 0, 128, dtype=BF16, device="cuda") for _ in range(2)))
    k, _ = api.kv4_read(cache, t, n, max_count=0)
    assert k.shape == (1, 2, 0, 128)
    # no blocks at all: every sequence is empty
    t0 = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    o, lse = api.decode_fwd_kv4(torch.ones(2, 4, 1, 128, dtype=BF16, device="cuda"), cache, t0,
                                torch.zeros(2, dtype=torch.int32, device="cuda"))
    api.get_status()
    assert (o == 0).all() and torch.isneginf(lse).all() and (cache == 0).all()
