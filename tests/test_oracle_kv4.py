"""Pins of the 4-bit cache reference in oracle/kv4.py, independent of it.

* the scale bytes against 16-bit floats (a library format: a scale byte is the
  eight bits behind their sign);
* ties, saturation and small groups from the format's definition, by hand;
* every level times every scale is exact in bf16 and fp16;
* a written token's bytes by hand for one place, and write / read as inverses
  with every byte of a tile used once.
"""
import numpy as np
import pytest
import torch

from oracle import kv4


def test_scale_bytes_are_sixteen_bit_floats():
    codes = np.arange(0xF8, dtype=np.uint16)
    ref = torch.from_numpy((codes << 7).view(np.int16)).view(torch.float16).double().numpy()
    assert np.array_equal(kv4.SCALES, ref)


def test_cached_values_are_exact_in_both_types():
    v = torch.from_numpy(np.outer(kv4.LEVELS, kv4.SCALES[kv4.SCALES <= 10240]))
    for dt in (torch.bfloat16, torch.float16):
        assert torch.equal(v.to(dt).double(), v)


def test_rounding_by_hand():
    x = np.zeros(16)
    x[:12] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -2.5, 0.26, 5.01]
    code, sc = kv4.quantize(x)
    assert kv4.SCALES[sc[0]] == 1.0
    # ties go to the even code
    want = [6, 0, 1, 1, 2, 2, 4, 4, 0, -2, 0.5, 6] + [0] * 4
    assert np.array_equal(kv4.dequantize(code, sc), want)
    assert code[8] == 8  # the sign of a value that rounds to zero stays


@pytest.mark.parametrize("amax,scale", [
    (6 * 1.0625, 1.0),        # a tie of the scale: 1.0625 between 1 and 1.125, to the even mantissa
    (6 * 1.1875, 1.25),
    (6 * 1.0626, 1.125),
    (6 * 1.9999, 2.0),        # carries into the next exponent
    (1e9, 10240.0),
    (np.inf, 10240.0),
    (6 * 2.0 ** -17, 2.0 ** -17),
    (3 * 2.0 ** -17, 0.0),    # a tie with zero
    (3.1 * 2.0 ** -17, 2.0 ** -17),
    (0.0, 0.0),
])
def test_scales_by_hand(amax, scale):
    x = np.zeros(16)
    x[3] = -amax
    code, sc = kv4.quantize(x)
    assert kv4.SCALES[sc[0]] == scale
    v = kv4.dequantize(code, sc)
    assert np.isfinite(v).all()
    assert v[3] == -6 * scale or amax < 1


@pytest.mark.parametrize("amax,value", [
    (6 * 2.0 ** -17, 6 * 2.0 ** -17),
    (3 * 2.0 ** -17, 0.0),              # a scale that ties with zero
    (3.1 * 2.0 ** -17, 3 * 2.0 ** -17),     # level 3, the nearest to 3.1 scales
    (5 * 2.0 ** -17, 4 * 2.0 ** -17),       # a tie between levels 4 and 6, to the even code
    (5.1 * 2.0 ** -17, 6 * 2.0 ** -17),
    (9 * 2.0 ** -17, 8 * 2.0 ** -17),       # 1.5 steps, a tie, to two: 4.5 scales, level 4
    (6 * 7 * 2.0 ** -17, 42 * 2.0 ** -17),
    (6 * 2.0 ** -14, 6 * 2.0 ** -14),
    (0.75, 0.75),
    (0.0, 0.0),
])
def test_largest_values_of_small_groups_by_hand(amax, value):
    for sign in (1, -1):
        x = np.zeros(16)
        x[3] = sign * amax
        v = kv4.dequantize(*kv4.quantize(x))
        assert v[3] == sign * value and not v[:3].any() and not v[4:].any()


def test_not_a_number_counts_as_zero():
    x = np.linspace(-1, 1, 16)
    y = x.copy()
    y[5] = np.nan
    x[5] = 0
    for a, b in zip(kv4.quantize(x), kv4.quantize(y)):
        assert np.array_equal(a, b)


def test_bytes_of_one_token_by_hand():
    # token 11 of a page, D = 128: place 11 of its strip, s % 8 = 3, s / 8 = 1
    cache = np.zeros((2, 2, 1, 1, 2, 576), np.uint8)
    k = np.zeros((1, 1, 128))
    v = np.zeros((1, 1, 128))
    k[0, 0, 64 + 37] = 6.0   # second tile, x = 37: group 2, byte (37 % 16) / 2 = 2, high nibble
    v[0, 0, 22] = -3.0       # first tile, x = 22: eighth 2, byte (22 % 8) / 2 = 3, low nibble
    kv4.write(cache, [1], 11, k, v)
    want = np.zeros_like(cache)
    want[1, 0, 0, 0, 1, (3 * 4 + 2) * 16 + 8 + 2] = 0x70
    want[1, 0, 0, 0, 1, 512 + 3 * 8 + 2 * 2 + 1] = 15 << 3           # scale 1
    want[1, 1, 0, 0, 0, (2 * 4 + 1) * 16 + 8 + 4 + 3] = 0x0F         # s % 2 = 1
    want[1, 1, 0, 0, 0, 512 + 1 * 16 + 1 * 4 + 2 + 1] = 14 << 3      # scale 0.5
    assert np.array_equal(cache, want)


@pytest.mark.parametrize("kv", [0, 1])
def test_a_tile_uses_every_byte_once(kv):
    at, odd, at_s = kv4._bytes(kv, np.arange(16), 128)
    used = np.concatenate([(2 * at + odd).ravel(), (2 * at_s).ravel(), (2 * at_s + 1).ravel()])
    assert np.array_equal(np.sort(used), np.arange(2 * 2 * 576))


def test_write_then_read():
    rng = np.random.default_rng(3)
    cache = rng.integers(0, 256, (5, 2, 2, 2, 1, 576), dtype=np.uint8)
    before = cache.copy()
    k, v = rng.standard_normal((2, 45, 2, 64))
    table = [3, 0, 4]
    kv4.write(cache, table, 21, k, v)
    rk, rv = kv4.read(cache, table, 21, 45)
    for x, y in ((k, rk), (v, rv)):
        code, sc = kv4.quantize(x)
        assert np.array_equal(y, kv4.dequantize(code, sc))
        # half a step of the widest gap (4 to 6), with a scale that is at most 1/16 under amax / 6
        assert np.all(np.abs(x - y) <= np.repeat(kv4.SCALES[sc], 16, -1).reshape(x.shape) * (1 + 6 / 16))
    # cells of other tokens keep their bytes
    kv4.write(cache, table, 21, *(kv4.read(before, table, 21, 45)))
    assert np.array_equal(cache[1:3], before[1:3])
    k0, _ = kv4.read(cache, table, 0, 21)
    k1, _ = kv4.read(before, table, 0, 21)
    assert np.array_equal(np.nan_to_num(k0), np.nan_to_num(k1))
