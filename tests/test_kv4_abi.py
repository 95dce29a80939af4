"""Host-side checks of the 4-bit cache's C entry points, without a GPU: every
invalid call is refused with its status and a message before any device work."""
import pytest

from tests.test_abi import FAKE, _view, lib  # noqa: F401  (the library where no GPU is visible)


def _cache(data=FAKE, pages=8, page_size=16, table=FAKE, blocks=4, stride=4):
    from head_dim_flash_gb300 import _ffi

    return _ffi.Kv4Cache(data, pages, page_size, table, blocks, stride)


VIEW = dict(sb=2 * 8 * 512, sh=8 * 512, sn=512)


def write(lib, dt=0, k=None, v=None, cache=None, start=FAKE, count=FAKE, B=2, Hkv=2, N=8, D=512):
    k, v = (_view(**VIEW) if x is None else x for x in (k, v))
    return lib.ffpa_kv4_write(dt, k, v, cache or _cache(), start, count, B, Hkv, N, D, None)


def read(lib, dt=0, k=None, v=None, cache=None, start=FAKE, count=FAKE, B=2, Hkv=2, N=8, D=512):
    k, v = (_view(**VIEW) if x is None else x for x in (k, v))
    return lib.ffpa_kv4_read(dt, cache or _cache(), k, v, start, count, B, Hkv, N, D, None)


def decode(lib, dt=0, q=None, o=None, cache=None, lens=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40, B=2, Hq=4, Hkv=2,
           Nq=1, D=512, scale=0.05):
    q, o = (_view(**VIEW) if x is None else x for x in (q, o))
    return lib.ffpa_decode_fwd_kv4(dt, q, cache or _cache(), lens, o, lse, ws, ws_bytes, B, Hq, Hkv, Nq, D, 0, scale,
                                   None)


COMMON = [
    (dict(dt=3), 2, "dtype"),
    (dict(D=96), 2, "multiple of 64"),
    (dict(D=1088), 2, "head dim"),
    (dict(B=-1), 1, "negative"),
    (dict(cache=dict(page_size=24)), 1, "page_size"),
    (dict(cache=dict(page_size=0)), 1, "page_size"),
    (dict(cache=dict(page_size=-16)), 1, "page_size"),
    (dict(cache=dict(pages=-1)), 1, "negative"),
    (dict(cache=dict(blocks=-1)), 1, "negative"),
    (dict(cache=dict(stride=3)), 1, "block_stride"),
    (dict(cache=dict(data=0)), 1, "cache data"),
    (dict(cache=dict(data=FAKE + 8)), 1, "aligned"),
    (dict(cache=dict(table=0)), 1, "block_table"),
    (dict(cache=dict(table=FAKE + 2)), 1, "block_table"),
]


@pytest.mark.parametrize("fn", [write, read, decode])
@pytest.mark.parametrize("kw,status,msg", COMMON)
def test_refusals_of_every_entry(lib, fn, kw, status, msg):  # noqa: F811
    kw = dict(kw)
    if "cache" in kw:
        kw["cache"] = _cache(**kw["cache"])
    assert fn(lib, **kw) == status
    assert msg in lib.ffpa_last_error().decode()


@pytest.mark.parametrize("fn", [write, read])
@pytest.mark.parametrize("kw,status,msg", [
    (dict(N=-1), 1, "negative"),
    (dict(Hkv=-2), 1, "head count"),
    (dict(k="null"), 1, "k"),
    (dict(v="stride"), 1, "v"),
    (dict(start=FAKE + 1), 1, "4-byte"),
    (dict(count=FAKE + 2), 1, "4-byte"),
    (dict(B=1 << 30, Hkv=1 << 20), 2, "launch grid"),
])
def test_write_and_read_refusals(lib, fn, kw, status, msg):  # noqa: F811
    bad = {"null": _view(ptr=0, **VIEW), "stride": _view(sb=VIEW["sb"], sh=VIEW["sh"], sn=12)}
    assert fn(lib, **{a: bad.get(x, x) if isinstance(x, str) else x for a, x in kw.items()}) == status
    assert msg in lib.ffpa_last_error().decode()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(Hq=3), 1, "multiple"),
    (dict(Hkv=0), 1, "multiple"),
    (dict(scale=float("nan")), 1, "scale"),
    (dict(lens=0), 1, "seq_lens"),
    (dict(lens=FAKE + 1), 1, "seq_lens"),
    (dict(lse=0), 1, "lse"),
    (dict(q="null"), 1, "q"),
    (dict(o="stride"), 1, "o"),
    (dict(Nq=-1), 1, "negative"),
    (dict(B=1 << 12, Hq=1 << 10, Hkv=1 << 10, Nq=1 << 10), 2, "query rows"),
])
def test_decode_refusals(lib, kw, status, msg):  # noqa: F811
    bad = {"null": _view(ptr=0, **VIEW), "stride": _view(sb=VIEW["sb"], sh=VIEW["sh"], sn=12)}
    assert decode(lib, **{a: bad.get(x, x) if isinstance(x, str) else x for a, x in kw.items()}) == status
    assert msg in lib.ffpa_last_error().decode()


def test_packed_entries_refuse_a_missing_cu_seqlens(lib):  # noqa: F811
    for fn, args in ((lib.ffpa_varlen_kv4_write, (0, FAKE, FAKE, _cache())),
                     (lib.ffpa_varlen_kv4_read, (0, _cache(), FAKE, FAKE))):
        assert fn(*args, None, FAKE, 2, 30, 20, 2, 512, None) == 1
        assert "cu_seqlens" in lib.ffpa_last_error().decode()
        assert fn(*args, FAKE + 1, FAKE, 2, 30, 20, 2, 512, None) == 1
        assert fn(*args, FAKE, FAKE, 2, -1, 20, 2, 512, None) == 1


def test_nothing_to_do_is_ok_without_a_launch(lib):  # noqa: F811
    empty = _view(ptr=0, **VIEW)
    none = _cache(data=0, table=0)
    assert write(lib, B=0, k=empty, v=empty, cache=none, start=None, count=None) == 0
    assert read(lib, N=0, k=empty, v=empty, cache=none) == 0
    assert decode(lib, B=0, q=empty, o=empty, lens=None, lse=None, ws=None, ws_bytes=0, cache=none) == 0
    assert lib.ffpa_varlen_kv4_write(0, None, None, none, FAKE, None, 3, 0, 20, 2, 512, None) == 0


def test_cache_bytes(lib):  # noqa: F811
    assert lib.ffpa_kv4_cache_bytes(7, 64, 8, 512) == 7 * 2 * 8 * 4 * 8 * 576
    assert lib.ffpa_kv4_cache_bytes(1 << 20, 64, 8, 512) == (1 << 20) * 294912
    for bad in ((7, 24, 8, 512), (7, 0, 8, 512), (7, 16, 8, 96), (7, 16, 8, 1088), (-1, 16, 8, 64)):
        assert lib.ffpa_kv4_cache_bytes(*bad) == 0


@pytest.mark.parametrize("B,Hq,Hkv,Nq,D", [(2, 4, 2, 1, 32), (2, 4, 2, 1, 96), (2, 4, 2, 1, 0), (2, 4, 2, 1, -64),
                                           (2, 4, 2, 1, 1088), (2, 4, 2, 1, 1 << 30), (0, 4, 2, 1, 64), (2, 3, 2, 1, 64),
                                           (2, 4, 0, 1, 64), (2, 4, 2, 0, 64)])
def test_workspace_of_sizes_outside_the_operation_is_empty(lib, B, Hq, Hkv, Nq, D):  # noqa: F811
    assert lib.ffpa_decode_kv4_workspace_bytes(0, B, Hq, Hkv, Nq, D) == 0


def test_workspace_covers_every_head_dim_and_row_count(lib):  # noqa: F811
    for D in range(64, 1025, 64):
        for Nq in (1, 2, 3, 1000):
            assert lib.ffpa_decode_kv4_workspace_bytes(0, 2, 8, 2, Nq, D) > 0
