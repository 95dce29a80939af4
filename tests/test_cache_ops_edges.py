"""Refusals of the cache operators at their edges (no GPU)."""
import pytest
import torch
from torch.autograd import forward_ad

from head_dim_flash_gb300 import _ffi, api
from tests.test_abi import lib  # noqa: F401
from tests.test_cache_ops_abi import FAKE, evict, shared, weigh


def test_unknown_flags_of_packed_positions(lib):  # noqa: F811
    plan = _ffi.RopePlan(FAKE, 512, 0, 1.0)

    def call(flags, total):
        return lib.ffpa_varlen_rope(0, FAKE, FAKE, FAKE, FAKE, plan, FAKE, FAKE, None, 2, total, 4, 2, 512, flags, None)

    for flags in (4, 5, -1, 1 << 20):
        assert call(flags, 100) == 1 and "flags" in lib.ffpa_last_error().decode()
    for flags in range(4):
        assert call(flags, 0) == 0  # no tokens


def test_token_counts_near_31_bits(lib):  # noqa: F811
    """Indexes run a block past the last token: 2^31 - 4097 tokens are the most."""
    most = 2 ** 31 - 4097
    for fn in (shared, weigh):
        assert fn(lib, N=2 ** 31 - 1, **(dict(Np=0) if fn is shared else {})) == 2
        assert "keys" in lib.ffpa_last_error().decode()
    for N, Np in ((most, 1), (1, most), (2 ** 30, 2 ** 30)):
        assert shared(lib, N=N, Np=Np) == 2 and "keys" in lib.ffpa_last_error().decode()
        assert lib.ffpa_decode_shared_workspace_bytes(0, 1, 1, 1, 1, Np, N, 64) == 0
    assert lib.ffpa_decode_weights_workspace_bytes(0, 1, 1, 1, 1, most + 1, 64) == 0
    assert lib.ffpa_decode_weights_workspace_bytes(0, 1, 1, 1, 1, most, 64) >= 4 * most
    for kw in (dict(N=2 ** 31 - 1, Nout=2 ** 31 - 1), dict(N=most + 1), dict(keep=2 ** 31 - 1), dict(keep=most + 1)):
        assert evict(lib, **kw) == 2 and "tokens" in lib.ffpa_last_error().decode()
    # within them, the next check speaks
    assert evict(lib, N=most, Nout=10, keep=most) == 1 and "N_out" in lib.ffpa_last_error().decode()


def test_what_an_eviction_keeps_is_checked_before_it_is_allocated(monkeypatch):
    k, w, n = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 4), torch.zeros(1).int()
    monkeypatch.setattr(api, "_evict_layout", lambda *a: (torch.device("cpu"), 0, 0, ((512, 256, 64),) * 2))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for keep, recent in ((0, 0), (4, 5), (4, -1), (4, 2 ** 32), (-3, 0)):
        with pytest.raises(ValueError, match="keep"):
            api.kv_evict(k, k.clone(), w, n, keep, recent)
    for keep in (2 ** 31 - 1, 2 ** 31 - 4096, 2 ** 33):
        with pytest.raises(NotImplementedError, match="keep"):
            api.kv_evict(k, k.clone(), w, n, keep)


def test_forward_mode_is_refused(monkeypatch):
    """A tangent is not dropped, whether or not a gradient is wanted."""
    def launched(*args):
        raise AssertionError("launched without its tangent")

    monkeypatch.setattr(api, "_rope_dense", launched)
    monkeypatch.setattr(api, "_rope_packed", launched)
    plan = api.rope_plan(64, device="cpu")
    x, cu = torch.zeros(1, 2, 4, 64), torch.zeros(2).int()
    with forward_ad.dual_level():
        d = forward_ad.make_dual(x, torch.ones_like(x))
        with torch.no_grad():
            e = forward_ad.make_dual(x, torch.ones_like(x))
        for q, k in ((d, x), (x, d), (d, None), (e, x)):
            for call in (lambda: api.rope(q, k, plan), lambda: api.rope(q, k, plan, q_out=x),
                         lambda: api.attention(q, q if k is None else k, x, rope=plan),
                         lambda: api.varlen_rope(q[0], None if k is None else k[0], plan, cu),
                         lambda: api.varlen_attention(q[0], (q if k is None else k)[0], x[0], cu, rope=plan)):
                for grad in (True, False):
                    with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError, match="forward-mode"):
                        call()
        with pytest.raises(AssertionError):
            api.rope(x, x, plan)  # tensors without a tangent
    with pytest.raises(AssertionError):
        api.rope(x, x, plan)
