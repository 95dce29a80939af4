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
