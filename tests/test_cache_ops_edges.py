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
