"""kfac_verify_draft refuses pointers that are not on their elements' boundaries: the kernels read whole elements."""
import ctypes

import pytest

from tests.test_verify_host import _vd
from second_order_optimisation_gb300 import kfac


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return kfac.load()


@pytest.mark.parametrize("bad", [dict(tokens=0x2004), dict(out_tokens=0x8004), dict(tokens=0x2002, token_i32=1), dict(out_tokens=0x8001, token_i32=1),
                                 dict(seq_offsets=0x3002), dict(accepted=0x7001), dict(logp=0x9002), dict(uniform=0x5002), dict(noise=0x6001)])
def test_refuses(lib, bad):
    d = ctypes.byref(_vd(**bad))
    assert lib.kfac_verify_draft_workspace_size(d) == 0
    assert lib.kfac_verify_draft(d, 0x100000, 1 << 40, None) == kfac.KFAC_ERR_INVALID


@pytest.mark.parametrize("good", [dict(tokens=0x2004, out_tokens=0x8004, token_i32=1), dict(uniform=0x5004, noise=0x6004, logp=0x900c),
                                  dict(greedy=1, uniform=0x5001, noise=0x6003)])
def test_takes(lib, good):
    assert lib.kfac_verify_draft_workspace_size(ctypes.byref(_vd(**good))) > 0
