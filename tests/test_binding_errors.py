"""Errors of the binding that no call on the GPU shows."""
import pytest

from second_order_optimisation_gb300 import kfac


class _Failing:
    """A library whose read of the launches fails."""

    def kfac_timing_read_launches(self, *args):
        return -1

    def kfac_status_string(self, status):
        return b"KFAC_ERR_CUDA"


def test_a_failed_read_of_the_launches_says_so(monkeypatch):
    monkeypatch.setattr(kfac, "load", lambda: _Failing())
    with pytest.raises(kfac.KfacError, match="kfac_timing_read_launches") as e:
        kfac.timing_read_launches(4)
    assert e.value.status == kfac.KFAC_ERR_CUDA
