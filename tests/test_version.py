"""The version tells callers of other headers that their descriptors have another size."""
import ctypes
import os
import re

from second_order_optimisation_gb300 import kfac

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kfac.h")


def test_version_of_the_header():
    import __graft_entry__
    __graft_entry__.build()
    text = open(HEADER).read()
    n = int(re.search(r"#define KFAC_VERSION (\d+)", text).group(1))
    assert kfac.load().kfac_version() == n > 200  # (200: kfac_factor_desc without scales and ldx)


def test_factor_descriptor_s_size():
    """What 300 stands for: two fields of 8 bytes behind the layout's."""
    d = kfac.FactorDesc
    assert d.scales.offset == d.layout.offset + 8 - d.layout.offset % 8 and d.ldx.offset == d.scales.offset + 8
    assert ctypes.sizeof(d) == d.ldx.offset + 8
