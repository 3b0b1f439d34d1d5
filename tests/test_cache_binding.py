"""What PagedCache hands to the library, seen on the CPU (nothing is launched)."""
import re

import pytest
import torch

from piecewise_approximate_attention_b200 import _lib as C
from piecewise_approximate_attention_b200.build import INCLUDE
from piecewise_approximate_attention_b200.runtime import PagedCache


def test_a_new_e4m3_pool_holds_scales_of_its_format():
    """-50 ... 50 with a bias of 127: a byte of 0 would be a scale that the kernels are promised not to meet."""
    c = PagedCache(3, 2, 2, 16, 64, "e4m3", device="cpu")
    for e in (c.k_exp, c.v_exp):
        assert bool(((e >= 127 - 50) & (e <= 127 + 50)).all())
    assert bool((c.k == 0).all()) and bool((c.v == 0).all())
    given = torch.full((3, 2, 16), 130, dtype=torch.uint8)
    c = PagedCache(3, 2, 2, 16, 64, "e4m3", device="cpu", k_exp=given)
    assert c.k_exp.data_ptr() == given.data_ptr() and bool((given == 130).all())
    header = open(INCLUDE + "/pisa_cache.h").read()
    for name in ("PISA_CACHE_EXP_MIN", "PISA_CACHE_EXP_MAX"):
        assert getattr(C, name) == int(re.search(rf"#define {name} (\d+)", header).group(1))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_other_pools_have_no_scales(dtype):
    c = PagedCache(3, 2, 2, 16, 64, dtype, device="cpu")
    assert c.k_exp is None and c.v_exp is None and bool((c.k == 0).all())


def test_the_testing_hook_rejects_unknown_faults():
    for fault in (1, 2, 4, -1):
        assert C.lib().pisa_testing_set_cache_fault(fault, 0) == C.PISA_ERR_INVALID_ARG
    assert C.lib().pisa_testing_set_cache_fault(0, 0) == C.PISA_OK
