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


# ---- numbers past 32 bits ------------------------------------------------------------------------
def test_bounds_that_do_not_fit_are_refused_and_not_cut():
    c = PagedCache(4, 2, 2, 16, 64, device="cpu")
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for kw in (dict(max_len=2 ** 32 + 32), dict(max_new=2 ** 32 + 1), dict(max_len=2 ** 31), dict(max_new=2 ** 31), dict(max_len=-1),
               dict(max_new=-2 ** 32 + 1)):
        with pytest.raises(ValueError):
            c.sequences(table, lens, **dict(dict(max_len=32, max_new=5), **kw))
    with pytest.raises(ValueError):
        PagedCache(2 ** 32 + 4, 2, 2, 16, 64, device="cpu")
    s = c.sequences(table, lens, max_len=2 ** 31 - 1, max_new=2 ** 31 - 1)
    assert s.c.max_len == s.c.max_new == 2 ** 31 - 1


def _calls(monkeypatch, cache):
    """The arguments that reach the library, from a cache that is made to look like one on another device."""
    seen = []

    class Device:
        current = 0

        def __init__(self, index):
            self.index = index if isinstance(index, int) else index.index

        def __enter__(self):
            self.before, Device.current = Device.current, self.index

        def __exit__(self, *a):
            Device.current = self.before

    cache.device = torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: Device.current)
    monkeypatch.setattr(C, "stream_handle", lambda stream, index: ("stream of", index))
    monkeypatch.setattr(C, "pisa_cache_attention", lambda *a: seen.append((Device.current, a)))
    monkeypatch.setattr(C, "pisa_read_device_error", lambda ws, stream=None: (seen.append((Device.current, stream)), (0, 0))[1])
    monkeypatch.setattr(cache, "_rows", lambda seqs, x, heads, name: name)
    return seen


@pytest.mark.parametrize("window,reaches", [(0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                                            (10 ** 30, 2 ** 31 - 1), (-1, -1), (-2 ** 32 + 5, -1)])
def test_a_window_of_any_size_means_what_it_says(monkeypatch, window, reaches):
    """Past 32 bits it is longer than any context; below zero the library refuses it."""
    c = PagedCache(4, 2, 2, 16, 64, device="cpu")
    seqs = c.sequences(torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), max_len=32, max_new=5)
    q = torch.zeros(1, 2, 5, 64, dtype=torch.bfloat16)
    seen = _calls(monkeypatch, c)
    c.attention(seqs, q, torch.zeros_like(q), window=window)
    assert seen[0][1][4] == reaches


def test_the_status_is_read_on_the_cache_s_device(monkeypatch):
    """Whatever the current one is: its stream orders the read after the cache's calls."""
    c = PagedCache(4, 2, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        c.device_error()
    seen = _calls(monkeypatch, c)
    assert c.device_error() == (0, 0) and c.device_error("a stream") == (0, 0)
    assert seen == [(1, None), (1, "a stream")]
