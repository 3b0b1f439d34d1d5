"""The cache attention's bounded waits, without a fault: keys that never come (needs a B200).

The test-only hook makes the load warps leave out the keys of their block's first tile, so a wait for them cannot
complete.  The kernel must report PISA_DEVERR_WAIT_TIMEOUT, stop loading, wait for what is in flight, free its tensor
memory and return; with the workspace zeroed, the next call on the same context must be right."""
import time

import pytest
import torch

from piecewise_approximate_attention_b200 import _lib as C
from piecewise_approximate_attention_b200.runtime import PagedCache
from tests.test_gpu_cache import Case

pytestmark = pytest.mark.gpu

SKIP_KEYS_LOAD = 3
WAIT_NS = 20_000_000          # 20 ms instead of the default 2 s


def failing_call(c, fault=SKIP_KEYS_LOAD, wait_ns=WAIT_NS):
    """Seconds that the call took with the fault set."""
    q = c.tokens(c.q, c.heads).cuda()
    o = torch.zeros_like(q)
    torch.cuda.synchronize()
    assert C.lib().pisa_testing_set_cache_fault(fault, wait_ns) == C.PISA_OK
    try:
        t = time.perf_counter()
        c.cache.attention(c.seqs, q, o, softmax_scale=c.scale)
        torch.cuda.synchronize()
        return time.perf_counter() - t
    finally:
        assert C.lib().pisa_testing_set_cache_fault(0, 0) == C.PISA_OK


# a token; rows for one, two and four row tiles; both slots on the same rows; pairs of slots
NEW = [1, 3, 10, 20, 40, 100, 300]


@pytest.mark.parametrize("dtype", ("bf16", "e4m3"))
@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("d,lens", [(128, [900]), (64, [3000, 41])])
def test_a_wait_that_runs_out_is_reported(dtype, new, d, lens):
    c = Case(dtype, 2, 1, d, 32, lens, [min(new, n) for n in lens])
    good = c.check(rows=(0, 1))
    took = failing_call(c)
    assert c.cache.device_error() == (C.PISA_ERR_DEVICE_TIMEOUT, C.PISA_DEVERR_WAIT_TIMEOUT)
    assert c.cache.device_error() == (C.PISA_OK, 0)           # read clears the status word
    assert took < 1.0                  # a few limits, not a tile's or an item's each
    c.cache.ws.zero_()
    assert torch.equal(c.check(rows=(0, 1)), good)


@pytest.mark.parametrize("dtype", ("bf16", "e4m3"))
@pytest.mark.parametrize("new", [1, 100, 300])
def test_a_long_share_ends_soon_after_its_wait(dtype, new):
    """Blocks with hundreds of tiles and several items: none of them waits for each tile anew."""
    n, kv = 9000, 160
    cache = PagedCache(71, kv, kv, 128, 64, dtype)
    table = torch.arange(71, dtype=torch.int32, device="cuda")[None]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    seqs = cache.sequences(table, i32(n), n, new, starts=i32(0, new))
    q = torch.randn(new, kv, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    lse = torch.empty(new, kv, device="cuda")

    def call():
        o = torch.full_like(q, 7.0)
        cache.attention(seqs, q, o, causal=False, lse=lse)
        torch.cuda.synchronize()
        return o

    assert bool((call() == 0).all())
    assert C.lib().pisa_testing_set_cache_fault(SKIP_KEYS_LOAD, WAIT_NS) == C.PISA_OK
    try:
        t = time.perf_counter()
        call()
        took = time.perf_counter() - t
    finally:
        assert C.lib().pisa_testing_set_cache_fault(0, 0) == C.PISA_OK
    assert cache.device_error() == (C.PISA_ERR_DEVICE_TIMEOUT, C.PISA_DEVERR_WAIT_TIMEOUT)
    assert took < 1.0
    cache.ws.zero_()
    assert bool((call() == 0).all())
    assert ((lse.double() - torch.tensor(float(n)).double().log().cuda()).abs() <= 2.0 ** -18).all()
    assert cache.device_error() == (C.PISA_OK, 0)


def test_rows_that_are_computed_by_themselves_do_not_run_into_the_limit():
    """One value of another size in each head sends whole shares through the routine that computes row by row, for
    longer than the waits' limit (set to 3 ms here; such an item takes more): nothing is wrong, and nothing may be
    reported.  Two items a block, so that its other warps wait for the second one's queries meanwhile."""
    n, new, kv, d = 8192, 200, 296, 64
    cache = PagedCache(64, kv, kv, 128, d, "e4m3")
    g = torch.Generator("cuda").manual_seed(3)
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(n, kv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    v[5000] *= 2.0 ** 12
    whole = cache.sequences(table, i32(n), n, n, starts=i32(0, n))
    cache.append(whole, k, v)
    cache.read(whole, k, v)
    q = torch.randn(new, kv, d, generator=g, device="cuda").bfloat16()
    seqs = cache.sequences(table, i32(n), n, new, starts=i32(0, new))
    torch.cuda.synchronize()
    assert C.lib().pisa_testing_set_cache_fault(0, 3_000_000) == C.PISA_OK
    try:
        t = time.perf_counter()
        o = cache.attention(seqs, q, causal=False, softmax_scale=0.125)
        torch.cuda.synchronize()
        took = time.perf_counter() - t
    finally:
        assert C.lib().pisa_testing_set_cache_fault(0, 0) == C.PISA_OK
    assert took > 0.006                                      # it did outlast the limit
    assert cache.device_error() == (C.PISA_OK, 0)
    for h in (0, 1, 147, 295):
        s = q[:, h].double() @ k[:, h].double().T * 0.125
        w = torch.softmax(s, -1)
        ref, size = w @ v[:, h].double(), w @ v[:, h].double().abs()
        # fp32 throughout: logits of at most 0.125 * 64 * 25 off by (d + 4) 2^-23 of it, sums of n terms, one rounding
        rel = 2 * ((d + 4) * 2.0 ** -23 * 200 + 2.0 ** -21) + 2 * n * 2.0 ** -23
        assert bool(((o[:, h].double() - ref).abs() <= size * rel * 1.01 + 2.0 ** -8 * ref.abs()).all()), h
