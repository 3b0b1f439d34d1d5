"""The paged cache on data at the edges of what it may hold: zeros, slots that were never written,
scales far apart (needs a B200).  Tolerances are cache_reference.bounds' unless a test says otherwise."""
import pytest
import torch

from piecewise_approximate_attention_b200 import _lib as C
from piecewise_approximate_attention_b200.runtime import PagedCache
from tests import cache_reference as R
from tests.test_gpu_cache import DTYPES, Case

pytestmark = pytest.mark.gpu


def stored(c):
    """Appends everything that the case's k and v hold, and takes its stored values anew."""
    whole = Case.__new__(Case)
    whole.__dict__.update(c.__dict__)
    whole.new, whole.max_new = list(c.lens), max(c.lens)
    c.cache.append(whole.sequences(c.lens), whole.tokens(c.k, c.kv_heads).cuda(), whole.tokens(c.v, c.kv_heads).cuda())
    c.kv64 = [[R.quantise(x)[0] if c.dtype == "e4m3" else x.double() for x in side] for side in (c.k, c.v)]
    return c


# ---- zeros -------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,lens,new", [(128, [150], [150]), (128, [131, 70, 300], [1, 1, 1]), (64, [299, 33], [20, 20]),
                                        (64, [333], [100]), (128, [333, 200], [300, 130]), (128, [1500], [260])])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 45)])
def test_zero_queries_over_zero_keys_take_the_mean(dtype, d, lens, new, causal, window):
    """As a warm-up on zeroed tensors has them, or padding: every visible value weighs the same."""
    c = Case(dtype, 4, 2, d, 16, lens, new, fill=False)
    c.k = [torch.zeros_like(x) for x in c.k]
    c.q = [torch.zeros_like(x) for x in c.q]
    rows = [0, 1, 2, 63, 64, 127, 128, 129, 255, 256, 259]
    stored(c).check(causal, window, rows=rows)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 5, 40, 150, 300])
def test_a_step_on_zeroed_tensors(dtype, new):
    """What test programs and graph captures run first: zeros are appended and attended over."""
    cache = PagedCache(40, 4, 2, 32, 128, dtype)
    table = torch.randperm(40, generator=torch.Generator().manual_seed(1))[:32].reshape(2, 16).to(torch.int32).cuda()
    lens = torch.tensor([new, new + 50], dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(2, n, new, 128, dtype=R.DTYPES[dtype], device="cuda") for n in (4, 2, 2))
    lse = torch.full((2, 4, new), 7.0, device="cuda")
    seqs = cache.sequences(table, lens, max_len=512, max_new=new)
    cache.append(seqs, k, v)
    o = cache.attention(seqs, q, torch.full_like(q, 7.0), softmax_scale=0.1, lse=lse)
    assert cache.device_error() == (C.PISA_OK, 0)
    assert bool((o == 0).all())
    seen = torch.arange(new)[None] + torch.tensor([1, 51])[:, None]
    # log of a count of at most 2^9 by log2 of it, each within 2^-22 of its size
    assert ((lse.cpu().double() - seen.double().log()[:, None]).abs() <= 2.0 ** -19).all()


# ---- slots that were never written -------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 5, 40, 150, 300])
def test_slots_of_a_new_pool_hold_zeros(dtype, new):
    """A pool that PagedCache makes holds zeros in the meaning of its type before anything is appended."""
    n = new + 37
    cache = PagedCache(24, 4, 2, 16, 128, dtype)
    table = torch.arange(24, dtype=torch.int32, device="cuda")[None]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q = torch.randn(new, 4, 128, generator=torch.Generator().manual_seed(2)).to(R.DTYPES[dtype]).cuda()
    lse = torch.full((new, 4), 7.0, device="cuda")
    o = cache.attention(cache.sequences(table, i32(n), 384, new, starts=i32(0, new)), q, torch.full_like(q, 7.0),
                        softmax_scale=0.1, lse=lse)
    assert cache.device_error() == (C.PISA_OK, 0)
    assert bool((o == 0).all())
    seen = torch.arange(38, n + 1).double()
    assert ((lse.cpu().double() - seen.log()[:, None]).abs() <= 2.0 ** -19).all()
    k, v = (torch.full((n, 2, 128), 7.0, dtype=q.dtype, device="cuda") for _ in range(2))
    cache.read(cache.sequences(table, i32(n), 384, n, starts=i32(0, n)), k, v)
    assert bool((k == 0).all()) and bool((v == 0).all())
