"""The paged cache on data at the edges of what it may hold: zeros, slots that were never written,
scales far apart (needs a B200).  Tolerances are cache_reference.bounds' unless a test says otherwise."""
import pytest
import torch

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
