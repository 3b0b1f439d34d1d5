"""The paged cache on data at the edges of what it may hold: zeros, slots that were never written,
scales far apart (needs a B200).  Tolerances are cache_reference.bounds' unless a test says otherwise."""
import math

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


# ---- the weights' own rounding -----------------------------------------------------------------
@pytest.mark.parametrize("heads,kv,d,lens,new,window", [
    (1, 1, 128, [70], [1], 0), (16, 2, 128, [577, 90], [1, 1], 0), (5, 1, 64, [300], [3], 0), (4, 2, 64, [1200, 31], [4, 8], 50),
    (8, 1, 128, [2500], [2], 0), (3, 3, 128, [260, 5], [16, 5], 0)])
def test_weights_of_few_rows_keep_sixteen_bits(heads, kv, d, lens, new, window):
    """bf16 pools, at most 16 rows: the bounds of cache_reference with weights that are off by 2^-16 in two parts
    (half a step of the second, 2^-8 of what the first left over, itself at most 2^-8) instead of 2^-8."""
    c = Case("bf16", heads, kv, d, 32, lens, new)
    q = c.tokens(c.q, heads).cuda()
    got = c.split(c.cache.attention(c.seqs, q, window=window, softmax_scale=c.scale))
    for b, (n, m) in enumerate(zip(lens, new)):
        for h in range(heads):
            kh = h // (heads // kv)
            ref = R.attention(c.q[b][h].double(), c.kv64[0][b][kh], c.kv64[1][b][kh], list(range(n - m, n)), True, window,
                              float(torch.tensor(c.scale, dtype=torch.float32)))
            rel = 2.0 ** -16 + 2 * ((d + 4) * 2.0 ** -23 * ref["size"] + 2.0 ** -21) + 2 * ref["seen"] * 2.0 ** -23
            bound = ref["mean_abs"] * rel[:, None] * 1.01 + 2.0 ** -8 * ref["o"].abs() + 1e-37
            assert bool(((got[b][h].double() - ref["o"]).abs() <= bound).all()), (b, h)


@pytest.mark.parametrize("dtype", ("bf16", "e4m3"))
@pytest.mark.parametrize("new", [1, 5, 16, 30, 64, 100, 128, 200, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_a_row_that_one_late_key_dominates(dtype, new, d):
    """A key whose logit is 7 + log2(1 + 2^-8) above the largest before it, in base 2: its weight against that maximum
    is where bf16 rounds farthest.  It holds all but 1/129 of the row, so the row is its value, and must not be off by
    that rounding: half a step of the result's type, and the weights' 2^-8 on the other key's share of twice the
    largest |v|."""
    n, late = 300, 256                       # a tile of every kernel further on, taken by the same warp or slot
    c = Case(dtype, 1, 1, d, 16, [n], [new], scale=math.log(2.0), fill=False)
    c.q[0] = torch.ones_like(c.q[0])
    c.k[0] = torch.full_like(c.k[0], -60.0 / d)
    c.k[0][0, 0] = 0.0
    c.k[0][0, late] = 0.0
    # 7 + 0.005615 from numbers that bf16 and e4m3 rows hold: 7.00390625 + 0.00170898
    c.k[0][0, late, :7] = 1.0
    c.k[0][0, late, 7] = 2.0 ** -8
    c.k[0][0, late, 8] = 2.0 ** -9 if dtype == "e4m3" else 7 * 2.0 ** -12
    stored(c)
    got = c.split(c.cache.attention(c.seqs, c.tokens(c.q, 1).cuda(), causal=False, softmax_scale=c.scale))[0][0].double()
    ref = R.attention(c.q[0][0].double(), c.kv64[0][0][0], c.kv64[1][0][0], list(range(n - new, n)), False, 0,
                      float(torch.tensor(c.scale, dtype=torch.float32)))["o"]
    step = torch.exp2(torch.floor(torch.log2(ref.abs())) - 7)
    bound = step / 2 + 2.0 ** -8 / 129 * 2 * c.kv64[1][0].abs().max() + 2.0 ** -18 * ref.abs()
    assert bool(((got - ref).abs() <= bound).all()), ((got - ref).abs() / bound).max()



@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("new,window,causal", [(4, 7, True), (7, 7, False), (30, 7, True), (30, 0, False), (8, 0, True)])
def test_rows_of_few_keys_and_values_of_many_sizes(seed, new, window, causal):
    """bf16 weights of 17 rows and more are off by 2^-8 each, not by that and what scaling a row would add."""
    c = Case("bf16", 8, 1, 128, 16, [120, 41], [new, new], fill=False, seed=seed)
    g = torch.Generator().manual_seed(seed)
    for b in range(2):
        c.k[b] = (c.k[b].float() * 2.0).bfloat16()
        c.v[b] = (c.v[b].float() * torch.exp2(torch.rand(c.v[b].shape[:2], generator=g)[..., None] * 24 - 12)).bfloat16()
    stored(c).check(causal, window)


# ---- zeros in front of ordinary tokens (e4m3: a share's unit) ------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("zeros", [1, 127, 128, 130, 300, 699])
@pytest.mark.parametrize("side,new", [("k", 70), ("v", 150), ("kv", 150), ("kv", 3), ("kv", 300)])
def test_zero_tokens_in_front(dtype, zeros, side, new):
    """Padding at a context's beginning: rows of zeros, +0 and -0, have no say in the scales of what follows."""
    c = Case(dtype, 2, 1, 128, 32, [700], [new], fill=False)
    for name in side:
        x = getattr(c, name)[0]
        x[:, :zeros] = 0.0
        x[:, 5:zeros:3] = -0.0
    stored(c).check(rows=(0, 1, new // 2, new - 1))
    c.check(causal=False, window=500, rows=(0, 1, new // 2, new - 1))


@pytest.mark.parametrize("new", [3, 150, 300])
@pytest.mark.parametrize("size", [2.0 ** -58, 2.0 ** 49])
def test_numbers_at_the_scales_ends(new, size):
    """Rows whose scale is the smallest there is without being zeros, and rows whose scale is the largest."""
    c = Case("e4m3", 2, 1, 64, 16, [400], [new], fill=False)
    c.v[0] = (c.v[0].float() * size).bfloat16()
    c.k[0] = (c.k[0].float() * size).bfloat16()
    c.q[0] = (c.q[0].float() / size).bfloat16()
    stored(c).check(rows=(0, 1, new // 2, new - 1))
    c.k[0][:, :200] = 0.0
    c.v[0][:, :130] = 0.0
    stored(c).check(rows=(0, 1, new // 2, new - 1))


def test_zero_tokens_in_front_cost_little():
    """They used to send whole shares through the routine for single rows, some tens of times slower."""
    n, new, kv, d = 4096, 256, 148, 64
    cache = PagedCache(32, kv, kv, 128, d, "e4m3")
    table = torch.arange(32, dtype=torch.int32, device="cuda")[None]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(n, kv, d, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(new, kv, d, device="cuda").bfloat16()
    seqs = cache.sequences(table, i32(n), n, new, starts=i32(0, new))

    def ms(zeros):
        k[:zeros] = 0.0
        v[:zeros] = 0.0
        v[:zeros:2] = -0.0
        cache.append(cache.sequences(table, i32(n), n, n, starts=i32(0, n)), k, v)
        for _ in range(2):
            cache.attention(seqs, q, causal=False, softmax_scale=0.125)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(4):
            cache.attention(seqs, q, causal=False, softmax_scale=0.125)
        b.record()
        b.synchronize()
        return a.elapsed_time(b) / 4

    plain = ms(0)
    assert max(ms(100), ms(128), ms(500)) < 2 * plain + 0.1
    assert cache.device_error() == (C.PISA_OK, 0)


# ---- bounds far above what is there --------------------------------------------------------------
@pytest.mark.parametrize("dtype", ("bf16", "e4m3"))
@pytest.mark.parametrize("new", [1, 3, 12, 30])
@pytest.mark.parametrize("lens", [[577], [1300, 90], [200], [900] * 40])
def test_the_bound_of_the_lengths_does_not_change_how_work_is_shared(dtype, new, lens):
    """As a captured step has it, sized for the longest context there may be: the parts that are joined, and so the
    bits, are those of a call with the bound at the lengths.  So for up to 64 rows a key/value head; above, the kernel's
    form is chosen on the host, which has the bound alone, and both results are held to their definition."""
    c = Case(dtype, 8, 2, 128, 32, lens, [new] * len(lens))
    q = c.tokens(c.q, 8).cuda()
    table = torch.full((len(lens), 2400), -1, dtype=torch.int32, device="cuda")
    table[:, :c.max_pages] = c.table.cuda()
    loose = c.cache.sequences(table, c.seqs.tensors[1], max_len=75600, max_new=new, starts=c.seqs.tensors[2])
    got = []
    for seqs in (c.seqs, loose):
        lse = torch.empty(q.shape[:-1], device="cuda")
        got.append((c.cache.attention(seqs, q, softmax_scale=c.scale, lse=lse), lse))
    if 4 * new <= 64:
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    else:
        c.check(rows=(0, new - 1))
        c.seqs = loose
        c.check(rows=(0, new - 1))
    assert c.cache.device_error() == (C.PISA_OK, 0)


@pytest.mark.parametrize("dtype", ("bf16", "e4m3"))
@pytest.mark.parametrize("new", [1, 3, 12, 30])
def test_what_lies_behind_a_window_does_not_change_how_work_is_shared(dtype, new):
    """A window over a long context is shared out like the same window over its last pages alone."""
    n, last = 20_000, 20_000 - 16_384              # the same place in a tile
    c = Case(dtype, 8, 2, 128, 128, [n], [new])
    q = c.tokens(c.q, 8).cuda()
    tail = c.table[:, 128:].contiguous().cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    short = c.cache.sequences(tail, i32(last), max_len=last, max_new=new, starts=i32(0, new))
    got = []
    for seqs in (c.seqs, short):
        lse = torch.empty(q.shape[:-1], device="cuda")
        got.append((c.cache.attention(seqs, q, window=1024, softmax_scale=c.scale, lse=lse), lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    c.check(window=1024, rows=(0, new - 1))


# ---- weights far below a row's largest -----------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 5, 20, 60, 70, 100, 150, 300])
def test_many_small_weights_beside_a_large_one_of_small_values(new, d):
    """e4m3: one key takes nearly all the weight, with values 2^-14 of the others', whose weights of 2^-22.6 make up most
    of the result.  The bounds of cache_reference, with what falls below fp16's normal range counted from weights that
    reach 2^8: half a step of 2^-24 over 2^8 a key, 2^-33 of the largest |v|."""
    n = 2000
    c = Case("e4m3", 1, 1, d, 32, [n], [new], scale=math.log(2.0), fill=False)
    c.q[0] = torch.ones_like(c.q[0])
    c.k[0] = torch.full_like(c.k[0], 0.0)
    c.k[0][0, 1:, 0] = -20.0
    c.k[0][0, 1:, 1] = -2.5
    c.k[0][0, 1:, 2] = -0.1015625                # -22.6
    c.v[0] = (c.v[0].float().abs() * 0.25 + 1.0).bfloat16()
    c.v[0][0, 0] = 2.0 ** -14
    stored(c)
    got = c.split(c.cache.attention(c.seqs, c.tokens(c.q, 1).cuda(), causal=False, softmax_scale=c.scale))[0][0].double()
    ref = R.attention(c.q[0][0].double(), c.kv64[0][0][0], c.kv64[1][0][0], list(range(n - new, n)), False, 0,
                      float(torch.tensor(c.scale, dtype=torch.float32)))
    rel = 2.0 ** -11 + 2 * ((d + 4) * 2.0 ** -23 * ref["size"] + 2.0 ** -21) + 2 * ref["seen"] * 2.0 ** -23
    bound = ref["mean_abs"] * rel[:, None] * 1.01 + 2.0 ** -8 * ref["o"].abs() + n * 2.0 ** -33 * ref["vmax"]
    err = (got - ref["o"]).abs()
    assert bool((err <= bound).all()), (err / ref["o"].abs()).max()
