"""The paged key/value cache on the GPU against its definition in float64 (needs a B200).

Every slot of a pool that a case does not fill holds NaN, so that reading a stale slot shows."""
import math

import pytest
import torch

from piecewise_approximate_attention_b200 import _lib as C
from piecewise_approximate_attention_b200.runtime import PagedCache, Pisa
from tests import cache_reference as R

pytestmark = pytest.mark.gpu
NAN_CODE, NAN_EXP = 0x7F, 177


class Case:
    """A cache that holds `lens` tokens a sequence, `new` of them new, with random pages."""

    def __init__(self, dtype, heads, kv_heads, d, page, lens, new, layout="packed", seed=0, max_len=None, max_new=None,
                 scale=None, fill=True):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.heads, self.kv_heads, self.d, self.page = dtype, heads, kv_heads, d, page
        self.lens, self.new, self.layout = lens, new, layout
        self.scale = scale if scale is not None else 1.0 / math.sqrt(d)
        t = R.DTYPES[dtype]
        per = [-(-n // page) for n in lens]
        pages = sum(per) + 2
        order = torch.randperm(pages, generator=g).to(torch.int32)
        self.max_pages = max(per + [1]) + 1
        self.table = torch.full((len(lens), self.max_pages), -7, dtype=torch.int32)     # unused entries are no pages
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        f8 = dtype == "e4m3"
        shape = (pages, kv_heads, page, d)
        if f8:
            pool = [torch.full(shape, NAN_CODE, dtype=torch.uint8) for _ in range(2)]
            exps = [torch.full(shape[:3], NAN_EXP, dtype=torch.uint8) for _ in range(2)]
        else:
            pool, exps = [torch.full(shape, float("nan"), dtype=t) for _ in range(2)], [None, None]
        # what each sequence holds, [kv_heads, len, d], as token tensors' numbers and as stored values
        self.k = [self.make(g, (kv_heads, n, d), 1.5).to(t) for n in lens]
        self.v = [self.make(g, (kv_heads, n, d), 0.0).to(t) for n in lens]
        self.kv64 = [[R.quantise(x)[0] if f8 else x.double() for x in side] for side in (self.k, self.v)]
        self.cache = PagedCache(pages, heads, kv_heads, page, d, dtype, "cuda", *(x.cuda() for x in pool),
                                *(x if x is None else x.cuda() for x in exps))
        self.t = t
        self.max_len = max_len or max(lens + [1])
        self.max_new = max_new or max(new + [1])
        self.seqs = self.sequences(new)
        if fill:                                       # everything that is there, through the append itself
            c = Case.__new__(Case)
            c.__dict__.update(self.__dict__)
            c.new, c.max_new = list(lens), max(lens + [1])
            full = c.sequences(lens)
            self.cache.append(full, c.tokens(self.k, kv_heads).cuda(), c.tokens(self.v, kv_heads).cuda())
        self.q = [self.make(g, (heads, m, d), 0.25).to(t) for m in new]

    @staticmethod
    def make(g, shape, shift):
        x = torch.randn(shape, generator=g)
        x[..., ::16] += shift
        return x

    def sequences(self, new):
        dev = "cuda"
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        kw = dict(starts=i32([0] + new).cumsum(0).to(torch.int32)) if self.layout == "packed" else \
            dict(counts=i32(new))
        return self.cache.sequences(self.table.to(dev), i32(self.lens), self.max_len, self.max_new, **kw)

    def tokens(self, per_seq, heads, fill=0.0):
        """Token tensor of the new (last) tokens of each sequence's [heads, n, d]."""
        if self.layout == "packed":
            return torch.cat([x[:, x.shape[1] - m:].transpose(0, 1) for x, m in zip(per_seq, self.new)]).contiguous()
        out = torch.full((len(self.lens), heads, self.max_new, self.d), fill, dtype=self.t)
        for b, (x, m) in enumerate(zip(per_seq, self.new)):
            out[b, :, :m] = x[:, x.shape[1] - m:]
        return out

    def split(self, x):
        """A token tensor's rows of each sequence, [heads, m, d] or, of an lse, [heads, m]."""
        if self.layout == "packed":
            return [y.transpose(0, 1) for y in x.cpu().split(self.new)]
        return [x[b, :, :m].cpu() for b, m in enumerate(self.new)]

    def values(self):
        """The pool as the values it stands for, float64 on the CPU, and K and V of it."""
        out = []
        for pool, e in ((self.cache.k, self.cache.k_exp), (self.cache.v, self.cache.v_exp)):
            x = pool.cpu()
            if e is not None:
                x = x.view(torch.float8_e4m3fn).double() * torch.exp2(e.cpu().double() - 127)[..., None]
            out.append(x.double())
        return out

    def check(self, causal=True, window=0, o=None, lse=True, rows=None):
        """Runs the attention and compares every new token (or `rows` of each) with the definition."""
        q = self.tokens(self.q, self.heads).cuda()
        o = torch.full_like(q, 7.0) if o is None else o
        ls = torch.full(q.shape[:-1], 7.0, device="cuda") if lse else None
        self.cache.attention(self.seqs, q, o, causal=causal, window=window, softmax_scale=self.scale, lse=ls)
        torch.cuda.synchronize()
        assert self.cache.device_error() == (C.PISA_OK, 0)
        got, got_lse = self.split(o), self.split(ls) if lse else None
        for b, (n, m) in enumerate(zip(self.lens, self.new)):
            pick = range(m) if rows is None else [r for r in rows if r < m]
            if not len(pick):
                continue
            pos = [n - m + r for r in pick]
            for h in range(self.heads):
                kh = h // (self.heads // self.kv_heads)
                ref = R.attention(self.q[b][h, pick].double(), self.kv64[0][b][kh], self.kv64[1][b][kh], pos, causal, window,
                                  float(torch.tensor(self.scale, dtype=torch.float32)))
                bo, bl = R.bounds(ref, self.dtype, self.d)
                err = (got[b][h, pick].double() - ref["o"]).abs()
                assert bool((err <= bo).all()), (b, h, (err / bo).max().item(), err.max().item())
                if lse:
                    gl = got_lse[b][h, pick].double()
                    empty = ref["seen"] == 0
                    assert bool((gl[empty] == -math.inf).all())
                    el = (gl - ref["lse"])[~empty].abs()
                    assert bool((el <= bl[~empty]).all()), (b, h, el.max().item())
        if self.layout == "padded":                     # rows behind a sequence's last are left as they were
            for b, m in enumerate(self.new):
                assert bool((o[b, :, m:] == 7.0).all())
        return o


DTYPES = ("bf16", "fp32", "e4m3")


# ---- append and read ---------------------------------------------------------------------------
MOVES = [
    # dtype, heads, d, page, lens, new, layout
    ("bf16", 2, 128, 64, [1, 64, 65, 130, 0], [1, 3, 65, 0, 0], "packed"),
    ("bf16", 3, 64, 16, [17, 33, 200], [17, 1, 133], "padded"),
    ("fp32", 1, 64, 16, [5, 47, 16], [5, 20, 16], "packed"),
    ("fp32", 4, 128, 128, [129, 300], [2, 300], "padded"),
    ("e4m3", 2, 128, 32, [1, 31, 33, 97], [1, 31, 2, 97], "packed"),
    ("e4m3", 5, 64, 16, [40, 16, 250], [40, 0, 131], "padded"),
    ("e4m3", 1, 64, 128, [700], [699], "packed"),
]


@pytest.mark.parametrize("dtype,heads,d,page,lens,new,layout", MOVES)
def test_append_writes_the_new_tokens_and_nothing_else(dtype, heads, d, page, lens, new, layout):
    c = Case(dtype, heads, heads, d, page, lens, new, layout, fill=False)
    before = [x.clone() for x in (c.cache.k, c.cache.v, c.cache.k_exp, c.cache.v_exp) if x is not None]
    c.cache.append(c.seqs, c.tokens(c.k, heads).cuda(), c.tokens(c.v, heads).cuda())
    torch.cuda.synchronize()
    assert c.cache.device_error() == (C.PISA_OK, 0)
    got = c.values()
    owned = torch.zeros(c.cache.k.shape[:3], dtype=torch.bool)
    for b, (n, m) in enumerate(zip(lens, new)):
        for p in range(n - m, n):
            pg, slot = int(c.table[b, p // page]), p % page
            owned[pg, :, slot] = True
            for side in range(2):
                assert torch.equal(got[side][pg, :, slot], c.kv64[side][b][:, p])
    after = [x for x in (c.cache.k, c.cache.v, c.cache.k_exp, c.cache.v_exp) if x is not None]
    for x, y in zip(before, after):
        kind = torch.uint8 if x.dtype == torch.uint8 else torch.int16 if x.element_size() == 2 else torch.int32
        assert torch.equal(x.cpu().view(kind)[~owned], y.cpu().view(kind)[~owned])


@pytest.mark.parametrize("dtype,heads,d,page,lens,new,layout", MOVES)
def test_read_gives_the_stored_values_back(dtype, heads, d, page, lens, new, layout):
    c = Case(dtype, heads, heads, d, page, lens, new, layout)
    shape = (sum(new), heads, d) if layout == "packed" else (len(lens), heads, c.max_new + 2, d)
    k, v = (torch.full(shape, 7.0, dtype=c.t, device="cuda") for _ in range(2))
    c.cache.read(c.seqs, k, v)
    torch.cuda.synchronize()
    assert c.cache.device_error() == (C.PISA_OK, 0)
    for side, x in enumerate((k, v)):
        for b, (y, m) in enumerate(zip(c.split(x), new)):
            assert torch.equal(y.double(), c.kv64[side][b][:, lens[b] - m:])
            if layout == "padded":
                assert bool((x[b, :, m:] == 7.0).all())


@pytest.mark.parametrize("d", [64, 128])
def test_quantised_rows_of_every_size(d):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 60, d, generator=g) * torch.exp2(torch.arange(60.0) * 4 - 120)[None, :, None]
    x[0, 5] = 0.0
    x[0, 6] = 448.0
    x[0, 7, 1:] = 0.0
    x[0, 8] = -0.0
    c = Case("e4m3", 1, 1, d, 32, [60], [60], fill=False)
    c.k = c.v = [x.bfloat16()]
    c.kv64 = [[R.quantise(x.bfloat16())[0]]] * 2
    c.cache.append(c.seqs, c.tokens(c.k, 1).cuda(), c.tokens(c.v, 1).cuda())
    k, v = (torch.zeros(60, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.cache.read(c.seqs, k, v)
    assert torch.equal(k.cpu().double().transpose(0, 1), c.kv64[0][0])
    assert torch.equal(v.cpu(), k.cpu())


def test_quantised_rows_with_infinities_and_nan():
    d = 64
    x = torch.ones(1, 3, d)
    x[0, 0, 3], x[0, 0, 4] = float("inf"), -float("inf")
    x[0, 1, 5] = float("nan")
    x[0, 2] = 3e38
    c = Case("e4m3", 1, 1, d, 16, [3], [3], fill=False)
    c.k = c.v = [x.bfloat16()]
    c.cache.append(c.seqs, c.tokens(c.k, 1).cuda(), c.tokens(c.v, 1).cuda())
    k, v = (torch.zeros(3, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.cache.read(c.seqs, k, v)
    k = k.cpu().float()[:, 0]
    top = 448.0 * 2.0 ** 50
    assert k[0, 3] == top and k[0, 4] == -top and k[0, 0] == 0.0
    assert bool(k[1, 5].isnan()) and bool((k[1, :5] == 1.0).all())        # NaN has no part in the scale
    assert bool((k[2] == top).all())


def test_strided_token_tensors():
    """k, v and q as the parts of one fused projection, o with its heads first."""
    g = torch.Generator().manual_seed(5)
    c = Case("bf16", 6, 2, 64, 16, [50, 33], [20, 33], fill=False)
    T = 53
    fused = torch.randn(T, (6 + 2 * 2), 64, generator=g).bfloat16().cuda()
    q, k, v = fused[:, :6], fused[:, 6:8], fused[:, 8:]
    old = [Case.make(g, (2, 30, 64), 0.0).bfloat16(), torch.zeros(2, 0, 64).bfloat16()]
    first = Case.__new__(Case)
    first.__dict__.update(c.__dict__)
    first.lens, first.new, first.max_new = [30, 0], [30, 0], 30
    first.cache.append(first.sequences([30, 0]), first.tokens(old, 2).cuda(), first.tokens(old, 2).cuda())
    c.cache.append(c.seqs, k, v)
    parts = [x.cpu().split([20, 33]) for x in (q, k, v)]
    c.q = [x.transpose(0, 1) for x in parts[0]]
    c.kv64 = [[torch.cat([o, n.transpose(0, 1)], 1).double() for o, n in zip(old, p)] for p in parts[1:]]
    o = torch.full((6, T, 64), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    o2 = c.check(o=o)
    contiguous = torch.empty(T, 6, 64, dtype=torch.bfloat16, device="cuda")
    c.cache.attention(c.seqs, q, contiguous, softmax_scale=c.scale)
    assert torch.equal(contiguous, o2)


# ---- attention ---------------------------------------------------------------------------------
ATTENTION = [
    # heads, kv_heads, d, page, lens, new, layout, causal, window
    (1, 1, 128, 16, [1], [1], "packed", True, 0),
    (4, 2, 64, 16, [1, 2, 15, 16, 17], [1, 1, 1, 1, 1], "packed", True, 0),
    (16, 4, 128, 32, [577], [1], "packed", True, 0),
    (5, 1, 128, 64, [300, 0, 64, 129], [1, 0, 1, 1], "padded", True, 0),
    (24, 3, 64, 128, [130, 1027], [1, 1], "padded", False, 0),
    (40, 8, 128, 64, [700, 63], [1, 1], "packed", True, 100),
    (6, 2, 128, 16, [95, 40, 301], [5, 4, 7], "packed", True, 0),
    (16, 1, 64, 32, [333], [4], "packed", True, 0),
    (3, 3, 128, 64, [100, 64, 257], [40, 64, 17], "padded", True, 0),
    (2, 2, 128, 128, [520], [130], "packed", False, 0),
    (4, 2, 128, 16, [300, 129, 5], [129, 129, 5], "packed", True, 0),
    (6, 2, 64, 64, [400, 90], [65, 90], "padded", True, 33),
    (2, 1, 128, 32, [600], [260], "packed", False, 77),
    (8, 1, 128, 64, [150], [150], "packed", True, 1),
    (10, 2, 64, 16, [90, 270], [13, 51], "packed", False, 0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv,d,page,lens,new,layout,causal,window", ATTENTION)
def test_attention_matches_its_definition(dtype, heads, kv, d, page, lens, new, layout, causal, window):
    Case(dtype, heads, kv, d, page, lens, new, layout, seed=len(lens) + d).check(causal, window)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 9, 70])
def test_queries_outside_the_cache(dtype, new):
    """Without a causal mask the queries need not be in the cache: an empty one gives zeros, and more
    queries than keys are fine; causal rows before the first position see nothing."""
    for causal in (False, True):
        c = Case(dtype, 2, 1, 128, 16, [0, 3, 40], [0, 0, 0], "padded", max_new=new)
        c.new = [new] * 3
        g = torch.Generator().manual_seed(1)
        c.q = [Case.make(g, (2, new, 128), 0.0).to(c.t) for _ in range(3)]
        c.seqs = c.sequences(c.new)
        c.check(causal=causal)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale,spread", [(1.0, 6.0), (0.02, 1.0), (1.0, 40.0)])
def test_peaked_and_flat_rows(dtype, scale, spread):
    """Logits far apart (one key holds nearly all the weight, the maximum grows late) and nearly equal."""
    c = Case(dtype, 2, 2, 128, 32, [400, 130], [1, 130], scale=scale / math.sqrt(128), fill=False)
    for b in range(2):
        n = c.lens[b]
        ramp = torch.linspace(0.1, spread, n)[None, :, None]
        c.k[b] = (c.k[b].float() * ramp).to(c.t)
    c.kv64[0] = [R.quantise(x)[0] if dtype == "e4m3" else x.double() for x in c.k]
    full = Case.__new__(Case)
    full.__dict__.update(c.__dict__)
    full.new, full.max_new = list(c.lens), max(c.lens)
    c.cache.append(full.sequences(c.lens), full.tokens(c.k, 2).cuda(), full.tokens(c.v, 2).cuda())
    c.check()


@pytest.mark.parametrize("new", [1, 6, 40, 140])
def test_values_of_very_different_sizes(new):
    """e4m3 scales from 2^-40 to 2^40 inside one sequence: the scale rides on the weights' exponents."""
    c = Case("e4m3", 2, 1, 128, 16, [200], [new], fill=False)
    size = torch.exp2(torch.linspace(-40, 40, 200))[torch.randperm(200, generator=torch.Generator().manual_seed(0))]
    c.v[0] = (c.v[0].float() * size[None, :, None]).bfloat16()
    c.v[0][:, 50] = 0
    c.kv64[1] = [R.quantise(c.v[0])[0]]
    full = Case.__new__(Case)
    full.__dict__.update(c.__dict__)
    full.new, full.max_new = list(c.lens), max(c.lens)
    c.cache.append(full.sequences(c.lens), full.tokens(c.k, 1).cuda(), full.tokens(c.v, 1).cuda())
    c.check()


@pytest.mark.parametrize("dtype,bad", [("bf16", math.nan), ("bf16", math.inf), ("fp32", math.nan), ("fp32", math.inf),
                                       ("e4m3", math.nan)])      # 8-bit rows hold no infinities
@pytest.mark.parametrize("new,late", [(1, False), (3, True), (8, False), (8, True), (100, False), (100, True), (200, True)])
def test_what_a_token_does_not_see_has_no_part(dtype, new, late, bad):
    """Keys and values that are not finite reach exactly the tokens that see them."""
    c = Case(dtype, 4, 2, 128, 16, [300], [new], fill=False)
    hit = [300 - new // 2, 299] if late else []        # in the middle of the chunk, its last token
    for p in [20] + hit:                               # behind the window (of most)
        c.k[0][:, p, ::7] = bad
        c.v[0][:, p, ::5] = bad
    full = Case.__new__(Case)
    full.__dict__.update(c.__dict__)
    full.new, full.max_new = list(c.lens), 300
    c.cache.append(full.sequences(c.lens), full.tokens(c.k, 2).cuda(), full.tokens(c.v, 2).cuda())
    q = c.tokens(c.q, 4).cuda()
    o = torch.zeros_like(q)
    c.cache.attention(c.seqs, q, o, window=250, softmax_scale=c.scale)
    got = c.split(o)[0]
    for r in range(new):
        pos = 300 - new + r
        dirty = any(pos - 250 < p <= pos for p in hit + [20])
        if dirty:
            assert bool(got[:, r].isnan().any()), r
            continue
        clean = [torch.where(x[0].isfinite(), x[0], 0) for x in (c.k, c.v)]       # what is not finite is not seen here
        clean = [R.quantise(x)[0] if dtype == "e4m3" else x.double() for x in clean]
        for h in range(4):
            ref = R.attention(c.q[0][h, r:r + 1].double(), clean[0][h // 2], clean[1][h // 2], [pos], True, 250,
                              float(torch.tensor(c.scale, dtype=torch.float32)))
            bo, _ = R.bounds(ref, dtype, 128)
            assert bool(((got[h, r].double() - ref["o"][0]).abs() <= bo[0]).all()), (r, h)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [3, 21, 150])
def test_a_query_that_is_not_finite_harms_its_own_row_only(dtype, new):
    c = Case(dtype, 4, 2, 128, 32, [310], [new])
    c.q[0][1, 0, 3], c.q[0][2, new - 1, 5] = math.inf, math.nan
    got = c.split(c.cache.attention(c.seqs, c.tokens(c.q, 4).cuda(), softmax_scale=c.scale))[0]
    assert bool(got[1, 0].isnan().all()) and bool(got[2, new - 1].isnan().all())
    for h in range(4):
        for r in {0, 1, new // 2, new - 1}:
            if (h, r) in ((1, 0), (2, new - 1)):
                continue
            ref = R.attention(c.q[0][h, r:r + 1].double(), c.kv64[0][0][h // 2], c.kv64[1][0][h // 2], [310 - new + r], True, 0,
                              float(torch.tensor(c.scale, dtype=torch.float32)))
            bo, _ = R.bounds(ref, dtype, 128)
            assert bool(((got[h, r].double() - ref["o"][0]).abs() <= bo[0]).all()), (r, h)


@pytest.mark.parametrize("new", [4, 100])
def test_fp32_numbers_of_any_size(new):
    """Values near the type's ends, and logits that lean on bits a shorter type does not hold."""
    c = Case("fp32", 2, 1, 64, 16, [200], [new], fill=False)
    g = torch.Generator().manual_seed(8)
    c.v[0] *= torch.exp2(torch.randint(-140, 120, c.v[0].shape, generator=g).float())
    c.v[0][:, 50, 3], c.v[0][:, 51, 4] = 3.4028e38, -3.4028e38
    c.k[0] = c.k[0] * 2.0 ** -40
    c.q[0] = c.q[0] * 2.0 ** 40
    full = Case.__new__(Case)
    full.__dict__.update(c.__dict__)
    full.new, full.max_new = list(c.lens), 200
    c.cache.append(full.sequences(c.lens), full.tokens(c.k, 1).cuda(), full.tokens(c.v, 1).cuda())
    got = c.split(c.cache.attention(c.seqs, c.tokens(c.q, 2).cuda(), softmax_scale=c.scale))[0]
    for h in range(2):
        for r in {0, new // 2, new - 1}:
            ref = R.attention(c.q[0][h, r:r + 1].double(), c.k[0][0].double(), c.v[0][0].double(), [200 - new + r], True, 0,
                              float(torch.tensor(c.scale, dtype=torch.float32)))
            bo, _ = R.bounds(ref, "fp32", 64)
            assert bool(((got[h, r].double() - ref["o"][0]).abs() <= bo[0]).all()), (r, h)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 3, 21, 90])
def test_many_sequences(dtype, new):
    """More sequences than a warp has lanes, with lengths from nothing to several tiles, some of them idle."""
    n = 75
    lens = [(37 * b * b) % 211 for b in range(n)]
    fresh = [min(m, new if b % 3 else 0) for b, m in enumerate(lens)]
    Case(dtype, 4, 2, 64, 16, lens, fresh, "packed" if new % 2 else "padded", seed=new).check(rows=(0, 1, 20, 89))


def test_no_rows_at_all():
    c = Case("bf16", 2, 2, 64, 16, [40, 50], [0, 0], max_new=4)
    before = c.cache.k.clone()
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    c.cache.append(c.seqs, none, none)
    c.cache.read(c.seqs, none, none.clone())
    assert c.cache.attention(c.seqs, none).shape == (0, 2, 64)
    torch.cuda.synchronize()
    assert c.cache.device_error() == (C.PISA_OK, 0)
    assert torch.equal(before.view(torch.int16), c.cache.k.view(torch.int16))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 20, 150])
def test_pages_before_a_window_may_be_gone(dtype, new):
    """A sliding window lets a program free the pages behind it: their table entries are not read."""
    c = Case(dtype, 4, 2, 128, 16, [700], [new])
    gone = (700 - new - 64 + 1) // 16          # whole pages before what the first new token sees
    c.seqs.tensors[0][0, :gone] = -1
    c.check(window=64)


def test_the_same_call_twice_gives_the_same_bits():
    """Parts of an item are joined in the order of the blocks, whichever ends last."""
    for dtype in DTYPES:
        for new in (1, 12, 300):
            c = Case(dtype, 4, 1, 128, 64, [3000], [new], seed=3)
            q = c.tokens(c.q, 4).cuda()
            outs = [c.cache.attention(c.seqs, q, softmax_scale=c.scale) for _ in range(4)]
            assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_contexts_of_few_heads(dtype):
    """One head's keys over many blocks, against torch in float64 on the device."""
    n, heads, d = 20011, 3, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    t = R.DTYPES[dtype]
    cache = PagedCache(700, heads, 1, 32, d, dtype)
    k, v = (torch.randn(n, 1, d, generator=g, device="cuda").to(t) for _ in range(2))
    table = torch.randperm(700, generator=torch.Generator().manual_seed(2))[None, :626].to(torch.int32).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    whole = cache.sequences(table, i32(n), n, n, starts=i32(0, n))
    cache.append(whole, k, v)
    kk, vv = torch.empty_like(k), torch.empty_like(v)
    cache.read(whole, kk, vv)
    for new in (1, 4, 20, 130, 1000):
        q = torch.randn(new, heads, d, generator=g, device="cuda").to(t)
        o = cache.attention(cache.sequences(table, i32(n), n, new, starts=i32(0, new)), q, softmax_scale=0.125)
        s = torch.einsum("qhd,kd->hqk", q.double(), kk[:, 0].double()) * 0.125
        s.masked_fill_(torch.arange(n, device="cuda")[None] > torch.arange(n - new, n, device="cuda")[:, None], -math.inf)
        w = torch.softmax(s, -1)
        ref, size = w @ vv[:, 0].double(), w @ vv[:, 0].double().abs()
        # the bounds of cache_reference.py: |logit| <= 0.125 * 64 * 25
        weight = {"bf16": 2.0 ** -8, "fp32": 0.0, "e4m3": 2.0 ** -11}[dtype]
        rel = weight + 2 * ((d + 4) * 2.0 ** -23 * 200 + 2.0 ** -21) + 2 * n * 2.0 ** -23
        bound = size * rel * 1.01 + R.HALF_STEP[dtype] * ref.abs() + (n * 2.0 ** -24 * vv.double().abs().max() if dtype == "e4m3" else 0)
        assert bool(((o.transpose(0, 1).double() - ref).abs() <= bound).all()), new
    assert cache.device_error() == (C.PISA_OK, 0)


def test_bad_lengths_and_pages_are_reported_and_not_followed():
    def fresh(layout="packed", new=(3, 4, 5)):
        return Case("bf16", 2, 2, 64, 16, [40, 50, 60], list(new), layout)

    # a length beyond the bound: that sequence counts as empty, the others are right
    c = fresh()
    good = c.check()
    c.seqs.tensors[1][1] = 61
    q = c.tokens(c.q, 2).cuda()
    o = torch.full_like(q, 7.0)
    c.cache.attention(c.seqs, q, o, softmax_scale=c.scale)
    assert c.cache.device_error() == (C.PISA_ERR_INVALID_ARG, C.PISA_DEVERR_BAD_LENGTH)
    assert c.cache.device_error() == (C.PISA_OK, 0)
    a, g = c.split(o), c.split(good)
    assert torch.equal(a[0], g[0]) and torch.equal(a[2], g[2]) and bool((a[1] == 0).all())
    # starts that leave the tensor or go backwards: skipped
    for bad in ([0, 3, 2, 12], [0, 3, 7, 13], [-1, 3, 7, 12], [0, 3, 9, 12]):
        c = fresh()
        c.seqs.tensors[2].copy_(torch.tensor(bad, dtype=torch.int32))
        o = torch.full_like(q, 7.0)
        c.cache.attention(c.seqs, c.tokens(c.q, 2).cuda(), o, softmax_scale=c.scale)
        assert c.cache.device_error()[1] == C.PISA_DEVERR_BAD_LENGTH
        k, v = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
        before = c.cache.k.clone()
        c.cache.read(c.seqs, k, v)
        assert c.cache.device_error()[1] == C.PISA_DEVERR_BAD_LENGTH
        if bad[1] == 3 and bad[0] == 0:
            assert torch.equal(k[:3].cpu().double().transpose(0, 1), c.kv64[0][0][:, 37:])
        assert torch.equal(before.view(torch.int16), c.cache.k.view(torch.int16))
    # more new tokens than the sequence has: neither append nor read touches it
    c = fresh("padded")
    c.seqs.tensors[1][0] = 2
    k, v = (torch.full((3, 2, 5, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.cache.read(c.seqs, k, v)
    assert c.cache.device_error()[1] == C.PISA_DEVERR_BAD_LENGTH
    assert bool((k[0] == 7.0).all()) and torch.equal(k[1, :, :4].cpu().double(), c.kv64[0][1][:, 46:])
    # a page out of range: its keys are not seen, its tokens neither written nor read
    for bad in (-1, 10**6):
        c = fresh("padded")
        c.seqs.tensors[0][2, 1] = bad                  # positions 16 ... 31 of the last sequence
        qp = c.tokens(c.q, 2).cuda()
        o = torch.full_like(qp, 7.0)
        c.cache.attention(c.seqs, qp, o, softmax_scale=c.scale)
        assert c.cache.device_error() == (C.PISA_ERR_INVALID_ARG, C.PISA_DEVERR_BAD_PAGE)
        keep = [p for p in range(60) if not 16 <= p < 32]
        for h in range(2):
            ref = R.attention(c.q[2][h].double(), c.kv64[0][2][h][keep], c.kv64[1][2][h][keep], [39 + r for r in range(5)],
                              True, 0, float(torch.tensor(c.scale, dtype=torch.float32)))
            bo, _ = R.bounds(ref, "bf16", 64)
            assert bool(((o[2, h].cpu().double() - ref["o"]).abs() <= bo).all())


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements, the sequence in its last pages."""
    pages, page, d = (1 << 31) // (128 * 128) + 40, 128, 128
    k = torch.zeros(pages, 1, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    cache = PagedCache(pages, 2, 1, page, d, k=k, v=v)
    n, m = 300, 200
    g = torch.Generator(device="cuda").manual_seed(2)
    kk, vv = (torch.randn(n, 1, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(m, 2, d, generator=g, device="cuda").bfloat16()
    table = torch.tensor([[pages - 1, pages - 30, pages - 2]], dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache.append(cache.sequences(table, i32(n), n, n, starts=i32(0, n)), kk, vv)
    assert torch.equal(k[pages - 1, 0], kk[:128, 0]) and torch.equal(v[pages - 2, 0, :44], vv[256:, 0])
    for m_ in (1, m):
        o = cache.attention(cache.sequences(table, i32(n), n, m_, starts=i32(0, m_)), q[m - m_:], softmax_scale=0.1)
        for h in range(2):
            s = (q[m - m_:, h].double() @ kk[:, 0].double().T) * 0.1
            s.masked_fill_(torch.arange(n, device="cuda")[None] > torch.arange(n - m_, n, device="cuda")[:, None], -math.inf)
            ref = torch.softmax(s, -1) @ vv[:, 0].double()
            assert (o[:, h].double() - ref).norm() <= 2 * 2.0 ** -8 * ref.norm()


# ---- together ----------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_chunk_and_then_token_after_token(dtype):
    """As a program uses them: a prompt enters in chunks, then tokens one by one, each attending."""
    g = torch.Generator().manual_seed(11)
    heads, kv, d, page, total = 4, 2, 64, 16, 75
    t = R.DTYPES[dtype]
    cache = PagedCache(8, heads, kv, page, d, dtype)
    k, v = (Case.make(g, (total, kv, d), 0.5).to(t) for _ in range(2))
    q = Case.make(g, (total, heads, d), 0.0).to(t)
    held = [R.quantise(x)[0] if dtype == "e4m3" else x.double() for x in (k, v)]
    table = torch.tensor([[5, 0, 7, 2, 6]], dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = 0
    for m in [30, 35] + [1] * 10:
        lens += m
        seqs = cache.sequences(table, lens, max_len=80, max_new=m)
        part = lambda x: x[at:at + m].transpose(0, 1)[None].cuda()
        cache.append(seqs, part(k), part(v))
        o = cache.attention(seqs, part(q), softmax_scale=0.125)
        for h in range(heads):
            ref = R.attention(q[at:at + m, h].double(), held[0][:at + m, h // 2], held[1][:at + m, h // 2],
                              list(range(at, at + m)), True, 0, 0.125)
            bo, _ = R.bounds(ref, dtype, d)
            assert bool(((o[0, h].cpu().double() - ref["o"]).abs() <= bo).all())
        at += m
    assert cache.device_error() == (C.PISA_OK, 0)


@pytest.mark.parametrize("dtype", ("bf16", "e4m3"))
def test_frames_through_the_cache_into_the_sparse_path(dtype):
    """Frames are appended, read back dense and given to PISA; with every block kept it is dense
    attention, which the cache's own attention over the same tokens has to equal."""
    g = torch.Generator(device="cuda").manual_seed(4)
    H, d, frame, frames, page = 2, 128, 96, 4, 64
    L = frame * frames
    cache = PagedCache(16, H, H, page, d, dtype)
    q, k, v = (torch.randn(1, H, L, d, generator=g, device="cuda").bfloat16() for _ in range(3))
    q = (q.float() / math.sqrt(d)).bfloat16()
    table = torch.randperm(16, generator=torch.Generator().manual_seed(0))[None, :6].to(torch.int32).cuda()
    for f in range(frames):
        lens = torch.tensor([frame * (f + 1)], dtype=torch.int32, device="cuda")
        s = cache.sequences(table, lens, max_len=L, max_new=frame)
        part = slice(f * frame, (f + 1) * frame)
        cache.append(s, k[:, :, part], v[:, :, part])
    whole = cache.sequences(table, lens, max_len=L, max_new=L)
    kd, vd = torch.empty_like(k), torch.empty_like(v)
    cache.read(whole, kd, vd)
    if dtype == "bf16":
        assert torch.equal(kd, k) and torch.equal(vd, v)
    o_cache = cache.attention(whole, q, causal=False)
    p = Pisa(1, H, L, d, 64, -(-L // 64), 0.5)
    o_pisa = p(q, kd, vd)
    torch.cuda.synchronize()
    assert cache.device_error() == (C.PISA_OK, 0) and p.device_error() == (C.PISA_OK, 0)
    for h in range(H):
        ref = R.attention(q[0, h].cpu().double(), kd[0, h].cpu().double(), vd[0, h].cpu().double(), list(range(L)), False, 0, 1.0)
        bo, _ = R.bounds(ref, "bf16", d)
        for o in (o_cache, o_pisa):
            assert bool(((o[0, h].cpu().double() - ref["o"]).abs() <= bo).all())


def test_joining_two_caches_by_lse():
    c = Case("bf16", 2, 1, 128, 16, [200], [9])
    o = c.check(causal=False)
    q = c.tokens(c.q, 2).cuda()
    parts = []
    for first, n in ((0, 96), (96, 104)):
        table = c.table[:, first // 16:].contiguous().cuda()
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        s = c.cache.sequences(table, lens, max_len=104, max_new=9, starts=torch.tensor([0, 9], dtype=torch.int32, device="cuda"))
        lse = torch.empty(9, 2, device="cuda")
        parts.append((c.cache.attention(s, q, causal=False, softmax_scale=c.scale, lse=lse).float(), lse))
    (a, la), (b, lb) = parts
    wa = torch.sigmoid(la - lb)[..., None]
    # three roundings to bf16 and the weights' own, each at most 2^-8
    assert ((a * wa + b * (1 - wa)) - o.float()).abs().max() <= 4 * 2.0 ** -8 * c.kv64[1][0].abs().max()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 20, 150])
def test_captured_step_follows_the_lengths(dtype, new):
    """append and attention recorded once as a CUDA graph and replayed as the sequence grows."""
    g = torch.Generator(device="cuda").manual_seed(9)
    heads, kv, d, page = 4, 2, 128, 32
    t = R.DTYPES[dtype]
    cache, eager = (PagedCache(40, heads, kv, page, d, dtype) for _ in range(2))
    table = torch.randperm(40, generator=torch.Generator().manual_seed(1))[:32].reshape(2, 16).to(torch.int32).cuda()
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(2, n, new, d, dtype=t, device="cuda") for n in (heads, kv, kv))
    o = torch.zeros_like(q)
    seqs, other = (c.sequences(table, lens, max_len=512, max_new=new) for c in (cache, eager))

    def step(c, s, out):
        c.append(s, k, v)
        c.attention(s, q, out, softmax_scale=0.1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lens += new
    with torch.cuda.stream(side):
        step(cache, seqs, o)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(cache, seqs, o)
    for i in range(3):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        if i:
            lens += torch.tensor([new, 0 if i == 2 else new], dtype=torch.int32, device="cuda")
        graph.replay()
        o2 = torch.zeros_like(o)
        step(eager, other, o2)
        assert torch.equal(o, o2)
    torch.cuda.synchronize()
    assert cache.device_error() == (C.PISA_OK, 0)


def test_calls_on_other_streams():
    c = Case("bf16", 8, 2, 128, 64, [900, 400], [1, 1])
    want = c.check()
    q = c.tokens(c.q, 8).cuda()
    torch.cuda.synchronize()
    caches = [PagedCache(c.cache.num_pages, 8, 2, 64, 128, k=c.cache.k, v=c.cache.v) for _ in range(3)]   # a workspace each
    outs = []
    for cache in caches:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        s = cache.sequences(*c.seqs.tensors[:2], max_len=c.max_len, max_new=1, starts=c.seqs.tensors[2])
        o = torch.zeros_like(q)
        torch.cuda.synchronize()
        for _ in range(20):
            cache.attention(s, q, o, softmax_scale=c.scale, stream=st)
        outs.append(o)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_an_output_made_by_the_call_belongs_to_its_stream():
    """The zeros that the call begins with are written before its results, on whichever stream it runs."""
    c = Case("bf16", 8, 2, 128, 64, [900, 400], [1, 1])
    want = c.check()
    q, st = c.tokens(c.q, 8).cuda(), torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        x = x @ x.clamp(-1, 1)               # the current stream is busy for some milliseconds
    o = c.cache.attention(c.seqs, q, softmax_scale=c.scale, stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(o, want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
def test_windows_as_long_as_the_type_allows(dtype, causal):
    """More new tokens than the sequence holds: the first ones stand before position 0."""
    c = Case(dtype, 4, 2, 64, 16, [40, 7], [60, 9], fill=False, max_new=60)
    whole = Case.__new__(Case)
    whole.__dict__.update(c.__dict__)
    whole.new, whole.max_new = list(c.lens), 40
    c.cache.append(whole.sequences(c.lens), whole.tokens(c.k, 2).cuda(), whole.tokens(c.v, 2).cuda())
    c.check(causal=causal, window=2 ** 31 - 1)
    c.check(causal=causal, window=50)
