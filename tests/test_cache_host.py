"""Host-side checks of the paged cache's entry points: what they refuse, before anything is launched."""
import ctypes

import pytest
import torch

from piecewise_approximate_attention_b200 import _lib as C
from piecewise_approximate_attention_b200.runtime import PagedCache
from tests import cache_reference as R

P = 1 << 28          # never dereferenced: every call below is refused, or has nothing to do


def _cache(**kw):
    base = dict(num_pages=9, kv_heads=2, page=64, head_dim=128, dtype=C.PISA_CACHE_BF16, k=P, v=P, k_exp=None, v_exp=None)
    base.update(kw)
    return C.PisaCache(**base)


def _seqs(**kw):
    base = dict(batch=3, max_pages=4, max_len=256, max_new=8, page_table=P, lens=P, starts=None, counts=None)
    base.update(kw)
    return C.PisaSequences(**base)


def _rows(**kw):
    base = dict(data=P, rows=8, seq_stride=8 * 4 * 128, row_stride=128, head_stride=8 * 128)
    base.update(kw)
    return C.PisaRows(**base)


def _append(cache, seqs, k=None, v=None, ws=P, n=1 << 40, fn="pisa_cache_append"):
    return getattr(C.lib(), fn)(cache, seqs, k or _rows(), v or _rows(), ws, n, None)


def _read(*a, **kw):
    return _append(*a, fn="pisa_cache_read", **kw)


def _attention(cache, seqs, q=None, o=None, heads=4, causal=1, window=0, scale=1.0, lse=None, ws=P, n=1 << 40):
    return C.lib().pisa_cache_attention(cache, seqs, heads, causal, window, scale, q or _rows(),
                                        o or _rows(data=2 * P), lse, ws, n, None)


CALLS = [_append, _read, _attention]
INV, UNS = C.PISA_ERR_INVALID_ARG, C.PISA_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,expect", [
    (dict(num_pages=0), INV), (dict(kv_heads=0), INV), (dict(page=0), INV), (dict(head_dim=0), INV),
    (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(k=P + 8), INV),
    (dict(head_dim=96), UNS), (dict(page=48), UNS), (dict(page=256), UNS), (dict(page=8), UNS),
    (dict(num_pages=1 << 25), UNS), (dict(kv_heads=1 << 20), UNS), (dict(num_pages=2**31 - 1, kv_heads=65535), UNS),
    (dict(dtype=C.PISA_CACHE_E4M3), INV), (dict(dtype=C.PISA_CACHE_E4M3, k_exp=P, v_exp=P + 4), INV),
])
def test_bad_caches_are_refused(call, kw, expect):
    assert call(_cache(**kw), _seqs()) == expect


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,expect", [
    (dict(batch=-1), INV), (dict(max_pages=-1), INV), (dict(max_len=-1), INV), (dict(max_new=-1), INV),
    (dict(max_len=257), INV), (dict(page_table=None), INV), (dict(lens=None), INV), (dict(lens=P + 2), INV),
    (dict(starts=P, counts=P), INV), (dict(batch=65536), UNS),
])
def test_bad_sequences_are_refused(call, kw, expect):
    assert call(_cache(), _seqs(**kw)) == expect


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw", [
    dict(data=None), dict(data=P + 8), dict(rows=-1), dict(rows=7), dict(row_stride=-128), dict(row_stride=132),
    dict(head_stride=1 << 50), dict(seq_stride=4),
])
def test_bad_token_tensors_are_refused(call, kw):
    for bad in (dict(), dict(second=True)):
        a, b = (_rows(data=2 * P), _rows(**kw)) if bad else (_rows(**kw), _rows(data=2 * P))
        assert call(_cache(), _seqs(), a, b) == INV


def test_outputs_whose_rows_fall_on_one_another_are_refused():
    for kw in (dict(row_stride=0), dict(row_stride=64), dict(head_stride=0), dict(seq_stride=64)):
        assert _read(_cache(), _seqs(), _rows(**kw)) == INV
        assert _attention(_cache(), _seqs(), o=_rows(data=2 * P, **kw)) == INV
    # the sequences' stride has no meaning for packed rows, and a single row or head needs none
    assert _attention(_cache(), _seqs(starts=P, max_new=0), o=_rows(data=2 * P, seq_stride=1)) == C.PISA_OK


def test_bad_workspaces_are_refused():
    n = C.pisa_cache_workspace_bytes(_cache())
    assert n >= 256
    for call in CALLS:
        for kw in (dict(ws=None), dict(ws=P + 4), dict(n=n - 1)):
            assert call(_cache(), _seqs(), **kw) == INV
    assert C.pisa_cache_workspace_bytes(_cache(head_dim=96)) == 0
    assert C.pisa_cache_workspace_bytes(_cache(dtype=9)) == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(heads=0), INV), (dict(heads=3), INV), (dict(heads=-2), INV), (dict(heads=1 << 20), UNS), (dict(window=-1), INV),
    (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(scale=3e38), INV),
    (dict(lse=P + 2), INV), (dict(o=_rows()), INV), (dict(o=_rows(data=2 * P, rows=8), q=_rows(rows=9)), INV),
])
def test_bad_attention_arguments_are_refused(kw, expect):
    assert _attention(_cache(), _seqs(), **kw) == expect


@pytest.mark.parametrize("call", CALLS)
def test_nothing_to_do_launches_nothing(call):
    # on a machine without a GPU a launch would report PISA_ERR_CUDA
    assert call(_cache(), _seqs(batch=0, lens=None, page_table=None)) == C.PISA_OK
    assert call(_cache(), _seqs(max_new=0)) == C.PISA_OK


@pytest.mark.parametrize("call", CALLS)
def test_an_empty_packed_tensor_is_nothing_to_do(call):
    none = _rows(data=None, rows=0)
    assert call(_cache(), _seqs(starts=P), none, none) == C.PISA_OK
    assert call(_cache(), _seqs(), none, none) == INV                              # padded rows are there
    assert call(_cache(), _seqs(starts=P), _rows(data=None, rows=1), none) == INV


def test_row_numbers_that_do_not_fit_are_refused():
    assert _attention(_cache(), _seqs(max_new=1 << 30), heads=4, q=_rows(rows=1 << 30), o=_rows(data=2 * P, rows=1 << 30)) == UNS
    big = dict(max_new=1 << 22, max_pages=1 << 20, max_len=1 << 26)
    assert _attention(_cache(), _seqs(**big), q=_rows(rows=1 << 22), o=_rows(data=2 * P, rows=1 << 22)) == UNS


def test_binding_checks_its_tensors():
    with pytest.raises(ValueError, match="dtype"):
        PagedCache(4, 2, 2, 16, 64, "fp16", device="cpu")
    with pytest.raises(ValueError, match="multiple"):
        PagedCache(4, 3, 2, 16, 64, device="cpu")
    with pytest.raises(C.PisaError):
        PagedCache(4, 2, 2, 24, 64, device="cpu")
    with pytest.raises(ValueError, match="k must be"):
        PagedCache(4, 2, 2, 16, 64, device="cpu", k=torch.zeros(4, 2, 16, 64))
    c = PagedCache(4, 4, 2, 16, 64, "e4m3", device="cpu")
    assert c.k.dtype == torch.uint8 and c.k_exp.shape == (4, 2, 16)
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(page_table=table.long(), lens=lens), dict(page_table=table, lens=lens.long()),
                dict(page_table=table[:2], lens=lens), dict(page_table=table, lens=lens, starts=lens),
                dict(page_table=table, lens=lens, counts=table[0]), dict(page_table=table.t(), lens=lens[:2]),
                dict(page_table=table, lens=lens, counts=lens, starts=torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            c.sequences(max_len=32, max_new=5, **bad)
    seqs = c.sequences(table, lens, max_len=32, max_new=5)
    good = torch.zeros(3, 2, 5, 64, dtype=torch.bfloat16)
    for bad in (good.float(), good[:2], good[:, :1], good[..., :32], good.transpose(2, 3), good[0]):
        with pytest.raises(ValueError):
            c.append(seqs, bad, good)
        with pytest.raises(ValueError):
            c.read(seqs, good, bad)
    q = torch.zeros(3, 4, 5, 64, dtype=torch.bfloat16)
    for kw in (dict(o=q[:, :, :4]), dict(lse=torch.zeros(3, 5, 4)), dict(lse=torch.zeros(3, 4, 5).double())):
        with pytest.raises(ValueError):
            c.attention(seqs, q, **kw)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        c.attention(seqs, q)


def test_reference_quantisation_is_e4m3():
    # against torch's own e4m3 type, at scales that are given
    x = torch.linspace(-448, 448, 4097).bfloat16().float()[None]
    got, e = R.quantise(x)
    assert e.item() == 0 and torch.equal(got.float(), x.to(torch.float8_e4m3fn).float())
    for top, e_want in ((448.0, 0), (450.0, 1), (447.0, 0), (1.75, -8), (1.7578125, -7), (2.0 ** -70, -50), (0.0, -50),
                        (3e38, 50)):
        got, e = R.quantise(torch.tensor([[top, -top / 2]]))
        assert e.item() == e_want, top


def test_reference_attention_by_hand():
    q = torch.zeros(2, 4, dtype=torch.float64)
    k = torch.randn(3, 4, dtype=torch.float64)
    v = torch.arange(3.0, dtype=torch.float64)[:, None].expand(3, 4).clone()
    v[2] = float("nan")
    r = R.attention(q, k, v, [0, 1], True, 0, 1.0)          # equal logits: means of what is seen
    assert r["o"][0, 0] == 0 and r["o"][1, 0] == 0.5 and torch.allclose(r["lse"].exp(), torch.tensor([1.0, 2.0]).double())
    r = R.attention(q, k, v, [1, -1], True, 1, 1.0)         # a window of one key; a row that sees nothing
    assert r["o"][0, 0] == 1.0 and r["o"][1].abs().sum() == 0 and r["lse"][1] == -float("inf")
