"""Buffers and call sequence for one PISA attention shape (pre-compute -> route -> attention).

All three steps run in the CUDA library through the C ABI; this module only allocates device
memory with torch and passes pointers and the current stream.
"""
from __future__ import annotations

from typing import Optional

from . import _lib as C


class Pisa:
    """Reusable PISA attention for a fixed [B, H, L, d] shape, block size, keep_k and lambda.

    ``pair=True`` asks the router for the query-block pairing order used by 128-row tiles when
    block == 64 (a scheduling choice: the output does not depend on it).  ``first_order=False``
    makes ``precompute`` write the zeroth-order statistics only (pisa_precompute_zeroth_order):
    enough for lambda = 0 routing and the keep-or-drop mode, i.e. an exact-only pipeline.
    """

    def __init__(self, batch: int, heads: int, seq_len: int, head_dim: int, block: int, keep_k: int,
                 lam: float, dtype: str = "bf16", softmax_scale: float = 1.0, device="cuda",
                 mode: int = C.PISA_MODE_PISA, with_H: bool = False, pair: bool = True,
                 first_order: bool = True):
        import torch
        if not first_order and (lam != 0.0 or mode != C.PISA_MODE_EXACT_ONLY):
            raise ValueError("the zeroth-order statistics serve lambda = 0 routing and PISA_MODE_EXACT_ONLY only")
        self.first_order = first_order
        self.shape = C.make_shape(batch, heads, seq_len, head_dim, block, dtype, softmax_scale)
        self.block, self.keep_k, self.lam, self.mode = block, keep_k, lam, mode
        self.nb = C.pisa_num_blocks(seq_len, block)
        self.device = torch.device(device)
        self.tdtype = torch.float32 if dtype == "fp32" else torch.bfloat16
        self.fp8 = dtype == "bf16_fp8qk"
        self._torch_f32 = torch.float32
        if mode == C.PISA_MODE_PER_BLOCK:
            with_H = True         # the per-block first-order matrices live in the stats
        self.stats = C.alloc_stats(self.shape, self.device, with_H)
        self.ws = C.alloc_workspace(self.shape, self.device, per_block=mode == C.PISA_MODE_PER_BLOCK)
        self.sel = torch.empty((batch, heads, self.nb, max(keep_k, 1)), dtype=torch.int32, device=self.device)
        self.order = torch.empty((batch, heads, self.nb), dtype=torch.int32, device=self.device) if pair else None

    def precompute(self, q, k, v, stream=None):
        if self.first_order:
            C.pisa_precompute(self.shape, q, k, v, self.stats, self.ws, stream)
        else:
            C.pisa_precompute_zeroth_order(self.shape, q, k, v, self.stats, self.ws, stream)

    def fused_short_step(self) -> bool:
        """Whether precompute_route(fused=True) is one cluster launch (bf16 inputs, head_dim 128,
        nb <= 128; the device must also fit every head's cluster at once)."""
        return self.first_order and self.tdtype != self._torch_f32 and self.shape.head_dim == 128 and self.nb <= 128

    def precompute_route(self, q, k, v, scores=None, stream=None, fused: bool = False):
        """Pre-computation and routing through pisa_precompute_route: the separate kernels, or with
        ``fused`` (short sequences) one cluster launch; the results are the same either way."""
        if not self.first_order:
            self.precompute(q, k, v, stream)
            self.route(scores, stream)
            return
        C.pisa_precompute_route(self.shape, q, k, v, self.stats, self.keep_k, self.lam, self.sel, self.order, scores,
                                self.ws, fused, stream)

    def route(self, scores=None, stream=None):
        C.pisa_route(self.shape, self.stats, self.keep_k, self.lam, self.sel, self.order, scores, stream)

    def attention(self, q, k, v, o, sel=None, order=None, mode: Optional[int] = None, stream=None):
        s = self.sel if sel is None else sel
        od = self.order if order is None else order
        C.pisa_attention(self.shape, q, k, v, self.stats, s, od, self.keep_k, self.mode if mode is None else mode,
                         o, self.ws, stream)

    def __call__(self, q, k, v, o=None, stream=None):
        import torch
        if o is None:
            o = torch.empty_like(q)
        self.precompute_route(q, k, v, stream=stream)
        self.attention(q, k, v, o, stream=stream)
        return o

    def capture(self, q, k, v, o, fused: bool = False):
        """Records one full step (pre-computation, routing, attention of q, k, v into o) as a CUDA
        graph and returns it; ``graph.replay()`` then re-runs the step on whatever the same
        buffers hold, with one launch from the host.  The buffers must stay allocated while the
        graph is used.  The step runs once eagerly first (outside the capture).  ``fused=True``
        records the fused pre-computation and routing (short sequences) instead of the separate
        calls."""
        import torch
        side = torch.cuda.Stream(self.device)
        side.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(side):
            self(q, k, v, o)
        torch.cuda.current_stream(self.device).wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            self.precompute_route(q, k, v, fused=fused)
            self.attention(q, k, v, o)
        return graph

    def launches_per_step(self) -> int:
        """Kernels one __call__ enqueues: pre-compute 3 (2 zeroth-order only on the bf16 path, 1 on
        the fp32 path; +3 e4m3 quantizations), routing 1 (+1 pairing), attention 1 (+1 for the
        per-block first-order kernel on the bf16 path)."""
        extra = 1 if (self.mode == C.PISA_MODE_PER_BLOCK and self.tdtype != self._torch_f32 and
                      self.keep_k < self.nb) else 0
        pre = 3 if self.first_order else (1 if self.tdtype == self._torch_f32 else 2)
        route = 1 + (1 if self.order is not None else 0)
        return pre + (3 if self.fp8 else 0) + route + 1 + extra

    def device_error(self, stream=None):
        return C.pisa_read_device_error(self.ws, stream)


_INT32_MAX = 2 ** 31 - 1


def _int32(name: str, x: int) -> int:
    """ctypes would cut what does not fit."""
    if not 0 <= x <= _INT32_MAX:
        raise ValueError(f"{name} must lie in [0, 2^31), not be {x}")
    return x


class Sequences:
    """Which tokens a call on a PagedCache is about; made by PagedCache.sequences, reusable for any
    number of calls (every layer of a step) while its tensors hold what is meant."""

    def __init__(self, c, packed: bool, batch: int, tensors):
        self.c, self.packed, self.batch, self.tensors = c, packed, batch, tensors


class PagedCache:
    """Keys and values of earlier tokens in pages of ``page`` tokens, for ``heads`` query heads on
    ``kv_heads`` key/value heads (pisa_cache.h): ``append`` stores new tokens, ``read`` gives stored
    tokens back dense, ``attention`` lets new tokens attend over them.

    ``dtype``: "bf16", "fp32", or "e4m3" (8-bit codes with a power-of-two scale per token and head,
    for bf16 tokens).  The pool tensors ``k``, ``v`` [num_pages, kv_heads, page, head_dim] (uint8 codes
    for e4m3) and ``k_exp``, ``v_exp`` [num_pages, kv_heads, page] (uint8) are allocated here unless given;
    a pool made here holds zeros.
    One workspace: calls on one PagedCache must not run at the same time on the device.
    """

    DTYPES = {"bf16": C.PISA_CACHE_BF16, "fp32": C.PISA_CACHE_FP32, "e4m3": C.PISA_CACHE_E4M3}

    def __init__(self, num_pages: int, heads: int, kv_heads: int, page: int, head_dim: int, dtype: str = "bf16",
                 device="cuda", k=None, v=None, k_exp=None, v_exp=None):
        import torch
        if dtype not in self.DTYPES:
            raise ValueError(f"dtype must be one of {sorted(self.DTYPES)}")
        if heads < 1 or kv_heads < 1 or heads % kv_heads:
            raise ValueError("heads must be a multiple of kv_heads")
        for name, x in (("num_pages", num_pages), ("heads", heads), ("page", page), ("head_dim", head_dim)):
            _int32(name, x)
        self.num_pages, self.heads, self.kv_heads, self.page, self.head_dim = num_pages, heads, kv_heads, page, head_dim
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.tdtype = torch.float32 if dtype == "fp32" else torch.bfloat16
        self.fp8 = dtype == "e4m3"
        sizes = C.PisaCache(num_pages, kv_heads, page, head_dim, self.DTYPES[dtype])
        n = C.pisa_cache_workspace_bytes(sizes)
        if n == 0:
            raise C.PisaError(C.PISA_ERR_UNSUPPORTED, "pisa_cache_workspace_bytes")
        shape = (num_pages, kv_heads, page, head_dim)
        pool = torch.uint8 if self.fp8 else self.tdtype

        def buffer(x, shape, dtype, name, fill=0):
            if x is None:
                return torch.full(shape, fill, dtype=dtype, device=self.device)
            if tuple(x.shape) != shape or x.dtype != dtype or x.device != self.device or not x.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on {self.device}")
            return x

        self.k, self.v = buffer(k, shape, pool, "k"), buffer(v, shape, pool, "v")
        # 2^-50 is the scale that a row of zeros is stored with; a byte of 0 is no scale of the format
        scale = C.PISA_CACHE_EXP_MIN
        self.k_exp = buffer(k_exp, shape[:3], torch.uint8, "k_exp", scale) if self.fp8 else None
        self.v_exp = buffer(v_exp, shape[:3], torch.uint8, "v_exp", scale) if self.fp8 else None
        self.ws = torch.zeros(n, dtype=torch.uint8, device=self.device)
        self._ws_at, self._ws_bytes = self.ws.data_ptr(), n
        self.c = C.PisaCache(num_pages, kv_heads, page, head_dim, self.DTYPES[dtype], C._ptr(self.k), C._ptr(self.v),
                             C._ptr(self.k_exp), C._ptr(self.v_exp))

    def sequences(self, page_table, lens, max_len: int, max_new: int, starts=None, counts=None) -> Sequences:
        """``page_table`` [batch, pages] and ``lens`` [batch] (new tokens included), int32 on the
        cache's device; ``max_len`` and ``max_new`` are upper bounds of the lengths and of a sequence's
        new tokens.  ``starts`` [batch + 1]: the sequences' rows in packed token tensors; else the token
        tensors are padded, with ``counts`` [batch] new tokens each (``max_new`` each if None)."""
        import torch
        batch = lens.shape[0]
        want = [(page_table, "page_table", 2, batch), (lens, "lens", 1, batch), (starts, "starts", 1, batch + 1),
                (counts, "counts", 1, batch)]
        for x, name, dims, n in want:
            if x is not None and (x.dtype != torch.int32 or x.device != self.device or x.dim() != dims or
                                  x.shape[0] != n or not x.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous int32 tensor of {dims} axes and {n} rows on {self.device}")
        if starts is not None and counts is not None:
            raise ValueError("starts (packed) and counts (padded) exclude one another")
        c = C.PisaSequences(batch, page_table.shape[1], _int32("max_len", max_len), _int32("max_new", max_new), C._ptr(page_table), C._ptr(lens),
                            C._ptr(starts), C._ptr(counts))
        return Sequences(c, starts is not None, batch, (page_table, lens, starts, counts))

    def _rows(self, seqs: Sequences, x, heads: int, name: str) -> C.PisaRows:
        """The token tensor's address and strides, after checking what the library cannot see."""
        shape, strides = x.shape, x.stride()
        if len(shape) != (3 if seqs.packed else 4) or (not seqs.packed and shape[0] != seqs.batch):
            raise ValueError(f"{name} must be [tokens, heads, d] (packed) or [batch, heads, rows, d] (padded)")
        if (x.dtype != self.tdtype or x.device != self.device or shape[-1] != self.head_dim or strides[-1] != 1 or
                shape[1] != heads):
            raise ValueError(f"{name} must be a {self.tdtype} tensor on {self.device} with {heads} heads of "
                             f"{self.head_dim} contiguous elements")
        if seqs.packed:
            return C.PisaRows(x.data_ptr(), shape[0], 0, strides[0], strides[1])
        return C.PisaRows(x.data_ptr(), shape[2], strides[0], strides[2], strides[1])

    def _device_index(self) -> int:
        if self.device.type != "cuda":
            raise ValueError(f"the cache is on {self.device}: the kernels take CUDA tensors only")
        return self.device.index

    def _call(self, fn, args, stream):
        """On the cache's device, whatever the current one is."""
        import torch
        index = self._device_index()
        if index == torch.cuda.current_device():
            fn(*args, self._ws_at, self._ws_bytes, C.stream_handle(stream, index))
        else:
            with torch.cuda.device(index):
                fn(*args, self._ws_at, self._ws_bytes, C.stream_handle(stream, index))

    def append(self, seqs: Sequences, k, v, stream=None):
        """Stores the new tokens' k and v (kv_heads heads) in their pages."""
        self._call(C.pisa_cache_append, (self.c, seqs.c, self._rows(seqs, k, self.kv_heads, "k"),
                                         self._rows(seqs, v, self.kv_heads, "v")), stream)

    def read(self, seqs: Sequences, k, v, stream=None):
        """Writes each sequence's last tokens (counts or starts say how many) from the pages into k and v."""
        self._call(C.pisa_cache_read, (self.c, seqs.c, self._rows(seqs, k, self.kv_heads, "k"),
                                       self._rows(seqs, v, self.kv_heads, "v")), stream)

    def attention(self, seqs: Sequences, q, o=None, causal: bool = True, window: int = 0, softmax_scale: float = 1.0,
                  lse=None, stream=None):
        """Attention of the new tokens' q (heads heads) over their sequence's cached tokens, into o.
        ``causal``: no later token is seen; ``window`` > 0: only keys less than that far back (of any size).  ``lse``
        (fp32, [tokens, heads] packed or [batch, heads, rows] padded) takes the log of the softmax sum."""
        if o is None:                    # rows that belong to no token are zero in a tensor made here
            import torch
            with torch.cuda.stream(stream):
                o = torch.zeros_like(q)
        if o.shape != q.shape:
            raise ValueError("o must have q's shape")
        if lse is not None:
            import torch
            shape = q.shape[:-1]
            if lse.dtype != torch.float32 or lse.shape != shape or not lse.is_contiguous() or lse.device != self.device:
                raise ValueError(f"lse must be a contiguous float32 tensor {tuple(shape)} on {self.device}")
        window = max(-1, min(int(window), _INT32_MAX))
        self._call(C.pisa_cache_attention, (self.c, seqs.c, self.heads, bool(causal), window, softmax_scale,
                                            self._rows(seqs, q, self.heads, "q"),
                                            self._rows(seqs, o, self.heads, "o"), lse), stream)
        return o

    def device_error(self, stream=None):
        """(status, code) of the calls so far on ``stream`` (the current one of the cache's device if None); clears it."""
        import torch
        with torch.cuda.device(self._device_index()):
            return C.pisa_read_device_error(self.ws, stream)


AXIS_ORDERS = ("thw", "twh", "htw", "hwt", "wth", "wht")


def reorder_tokens(x, perm, out=None, stream=None):
    """x [B, H, L, d] with its rows gathered through perm ([L], or [B*H, L] per head) on the GPU."""
    import torch
    out = torch.empty_like(x) if out is None else out
    C.pisa_permute_rows(x, out, perm, inverse=False, stream=stream)
    return out


def restore_tokens(x, perm, out=None, stream=None):
    """Inverse of reorder_tokens: rows of x scattered back to their original positions."""
    import torch
    out = torch.empty_like(x) if out is None else out
    C.pisa_permute_rows(x, out, perm, inverse=True, stream=stream)
    return out


def axis_order_permutations(grid, extra_tokens: int = 0, device="cuda"):
    """Device int32 permutations [6, L] for the six axis orders of a (frames, height, width) grid."""
    import torch
    return torch.stack([torch.from_numpy(C.pisa_axis_permutation(grid, o, extra_tokens)) for o in AXIS_ORDERS]).to(device)


def choose_axis_order(pisa: "Pisa", q, k, v, perms):
    """Per head, the axis order whose blocks have the smallest total first-order spread sum_j M_j
    (the method's own covariance measure, from the pre-computation on the reordered tokens).
    Returns (per-head permutation [B*H, L] int32, chosen order index per head).  A calibration
    step: six pre-computations."""
    import torch
    B, H = q.shape[0], q.shape[1]
    scores = []
    for r in range(perms.shape[0]):
        qq, kk, vv = (reorder_tokens(x, perms[r]) for x in (q, k, v))
        pisa.precompute(qq, kk, vv)
        scores.append(pisa.stats.M.reshape(B * H, -1).sum(dim=1))
    best = torch.stack(scores).argmin(dim=0)
    return perms[best].contiguous(), best


class HostPipeline:
    """Steps whose inputs and outputs live in (pinned) host memory, with the copies overlapped:
    the inputs of step i+1 are uploaded and the output of step i-1 is downloaded while step i
    runs.  Two device buffer sets and three streams (upload, compute, download), ordered by
    events; the statistics and routing buffers of `pisa` are reused by consecutive steps on the
    compute stream.  ``submit`` only enqueues; ``synchronize`` waits for everything submitted."""

    def __init__(self, pisa: "Pisa", q_like):
        import torch
        self.p = pisa
        dev = pisa.device
        self.bufs = [[torch.empty(q_like.shape, dtype=q_like.dtype, device=dev) for _ in range(4)] for _ in range(2)]
        self.s_in, self.s_cmp, self.s_out = (torch.cuda.Stream(dev) for _ in range(3))
        self.ev_in = [torch.cuda.Event() for _ in range(2)]
        self.ev_cmp = [torch.cuda.Event() for _ in range(2)]
        self.ev_out = [torch.cuda.Event() for _ in range(2)]
        self.i = 0

    def submit(self, qh, kh, vh, oh):
        import torch
        b = self.i % 2
        q, k, v, o = self.bufs[b]
        with torch.cuda.stream(self.s_in):
            self.s_in.wait_event(self.ev_cmp[b])          # step i-2 has finished reading q, k, v
            q.copy_(qh, non_blocking=True)
            k.copy_(kh, non_blocking=True)
            v.copy_(vh, non_blocking=True)
            self.ev_in[b].record(self.s_in)
        with torch.cuda.stream(self.s_cmp):
            self.s_cmp.wait_event(self.ev_in[b])
            self.s_cmp.wait_event(self.ev_out[b])         # the download of step i-2 has read o
            self.p.precompute(q, k, v, stream=self.s_cmp)
            self.p.route(stream=self.s_cmp)
            self.p.attention(q, k, v, o, stream=self.s_cmp)
            self.ev_cmp[b].record(self.s_cmp)
        with torch.cuda.stream(self.s_out):
            self.s_out.wait_event(self.ev_cmp[b])
            oh.copy_(o, non_blocking=True)
            self.ev_out[b].record(self.s_out)
        self.i += 1

    def synchronize(self):
        for s in (self.s_in, self.s_cmp, self.s_out):
            s.synchronize()
