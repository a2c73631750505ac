"""Python binding of the WildCat C ABI (include/wildcat.h).

Argument marshalling only: every step runs in libwildcat.so's CUDA kernels.
Tensors are torch CUDA tensors (PyTorch supplies device memory and streams);
the functions raise if the library is missing or a call fails.

    from coreset_attention_approximation_b200 import wildcat
    res = wildcat.forward(Q, K, V, r=64, seed=0)        # dict with out, piv, rank, F, Ks, W
"""

from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libwildcat.so")

WC_F32, WC_BF16 = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "CUDA error", 3: "device-side wait timed out",
          4: "unsupported shape", 5: "workspace too small", 6: "non-finite value on the device",
          7: "index outside its buffer (debug build)"}


class WildcatError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)} ({code})")
        self.code = code


class WcShape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32),
        ("n_k", ctypes.c_int32), ("n_q", ctypes.c_int32), ("d", ctypes.c_int32),
        ("dv", ctypes.c_int32), ("r", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("scale", ctypes.c_float), ("eps_stop", ctypes.c_float), ("wait_timeout_ms", ctypes.c_uint32),
        ("seed", ctypes.c_uint64), ("bins", ctypes.c_int32), ("center", ctypes.c_int32),
        ("unit_base", ctypes.c_int32),
    ]


class WcCache(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32),
        ("d", ctypes.c_int32), ("dv", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("page", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("k_page", ctypes.c_int64), ("k_head", ctypes.c_int64), ("k_token", ctypes.c_int64),
        ("v_page", ctypes.c_int64), ("v_head", ctypes.c_int64), ("v_token", ctypes.c_int64),
    ]


class WcRowStrides(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("head", ctypes.c_int64), ("row", ctypes.c_int64)]


EXPORTS = [
    "wc_f_ld", "wc_workspace_bytes", "wc_forward_workspace_bytes", "wc_select", "wc_weights", "wc_attend",
    "wc_forward", "wc_check_device_status", "wc_selftest_wait_timeout", "wc_status_string",
    "wc_attend_noalloc", "wc_selftest_exp2", "wc_read_bandwidth_probe", "wc_cache_workspace_bytes",
    "wc_cache_append", "wc_cache_attend", "wc_cache_evict",
]

_lib = None


def use_debug_library(debug: bool = True) -> None:
    """Switch to the bounds-checked build (libwildcat_debug.so, built by
    `python -m coreset_attention_approximation_b200.build --debug`): its kernels
    check every data-dependent index (pivots, ranks) against its buffer and
    record WC_ERR_BOUNDS instead of making the access.  Takes effect for calls
    made after it."""
    global LIB_PATH, _lib
    LIB_PATH = os.path.join(HERE, "libwildcat_debug.so" if debug else "libwildcat.so")
    _lib = None


def lib():
    """Load libwildcat.so (built by `python -m coreset_attention_approximation_b200.build`)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m coreset_attention_approximation_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        sp = ctypes.POINTER(WcShape)
        L.wc_f_ld.argtypes, L.wc_f_ld.restype = [ctypes.c_int32], ctypes.c_int64
        L.wc_workspace_bytes.argtypes, L.wc_workspace_bytes.restype = [sp], sz
        L.wc_forward_workspace_bytes.argtypes, L.wc_forward_workspace_bytes.restype = [sp], sz
        L.wc_select.argtypes, L.wc_select.restype = [sp, vp, vp, vp, vp, vp, sz, vp], i32
        L.wc_weights.argtypes, L.wc_weights.restype = [sp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32
        L.wc_attend.argtypes, L.wc_attend.restype = [sp, vp, vp, vp, vp, vp, vp, sz, vp], i32
        L.wc_forward.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.wc_forward.restype = i32
        L.wc_check_device_status.argtypes, L.wc_check_device_status.restype = [vp, vp], i32
        L.wc_selftest_wait_timeout.argtypes = [vp, sz, ctypes.c_uint32, vp]
        L.wc_selftest_wait_timeout.restype = i32
        L.wc_status_string.argtypes, L.wc_status_string.restype = [i32], ctypes.c_char_p
        L.wc_attend_noalloc.argtypes, L.wc_attend_noalloc.restype = [sp, vp, vp, vp, vp, vp, vp], i32
        L.wc_selftest_exp2.argtypes = [vp, vp, ctypes.c_int64, ctypes.c_int32, vp]
        L.wc_selftest_exp2.restype = i32
        L.wc_read_bandwidth_probe.argtypes = [vp, ctypes.c_int64, vp, vp]
        L.wc_read_bandwidth_probe.restype = i32
        cp, rp, i64, c32 = ctypes.POINTER(WcCache), ctypes.POINTER(WcRowStrides), ctypes.c_int64, ctypes.c_int32
        L.wc_cache_workspace_bytes.argtypes, L.wc_cache_workspace_bytes.restype = [cp, c32], sz
        L.wc_cache_append.argtypes = [cp, c32, vp, rp, vp, rp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.wc_cache_append.restype = i32
        L.wc_cache_attend.argtypes = [cp, vp, i64, i64, vp, vp, vp, vp, c32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.wc_cache_attend.restype = i32
        L.wc_cache_evict.argtypes = [cp, c32, c32, c32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.wc_cache_evict.restype = i32
        _lib = L
    return _lib


def _check(code: int, what: str):
    if code != 0:
        raise WildcatError(code, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def make_shape(batch, hq, hkv, n_k, n_q, d, dv, r, dtype, scale=0.0, eps_stop=0.0, seed=0,
               wait_timeout_ms=0, bins=1, center=False, unit_base=0) -> WcShape:
    code = {torch.float32: WC_F32, torch.bfloat16: WC_BF16}.get(dtype, dtype)
    return WcShape(batch, hq, hkv, n_k, n_q, d, dv, r, code, scale, eps_stop, wait_timeout_ms, seed,
                   int(bins), int(bool(center)), int(unit_base))


def shape_of(Q, K, V, r, **kw) -> WcShape:
    B, Hkv, n, d = K.shape
    dv = V.shape[-1]
    if Q is None:
        Hq, nq = Hkv, 0
    else:
        Hq, nq = Q.shape[1], Q.shape[2]
    return make_shape(B, Hq, Hkv, n, nq, d, dv, r, K.dtype, **kw)


def f_ld(n_k: int) -> int:
    return int(lib().wc_f_ld(n_k))


def workspace_bytes(shape: WcShape) -> int:
    return int(lib().wc_workspace_bytes(ctypes.byref(shape)))


def forward_workspace_bytes(shape: WcShape) -> int:
    return int(lib().wc_forward_workspace_bytes(ctypes.byref(shape)))


def workspace(shape: WcShape, device, forward_room: bool = False) -> torch.Tensor:
    n = forward_workspace_bytes(shape) if forward_room else workspace_bytes(shape)
    if n == 0:
        raise WildcatError(1, "workspace size")
    # the device status word at offset 0 starts clear
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _outputs(shape: WcShape, device, dtype):
    B, Hkv, r, n = shape.batch, shape.hkv, shape.r, shape.n_k
    nb = max(shape.bins, 1)
    if nb > 1:
        # bins: per-bin ranks and per-bin factors over each bin's keys
        rank = torch.empty(B, Hkv, nb, dtype=torch.int32, device=device)
        F = torch.empty(B, Hkv, nb, r // nb, f_ld(n // nb), dtype=torch.float32, device=device)
    else:
        rank = torch.empty(B, Hkv, dtype=torch.int32, device=device)
        F = torch.empty(B, Hkv, r, f_ld(n), dtype=torch.float32, device=device)
    return dict(
        piv=torch.empty(B, Hkv, r, dtype=torch.int32, device=device),
        rank=rank,
        F=F,
        Ks=torch.empty(B, Hkv, r, shape.d, dtype=dtype, device=device),
        W=torch.empty(B, Hkv, r, shape.dv + 1, dtype=torch.float32, device=device),
    )


def select(K, r, seed=0, *, ws=None, stream=None, **kw):
    shape = shape_of(None, K, K[..., :8], r, seed=seed, **kw)
    o = _outputs(shape, K.device, K.dtype)
    ws = workspace(shape, K.device) if ws is None else ws
    _check(lib().wc_select(ctypes.byref(shape), _ptr(K), _ptr(o["piv"]), _ptr(o["F"]), _ptr(o["rank"]),
                           _ptr(ws), ws.numel(), _stream(stream)), "wc_select")
    return dict(piv=o["piv"], F=o["F"], rank=o["rank"], ws=ws)


def weights(K, V, piv, F, rank, r, *, ws=None, stream=None, **kw):
    shape = shape_of(None, K, V, r, **kw)
    o = _outputs(shape, K.device, K.dtype)
    ws = workspace(shape, K.device) if ws is None else ws
    _check(lib().wc_weights(ctypes.byref(shape), _ptr(K), _ptr(V), _ptr(piv), _ptr(F), _ptr(rank),
                            _ptr(o["Ks"]), _ptr(o["W"]), _ptr(ws), ws.numel(), _stream(stream)), "wc_weights")
    return dict(Ks=o["Ks"], W=o["W"], ws=ws)


def attend(Q, Ks, W, rank, n_k, *, ws=None, stream=None, **kw):
    B, Hq, nq, d = Q.shape
    Hkv, r, dv = Ks.shape[1], Ks.shape[2], W.shape[-1] - 1
    shape = make_shape(B, Hq, Hkv, n_k, nq, d, dv, r, Q.dtype, **kw)
    out = torch.empty(B, Hq, nq, dv, dtype=torch.float32, device=Q.device)
    ws = workspace(shape, Q.device) if ws is None else ws
    _check(lib().wc_attend(ctypes.byref(shape), _ptr(Q), _ptr(Ks), _ptr(W), _ptr(rank), _ptr(out),
                           _ptr(ws), ws.numel(), _stream(stream)), "wc_attend")
    return out


def attend_noalloc(Q, Ks, W, rank, n_k, *, out=None, stream=None, **kw):
    """wc_attend_noalloc: attention with the library's fixed device scratch,
    for callers that cannot allocate.  `out` may be preallocated."""
    B, Hq, nq, d = Q.shape
    Hkv, r, dv = Ks.shape[1], Ks.shape[2], W.shape[-1] - 1
    shape = make_shape(B, Hq, Hkv, n_k, nq, d, dv, r, Q.dtype, **kw)
    if out is None:
        out = torch.empty(B, Hq, nq, dv, dtype=torch.float32, device=Q.device)
    _check(lib().wc_attend_noalloc(ctypes.byref(shape), _ptr(Q), _ptr(Ks), _ptr(W), _ptr(rank), _ptr(out),
                                   _stream(stream)), "wc_attend_noalloc")
    return out


def forward(Q, K, V, r, seed=0, *, ws=None, stream=None, outputs=None, **kw):
    """Whole path on the GPU: select -> weights -> attend.

    Q [B,Hq,nq,d], K [B,Hkv,n,d], V [B,Hkv,n,dv] CUDA tensors (bf16 or fp32,
    contiguous).  `outputs` may hold preallocated tensors (out, piv, rank, F,
    Ks, W); missing ones are allocated.  Returns the dict of all of them.
    """
    shape = shape_of(Q, K, V, r, seed=seed, **kw)
    o = dict(outputs or {})
    if any(k not in o for k in ("piv", "rank", "F", "Ks", "W")):
        for k, v in _outputs(shape, K.device, K.dtype).items():
            o.setdefault(k, v)
    o.setdefault("out", torch.empty(Q.shape[0], Q.shape[1], Q.shape[2], shape.dv, dtype=torch.float32,
                                    device=K.device))
    ws = workspace(shape, K.device) if ws is None else ws
    _check(lib().wc_forward(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V), _ptr(o["out"]), _ptr(o["piv"]),
                            _ptr(o["rank"]), _ptr(o["F"]), _ptr(o["Ks"]), _ptr(o["W"]), _ptr(ws), ws.numel(),
                            _stream(stream)), "wc_forward")
    o["ws"] = ws
    return o


class ForwardGraph:
    """wc_forward captured once into a CUDA graph, then replayed: repeated
    forward passes over the same device buffers cost one graph launch instead
    of the path's kernel launches and memsets.  Refill Q, K, V in place (for
    example with copy_) before each `replay()`; the outputs (out, piv, rank, F,
    Ks, W) are overwritten in place and returned."""

    def __init__(self, Q, K, V, r, seed=0, *, ws=None, outputs=None, **kw):
        self.Q, self.K, self.V = Q, K, V
        self.shape = shape_of(Q, K, V, r, seed=seed, **kw)
        self.ws = workspace(self.shape, K.device) if ws is None else ws
        o = dict(outputs or {})
        if any(k not in o for k in ("piv", "rank", "F", "Ks", "W")):
            for k, v in _outputs(self.shape, K.device, K.dtype).items():
                o.setdefault(k, v)
        o.setdefault("out", torch.empty(Q.shape[0], Q.shape[1], Q.shape[2], self.shape.dv, dtype=torch.float32,
                                        device=K.device))
        self.outputs = o
        # one eager pass first: function attributes and tensor maps are set up outside the capture
        self._launch(torch.cuda.current_stream(K.device))
        torch.cuda.current_stream(K.device).synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self._launch(torch.cuda.current_stream(K.device))

    def _launch(self, stream):
        o = self.outputs
        _check(lib().wc_forward(ctypes.byref(self.shape), _ptr(self.Q), _ptr(self.K), _ptr(self.V), _ptr(o["out"]),
                                _ptr(o["piv"]), _ptr(o["rank"]), _ptr(o["F"]), _ptr(o["Ks"]), _ptr(o["W"]),
                                _ptr(self.ws), self.ws.numel(), _stream(stream)), "wc_forward")

    def replay(self):
        self.graph.replay()
        return self.outputs


class HostPipeline:
    """Forward passes over a sequence of host batches, with the copies
    overlapped: batch i+1's host-to-device copy and batch i-1's device-to-host
    copy run on their own streams while batch i computes.  Two device copies
    of Q, K, V and out alternate; the factor, weights and workspace are shared
    (the passes themselves run one after another on the compute stream).

    Host tensors must be pinned for the copies to overlap.  Every batch has
    the shapes and dtype of the (Q, K, V) given here."""

    def __init__(self, Q, K, V, r, seed=0, *, device="cuda", stream=None, ws=None, outputs=None, **kw):
        """Q, K, V: host tensors of the batches' shapes and dtype (only their
        shapes are read).  ws / outputs: optional workspace and (piv, rank, F,
        Ks, W) device tensors to reuse; the last batch's stay there."""
        self.device = torch.device(device)
        self.r, self.seed, self.kw = r, seed, kw
        self.shape = shape_of(Q, K, V, r, seed=seed, **kw)
        self.ws = workspace(self.shape, self.device) if ws is None else ws
        self.shared = {k: v for k, v in (outputs or {}).items() if k != "out"}
        if any(k not in self.shared for k in ("piv", "rank", "F", "Ks", "W")):
            for k, v in _outputs(self.shape, self.device, K.dtype).items():
                self.shared.setdefault(k, v)
        out_shape = (Q.shape[0], Q.shape[1], Q.shape[2], self.shape.dv)
        self.bufs = [dict(Q=torch.empty(Q.shape, dtype=Q.dtype, device=self.device),
                          K=torch.empty(K.shape, dtype=K.dtype, device=self.device),
                          V=torch.empty(V.shape, dtype=V.dtype, device=self.device),
                          out=torch.empty(out_shape, dtype=torch.float32, device=self.device)) for _ in range(2)]
        self.compute = stream or torch.cuda.current_stream(self.device)
        self.h2d = torch.cuda.Stream(self.device)
        self.d2h = torch.cuda.Stream(self.device)
        self.loaded = [torch.cuda.Event() for _ in range(2)]
        self.computed = [torch.cuda.Event() for _ in range(2)]
        self.drained = [torch.cuda.Event() for _ in range(2)]
        self.started = [False, False]

    def run(self, batches):
        """batches: iterable of (Q, K, V, out) host tensors; out [B, Hq, nq, dv]
        fp32 receives the batch's output.  The copies and passes are queued
        behind whatever the compute stream already holds; returns once the
        last output has been queued (call `wait()` before reading it)."""
        for i, (Qh, Kh, Vh, oh) in enumerate(batches):
            j = i % 2
            b = self.bufs[j]
            with torch.cuda.stream(self.h2d):
                if i == 0:
                    self.h2d.wait_stream(self.compute)            # after whatever the caller queued
                if self.started[j]:
                    self.h2d.wait_event(self.computed[j])     # batch i-2 has finished reading buffer j
                b["Q"].copy_(Qh, non_blocking=True)
                b["K"].copy_(Kh, non_blocking=True)
                b["V"].copy_(Vh, non_blocking=True)
                self.loaded[j].record(self.h2d)
            self.compute.wait_event(self.loaded[j])
            if self.started[j]:
                self.compute.wait_event(self.drained[j])       # batch i-2's output has left buffer j
            forward(b["Q"], b["K"], b["V"], self.r, self.seed, ws=self.ws, stream=self.compute,
                    outputs=dict(self.shared, out=b["out"]), **self.kw)
            self.computed[j].record(self.compute)
            with torch.cuda.stream(self.d2h):
                self.d2h.wait_event(self.computed[j])
                oh.copy_(b["out"], non_blocking=True)
                self.drained[j].record(self.d2h)
            self.started[j] = True
        # the compute stream ends after the last copy out
        self.compute.wait_stream(self.d2h)

    def wait(self):
        self.compute.synchronize()
        return check_device_status(self.ws, self.compute)


def _strides(t):
    """Strides of a 4-axis tensor's first three axes, 0 where the axis has one entry."""
    (a, b, c, _), (x, y, z, _) = t.shape, t.stride()
    return x if a > 1 else 0, y if b > 1 else 0, z if c > 1 else 0


class PagedCache:
    """Exact keys and values in pages, beside (or instead of) a coreset: rows
    appended as tokens are generated, attention of one new token per sequence
    over them, eviction by accumulated attention weight.

    k_pages [n_pages, Hkv, page, d] and v_pages [n_pages, Hkv, page, dv] are
    CUDA tensors (bf16 or fp32) with contiguous rows; a pool kept in the order
    [n_pages, page, Hkv, d] is passed as its transpose(1, 2).  table
    [B, max_pages] int32 (contiguous): token t of sequence b is in slot
    t % page of page table[b, t // page].  hq: query heads.  scores
    [B, Hkv, max_pages * page] fp32 (contiguous): accumulated attention
    weights, needed to accumulate and to evict; a cache with scores keeps
    4 B hq max_pages page bytes of workspace for a step's logits as well.

    Lengths, positions and counts are int32 CUDA tensors that the caller keeps
    and advances, so a captured graph serves a growing cache.  The tensors
    given here are kept by reference and changed in place.  Lengths and page
    numbers are checked on the device (`check()` reports).  To use other
    tensors, make another PagedCache.  The cache's calls
    share one workspace: calls that may overlap on the GPU (two streams, two
    graphs replayed at once) need a PagedCache each.

        cache = wildcat.PagedCache(k_pages, v_pages, table, hq=32, scores=scores)
        cache.append(K, V, lens); lens += 1                   # K, V [B, Hkv, 1, d]
        out = cache.attend(Q, lens, accumulate=True)          # Q [B, Hq, d]
        lens = cache.evict(lens, keep=1024, sink=4, recent=64)["lens"]
        out = cache.attend(Q, lens, coreset=(Ks, W, rank))    # a compressed prompt and the exact tail
    """

    def __init__(self, k_pages, v_pages, table, hq, *, scores=None, scale=0.0):
        if k_pages.dim() != 4 or v_pages.dim() != 4 or table.dim() != 2:
            raise WildcatError(1, "PagedCache: k_pages and v_pages have 4 axes, table 2")
        self.device = k_pages.device
        n_pages, hkv, page, d = k_pages.shape
        self.dtype = k_pages.dtype
        if self.dtype not in (torch.float32, torch.bfloat16) or v_pages.dtype != self.dtype:
            raise WildcatError(1, "PagedCache: k_pages and v_pages are both bf16 or both fp32")
        if tuple(v_pages.shape[:3]) != (n_pages, hkv, page):
            raise WildcatError(1, "PagedCache: v_pages differs from k_pages in more than its width")
        if k_pages.stride(3) != 1 or v_pages.stride(3) != 1:
            raise WildcatError(1, "PagedCache: rows of k_pages and v_pages are contiguous")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.batch, self.max_pages = table.shape
        self.hkv, self.d, self.dv, self.hq = hkv, d, v_pages.shape[3], int(hq)
        self.cap = self.max_pages * page
        self._on_device(v_pages, "v_pages")
        self.table = self._tensor(table, "table", (self.batch, self.max_pages), torch.int32)
        self.scores = None if scores is None else self._scores(scores, "scores")
        self.shape = WcCache(self.batch, self.hq, hkv, d, self.dv,
                             WC_BF16 if self.dtype == torch.bfloat16 else WC_F32, page, n_pages, self.max_pages,
                             scale, *_strides(k_pages), *_strides(v_pages))
        n = int(lib().wc_cache_workspace_bytes(ctypes.byref(self.shape), int(scores is not None)))
        if n == 0:
            raise WildcatError(1, "PagedCache: sizes or strides")
        if self.device.type != "cuda":
            raise WildcatError(1, "PagedCache: the pages are on a GPU")
        self.ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        self.ws[: 256 + 8 * n_pages].zero_()     # the status word and the page counts; the rest is written first
        # No caller sees the workspace, so none can order its first use on another stream behind these zeros (and
        # behind whatever used this memory before): they are waited for here, once.  A capture orders its own work.
        with torch.cuda.device(self.device):
            made_on = torch.cuda.current_stream()
            if not torch.cuda.is_current_stream_capturing():
                made_on.synchronize()
        self._streams = {made_on.cuda_stream}    # that the allocator knows to use the workspace
        # what every call passes on, looked up once (a decode step's kernels are as short as the calls that launch them)
        self._shape_ref = ctypes.byref(self.shape)
        self._pools = (k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr())
        self._p_scores = None if scores is None else scores.data_ptr()
        self._room = (self.ws.data_ptr(), n)
        self._q_shape, self._o_shape = (self.batch, self.hq, self.d), (self.batch, self.hq, self.dv)
        self._seqs, self._index = (self.batch,), self.device.index
        self._k_row, self._v_row = WcRowStrides(hkv * d, d, d), WcRowStrides(hkv * self.dv, self.dv, self.dv)
        self._kept = (self.k_pages, self.v_pages, self.table, self.scores, self.ws)
        L = lib()
        self._append, self._attend, self._evict = L.wc_cache_append, L.wc_cache_attend, L.wc_cache_evict

    # ---- arguments

    def _on_device(self, t, name):
        if t.device != self.device:
            raise WildcatError(1, f"PagedCache: {name} is on {t.device}, the pages on {self.device}")

    def _tensor(self, t, name, shape, dtype):
        if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
            raise WildcatError(1, f"PagedCache: {name} is a contiguous {dtype} tensor of shape {tuple(shape)}, got "
                                  f"{t.dtype} {tuple(t.shape)}")
        self._on_device(t, name)
        return t

    def _scores(self, t, name):
        return self._tensor(t, name, (self.batch, self.hkv, self.cap), torch.float32)

    def _rows(self, t, name, shape):
        """A strided tensor of rows in the pages' type."""
        if t.shape != shape or t.dtype != self.dtype:
            raise WildcatError(1, f"PagedCache: {name} is a {self.dtype} tensor of shape {tuple(shape)}, got "
                                  f"{t.dtype} {tuple(t.shape)}")
        if t.stride(-1) != 1:
            raise WildcatError(1, f"PagedCache: rows of {name} are contiguous")
        self._on_device(t, name)
        return t

    def _launch(self, call, what, stream, args, tensors):
        """call(*args, stream) on the given stream, or the device's current
        one, with the pages' device current.  The caching allocator is told of
        the tensors' use on a given stream, and of the workspace's on any."""
        handle = torch._C._cuda_getCurrentRawStream(self._index)
        # (the default streams of all devices have one handle, so it alone does not tell whose a stream is)
        if stream is not None and stream.device != self.device:
            raise WildcatError(1, f"{what}: the stream is another device's")
        if stream is not None and stream.cuda_stream != handle:
            for t in tensors + self._kept:
                if t is not None:
                    t.record_stream(stream)
            handle = stream.cuda_stream
        if handle not in self._streams:          # the workspace outlives the cache until their work is done
            self.ws.record_stream(stream or torch.cuda.current_stream(self.device))
            self._streams.add(handle)
        if torch.cuda.current_device() == self._index:
            code = call(*args, handle)
        else:
            with torch.cuda.device(self.device):
                code = call(*args, handle)
        if code != 0:
            raise WildcatError(code, what)

    def _empty(self, shape, strides, dtype, stream):
        """An output, allocated for the stream that writes it (the strides are
        those of a contiguous tensor; given, they spare a microsecond)."""
        if stream is None:
            return torch.empty_strided(shape, strides, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty_strided(shape, strides, dtype=dtype, device=self.device)

    # ---- calls

    def append(self, K, V, pos, count=None, *, stream=None):
        """Writes row j < count[b] (count None: every row) of K [B, Hkv, t, d]
        and V [B, Hkv, t, dv] to position pos[b] + j of sequence b; the scores
        there become 0.  pos, count: int32 [B].  K and V may be strided in
        steps of 16 bytes.  Rows beyond the cache's end are not written and
        reported by `check()`.  Two rows sent to one place (a page that two
        sequences name) leave pieces of both there."""
        t = K.shape[2] if K.dim() == 4 else -1
        self._rows(K, "K", (self.batch, self.hkv, t, self.d))
        self._rows(V, "V", (self.batch, self.hkv, t, self.dv))
        self._tensor(pos, "pos", self._seqs, torch.int32)
        if count is not None:
            self._tensor(count, "count", self._seqs, torch.int32)
        if t == 1 and K.is_contiguous() and V.is_contiguous():     # a decode step's rows
            ks, vs = self._k_row, self._v_row
        else:
            ks, vs = WcRowStrides(*_strides(K)), WcRowStrides(*_strides(V))
        self._launch(self._append, "wc_cache_append", stream,
                     (self._shape_ref, t, K.data_ptr(), ks, V.data_ptr(), vs, pos.data_ptr(),
                      None if count is None else count.data_ptr(), *self._pools, self._p_scores, *self._room),
                     (K, V, pos, count))

    def attend(self, Q, lens, *, coreset=None, accumulate=False, return_lse=False, out=None, stream=None):
        """Attention of one new token per sequence: Q [B, Hq, d] over the first
        lens[b] tokens of sequence b, and over coreset = (Ks, W, rank) beside
        them (as `weights` and `select` return them, with bins or without;
        rank None: all r rows).
        Returns out [B, Hq, dv] fp32, or (out, lse [B, Hq]).  accumulate: adds
        each key's attention weight, summed over its queries, to `scores`."""
        self._rows(Q, "Q", self._q_shape)
        self._tensor(lens, "lens", self._seqs, torch.int32)
        if accumulate and self.scores is None:
            raise WildcatError(1, "PagedCache.attend: accumulate needs scores")
        Ks = W = rank = None
        r = 0
        if coreset is not None:
            Ks, W, rank = coreset
            r = Ks.shape[2] if Ks.dim() == 4 else -1
            self._tensor(Ks, "Ks", (self.batch, self.hkv, r, self.d), self.dtype)
            self._tensor(W, "W", (self.batch, self.hkv, r, self.dv + 1), torch.float32)
            if rank is not None and rank.dim() == 3:     # of a binned selection: [B, Hkv, bins]
                bins = rank.shape[2]
                self._tensor(rank, "rank", (self.batch, self.hkv, bins), torch.int32)
                if bins < 1 or r % bins:
                    raise WildcatError(1, f"PagedCache.attend: {r} coreset rows in {bins} bins")
                rank = None      # every bin's rows count; those beyond its rank have weight 0 in W
            elif rank is not None:
                self._tensor(rank, "rank", (self.batch, self.hkv), torch.int32)
        if out is None:
            out = self._empty(self._o_shape, (self.hq * self.dv, self.dv, 1), torch.float32, stream)
        else:
            self._tensor(out, "out", self._o_shape, torch.float32)
        lse = self._empty((self.batch, self.hq), (self.hq, 1), torch.float32, stream) if return_lse else None
        sq = Q.stride()
        self._launch(self._attend, "wc_cache_attend", stream,
                     (self._shape_ref, Q.data_ptr(), sq[0], sq[1], *self._pools, lens.data_ptr(), r,
                      None if r == 0 else Ks.data_ptr(), None if r == 0 else W.data_ptr(),
                      None if rank is None else rank.data_ptr(), out.data_ptr(),
                      None if lse is None else lse.data_ptr(), self._p_scores if accumulate else None, *self._room),
                     (Q, lens, Ks, W, rank, out, lse))
        return (out, lse) if return_lse else out

    def evict(self, lens, keep, *, sink=0, recent=0, into=None, scores_into=None, lens_out=None, stream=None):
        """Shortens every sequence to at most `keep` tokens, each kv head by
        itself: the first `sink`, the last `recent` and those of the largest
        scores in between (ties: the lower position).  The kept rows move, in
        order, to the front of the sequence's pages, or to the pages of `into`
        (a table like `table`, which is not changed; needed where pages are
        shared), their scores to the front of `scores`, or of `scores_into`.
        Returns idx [B, Hkv, keep] (kept positions, -1 beyond) and lens [B]
        (lens_out may be lens itself).  A sequence that cannot be moved (a page
        outside the pool, a page to be written that is named twice) stays as it
        is; `check()` reports it."""
        self._tensor(lens, "lens", self._seqs, torch.int32)
        if self.scores is None:
            raise WildcatError(1, "PagedCache.evict: needs scores")
        if into is not None:
            self._tensor(into, "into", (self.batch, self.max_pages), torch.int32)
        if scores_into is not None:
            self._scores(scores_into, "scores_into")
        keep, sink, recent = int(keep), int(sink), int(recent)
        if not (1 <= keep <= self.cap and sink >= 0 and recent >= 0 and sink + recent <= keep):
            raise WildcatError(1, "PagedCache.evict: 1 <= keep <= capacity, sink + recent <= keep")
        idx = self._empty((self.batch, self.hkv, keep), (self.hkv * keep, keep, 1), torch.int32, stream)
        if lens_out is None:
            lens_out = self._empty(self._seqs, (1,), torch.int32, stream)
        else:
            self._tensor(lens_out, "lens_out", self._seqs, torch.int32)
        self._launch(self._evict, "wc_cache_evict", stream,
                     (self._shape_ref, keep, sink, recent, *self._pools, None if into is None else into.data_ptr(),
                      lens.data_ptr(), self._p_scores, None if scores_into is None else scores_into.data_ptr(),
                      idx.data_ptr(), lens_out.data_ptr(), *self._room), (lens, into, scores_into, idx, lens_out))
        return dict(idx=idx, lens=lens_out)

    def check(self, stream=None) -> int:
        """The first error the cache's kernels recorded since the last check
        (0: none), after waiting for the stream; clears it."""
        with torch.cuda.device(self.device):
            return check_device_status(self.ws, stream)


def check_device_status(ws, stream=None) -> int:
    return int(lib().wc_check_device_status(_ptr(ws), _stream(stream)))


def selftest_wait_timeout(ws, timeout_ms, stream=None) -> int:
    return int(lib().wc_selftest_wait_timeout(_ptr(ws), ws.numel(), timeout_ms, _stream(stream)))


def read_probe(buf, sink, stream=None):
    """Reads the CUDA tensor `buf` once as a read-only stream (the read
    bandwidth probe); `sink` (one int32 on the device) receives the XOR of its
    32-bit words."""
    _check(lib().wc_read_bandwidth_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), _stream(stream)),
           "wc_read_bandwidth_probe")


def selftest_exp2(x, method=0, stream=None):
    """2^x for an fp32 CUDA tensor as the tensor-core kernels compute it:
    method 0 on the FMA / ALU pipes (the polynomial), 1 on the exponential unit."""
    y = torch.empty_like(x)
    _check(lib().wc_selftest_exp2(_ptr(x), _ptr(y), x.numel(), method, _stream(stream)), "wc_selftest_exp2")
    return y
