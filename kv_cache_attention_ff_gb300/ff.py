"""ctypes binding of libff.so (argument marshalling only).

Every step of the renderer bank-attention path runs in the library's CUDA
kernels; this module only converts torch tensors and streams to pointers and
status codes to exceptions.  If the library is missing it raises: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libff.so")

FF_OK = 0
STATUS = {
    0: "FF_OK", 1: "FF_ERR_ARG", 2: "FF_ERR_ORDER", 3: "FF_ERR_ANCHOR_MISSING", 4: "FF_ERR_OOM",
    5: "FF_ERR_CUDA", 6: "FF_ERR_DEVICE_TIMEOUT", 7: "FF_ERR_UNSUPPORTED", 8: "FF_ERR_CAPACITY",
}

# Every entry point declared in include/ff.h.
EXPORTS = [
    "ff_desc_default", "ff_bank_create", "ff_anchor_publish", "ff_render_attn", "ff_bank_destroy",
    "ff_bank_gamma", "ff_bank_slot_info", "ff_bank_bytes", "ff_bank_error_poll", "ff_status_string",
    "ff_plan_chunk", "ff_bank_set_timing", "ff_bank_read_timing", "ff_render_kernel_count",
    "ff_attention_noalloc", "ff_bank_wait_probe", "ff_planner_attn", "ff_plan_planner_block",
    "ff_packed_workspace_bytes", "ff_packed_render_attn", "ff_render_attn_batch",
    "ff_kv8_desc_default", "ff_kv8_create", "ff_kv8_destroy", "ff_kv8_bytes", "ff_kv8_layer_info",
    "ff_kv8_append", "ff_kv8_load", "ff_kv8_attn", "ff_kv8_evict", "ff_kv8_error_poll",
    "ff_paged_desc_default", "ff_paged_create", "ff_paged_destroy", "ff_paged_bytes", "ff_paged_info",
    "ff_paged_layer_info", "ff_paged_plan", "ff_paged_store", "ff_paged_attn", "ff_paged_error_poll",
]


class FFError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        self.code = STATUS.get(status, str(status))
        super().__init__(f"{what}: {self.code} ({_lib().ff_status_string(status).decode()})")


class BankDesc(ctypes.Structure):
    _fields_ = [
        ("n_layers", ctypes.c_int), ("n_stages", ctypes.c_int), ("history", ctypes.c_int),
        ("chunk_frames", ctypes.c_int), ("anchor_stride", ctypes.c_int), ("anchor_capacity", ctypes.c_int),
        ("total_frames", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("frame_h", ctypes.c_int), ("frame_w", ctypes.c_int), ("rope_theta", ctypes.c_double),
        ("max_bytes", ctypes.c_size_t), ("device", ctypes.c_int), ("planner_block", ctypes.c_int),
        ("planner_history", ctypes.c_int),
    ]


class ChunkPlan(ctypes.Structure):
    _fields_ = [
        ("first_frame", ctypes.c_int), ("n_frames", ctypes.c_int), ("n_anchors", ctypes.c_int),
        ("anchors", ctypes.c_int * 2), ("n_hist", ctypes.c_int), ("hist_first", ctypes.c_int),
        ("hist_frames", ctypes.c_int), ("slot", ctypes.c_int), ("key_frames", ctypes.c_int),
    ]


class PlannerPlan(ctypes.Structure):
    _fields_ = [
        ("first_anchor", ctypes.c_int), ("n_anchors", ctypes.c_int), ("hist_first_block", ctypes.c_int),
        ("n_hist_blocks", ctypes.c_int), ("hist_frames", ctypes.c_int), ("key_frames", ctypes.c_int),
    ]


class KernelTimes(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_int), ("publish_ms", ctypes.c_double), ("attn_ms", ctypes.c_double),
                ("combine_ms", ctypes.c_double), ("launches", ctypes.c_int)]


class KV8Desc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("batch", ctypes.c_int), ("capacity", ctypes.c_int),
                ("heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("max_tokens", ctypes.c_int), ("device", ctypes.c_int), ("max_bytes", ctypes.c_size_t)]


class PagedDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("pages", ctypes.c_int), ("page_rows", ctypes.c_int),
                ("requests", ctypes.c_int), ("capacity", ctypes.c_int), ("heads", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("max_rows", ctypes.c_int),
                ("device", ctypes.c_int), ("max_bytes", ctypes.c_size_t)]


class RenderCall(ctypes.Structure):
    _fields_ = [("layer", ctypes.c_int), ("stage", ctypes.c_int), ("chunk", ctypes.c_int),
                ("q_pre", ctypes.c_void_p), ("k_pre", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("out", ctypes.c_void_p)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libff.so not built ({LIB_PATH}); run kv_cache_attention_ff_gb300.build.build()")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, V = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
        lib.ff_desc_default.argtypes = [ctypes.POINTER(BankDesc)]
        lib.ff_bank_create.argtypes = [ctypes.POINTER(BankDesc), ctypes.POINTER(P)]
        lib.ff_anchor_publish.argtypes = [P, I, I, I, V, V, V]
        lib.ff_render_attn.argtypes = [P, I, I, I, V, V, V, V, V]
        lib.ff_bank_destroy.argtypes = [P]
        lib.ff_bank_gamma.argtypes = [P, I, ctypes.POINTER(I), ctypes.POINTER(I), ctypes.POINTER(I)]
        lib.ff_bank_slot_info.argtypes = [P, I, I, I, ctypes.POINTER(I), ctypes.POINTER(I), ctypes.POINTER(P),
                                          ctypes.POINTER(P)]
        lib.ff_bank_bytes.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        lib.ff_bank_error_poll.argtypes = [P]
        lib.ff_status_string.argtypes = [I]
        lib.ff_status_string.restype = ctypes.c_char_p
        lib.ff_plan_chunk.argtypes = [ctypes.POINTER(BankDesc), I, ctypes.POINTER(ChunkPlan)]
        lib.ff_bank_set_timing.argtypes = [P, I]
        lib.ff_bank_read_timing.argtypes = [P, ctypes.POINTER(KernelTimes)]
        lib.ff_render_kernel_count.argtypes = [P, I, ctypes.POINTER(I)]
        lib.ff_attention_noalloc.argtypes = [V, V, V, V, I, I, I, I, V]
        lib.ff_bank_wait_probe.argtypes = [P, I, V]
        lib.ff_planner_attn.argtypes = [P, I, I, V, V, V, V, V]
        lib.ff_packed_workspace_bytes.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        lib.ff_packed_render_attn.argtypes = [P, V, V, V, V, V, V, V, ctypes.c_size_t, V]
        lib.ff_plan_planner_block.argtypes = [ctypes.POINTER(BankDesc), I, ctypes.POINTER(PlannerPlan)]
        lib.ff_render_attn_batch.argtypes = [P, I, ctypes.POINTER(RenderCall), V]
        lib.ff_kv8_desc_default.argtypes = [ctypes.POINTER(KV8Desc)]
        lib.ff_kv8_create.argtypes = [ctypes.POINTER(KV8Desc), ctypes.POINTER(P)]
        lib.ff_kv8_destroy.argtypes = [P]
        lib.ff_kv8_bytes.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        lib.ff_kv8_layer_info.argtypes = [P, I] + [ctypes.POINTER(P)] * 5
        lib.ff_kv8_append.argtypes = [P, I, I, V, V, V, V, V]
        lib.ff_kv8_load.argtypes = [P, I, I, V, V, V, V]
        lib.ff_kv8_attn.argtypes = [P, I, I, V, V, I, V, V, V, V, V]
        lib.ff_kv8_evict.argtypes = [P, I, P, I, I, I, V, V, V, V]
        lib.ff_kv8_error_poll.argtypes = [P]
        lib.ff_paged_desc_default.argtypes = [ctypes.POINTER(PagedDesc)]
        lib.ff_paged_create.argtypes = [ctypes.POINTER(PagedDesc), ctypes.POINTER(P)]
        lib.ff_paged_destroy.argtypes = [P]
        lib.ff_paged_bytes.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        lib.ff_paged_info.argtypes = [P] + [ctypes.POINTER(P)] * 7
        lib.ff_paged_layer_info.argtypes = [P, I, ctypes.POINTER(P), ctypes.POINTER(P)]
        lib.ff_paged_plan.argtypes = [P, I, V, V, V]
        lib.ff_paged_store.argtypes = [P, I, I, V, V, V]
        lib.ff_paged_attn.argtypes = [P, I, I, I, V, V, V, V]
        lib.ff_paged_error_poll.argtypes = [P]
        for name in EXPORTS:
            if name != "ff_status_string":
                getattr(lib, name).restype = ctypes.c_int
        _LIB = lib
    return _LIB


def lib():
    """The loaded ctypes library (raises ImportError if it was not built)."""
    return _lib()


def _check(status: int, what: str) -> None:
    if status != FF_OK:
        raise FFError(status, what)


def make_desc(**kw) -> BankDesc:
    d = BankDesc()
    _check(_lib().ff_desc_default(ctypes.byref(d)), "ff_desc_default")
    for k, v in kw.items():
        if not hasattr(d, k):
            raise TypeError(f"unknown bank field {k}")
        setattr(d, k, v)
    return d


def plan_chunk(desc: BankDesc, chunk: int) -> ChunkPlan:
    p = ChunkPlan()
    _check(_lib().ff_plan_chunk(ctypes.byref(desc), chunk, ctypes.byref(p)), "ff_plan_chunk")
    return p


def plan_planner_block(desc: BankDesc, block: int) -> PlannerPlan:
    p = PlannerPlan()
    _check(_lib().ff_plan_planner_block(ctypes.byref(desc), block, ctypes.byref(p)), "ff_plan_planner_block")
    return p


def attention_noalloc(q, k, v, out, stream=None):
    """Attention over a caller-held context without any device allocation
    (see ff_attention_noalloc in include/ff.h).  All four tensors must be on
    one device; the call runs with that device current."""
    import torch
    nq, heads, d = q.shape
    nk = k.shape[0]
    if any(t.device != q.device for t in (k, v, out)):
        raise ValueError("q, k, v and out must be on one device")
    if stream is not None and stream.device != q.device:
        raise ValueError("stream belongs to another device than the tensors")
    with torch.cuda.device(q.device):
        _check(_lib().ff_attention_noalloc(_ptr(q, (nq, heads, d), "q"), _ptr(k, (nk, heads, d), "k"),
                                           _ptr(v, (nk, heads, d), "v"), _ptr(out, (nq, heads, d), "out"),
                                           nq, nk, heads, d, _stream(stream, q.device)), "ff_attention_noalloc")


class _DevView:
    """__cuda_array_interface__ wrapper so torch can view bank memory without a copy."""

    def __init__(self, ptr: int, shape, device: int, typestr: str = "<u2", owner=None):
        self.owner = owner  # whoever frees the memory lives as long as the view
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr, "data": (ptr, False),
                                         "version": 3, "strides": None}


def _ptr(t, shape, name):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous bf16 CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


class Bank:
    """Owner of one libff bank (stage banks, anchor ring and scratch of all layers)."""

    def __init__(self, **kw):
        self.desc = make_desc(**kw)
        self.handle = ctypes.c_void_p()
        _check(_lib().ff_bank_create(ctypes.byref(self.desc), ctypes.byref(self.handle)), "ff_bank_create")
        d = self.desc
        self.T = d.frame_h * d.frame_w
        self.device = d.device

    # -- core calls ---------------------------------------------------------
    def anchor_publish(self, layer, first_anchor_frame, n_anchors, k_pre, v, stream=None):
        shape = (n_anchors * self.T, self.desc.heads, self.desc.head_dim)
        _check(_lib().ff_anchor_publish(self.handle, layer, first_anchor_frame, n_anchors, _ptr(k_pre, shape, "k_pre"),
                                        _ptr(v, shape, "v"), _stream(stream, self.device)), "ff_anchor_publish")

    def render_attn(self, layer, stage, chunk, q_pre, k_pre, v, out, stream=None):
        frames = plan_chunk(self.desc, chunk).n_frames if 0 <= chunk < self.n_chunks else self.desc.chunk_frames
        shape = (frames * self.T, self.desc.heads, self.desc.head_dim)
        _check(_lib().ff_render_attn(self.handle, layer, stage, chunk, _ptr(q_pre, shape, "q_pre"),
                                     _ptr(k_pre, shape, "k_pre"), _ptr(v, shape, "v"), _ptr(out, shape, "out"),
                                     _stream(stream, self.device)), "ff_render_attn")

    def render_attn_batch(self, calls, stream=None):
        """Independent renderer calls, one per stage, issued together.
        `calls`: sequence of (layer, stage, chunk, q_pre, k_pre, v, out)."""
        arr = (RenderCall * len(calls))()
        for j, (layer, stage, chunk, q_pre, k_pre, v, out) in enumerate(calls):
            frames = plan_chunk(self.desc, chunk).n_frames if 0 <= chunk < self.n_chunks else self.desc.chunk_frames
            shape = (frames * self.T, self.desc.heads, self.desc.head_dim)
            arr[j] = RenderCall(layer, stage, chunk, _ptr(q_pre, shape, "q_pre"), _ptr(k_pre, shape, "k_pre"),
                                _ptr(v, shape, "v"), _ptr(out, shape, "out"))
        _check(_lib().ff_render_attn_batch(self.handle, len(calls), arr, _stream(stream, self.device)),
               "ff_render_attn_batch")

    def render_attn_batch_raw(self, calls, stream_handle) -> int:
        """Pointer-level batch: `calls` of (layer, stage, chunk, q_ptr, k_ptr, v_ptr, out_ptr); returns the status."""
        arr = (RenderCall * len(calls))(*[RenderCall(*c) for c in calls])
        return _lib().ff_render_attn_batch(self.handle, len(calls), arr, ctypes.c_void_p(stream_handle))

    def planner_attn(self, layer, block, q_pre, k_pre, v, out, stream=None):
        n = plan_planner_block(self.desc, block).n_anchors
        shape = (n * self.T, self.desc.heads, self.desc.head_dim)
        _check(_lib().ff_planner_attn(self.handle, layer, block, _ptr(q_pre, shape, "q_pre"), _ptr(k_pre, shape, "k_pre"),
                                      _ptr(v, shape, "v"), _ptr(out, shape, "out"), _stream(stream, self.device)),
               "ff_planner_attn")

    def packed_workspace_bytes(self) -> int:
        n = ctypes.c_size_t()
        _check(_lib().ff_packed_workspace_bytes(self.handle, ctypes.byref(n)), "ff_packed_workspace_bytes")
        return n.value

    def packed_render_attn(self, q_pre, k_pre, v, anchor_k_pre, anchor_v, out, workspace, stream=None):
        """All chunks of one stage in one block-causal call; `workspace` is a
        device uint8 tensor of at least packed_workspace_bytes()."""
        d = self.desc
        shape = (d.total_frames * self.T, d.heads, d.head_dim)
        ashape = (((d.total_frames - 1) // d.anchor_stride + 1) * self.T, d.heads, d.head_dim)
        if not workspace.is_cuda or workspace.numel() * workspace.element_size() < self.packed_workspace_bytes():
            raise ValueError("workspace too small")
        _check(_lib().ff_packed_render_attn(
            self.handle, _ptr(q_pre, shape, "q_pre"), _ptr(k_pre, shape, "k_pre"), _ptr(v, shape, "v"),
            _ptr(anchor_k_pre, ashape, "anchor_k_pre"), _ptr(anchor_v, ashape, "anchor_v"), _ptr(out, shape, "out"),
            ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(),
            _stream(stream, self.device)), "ff_packed_render_attn")

    def render_attn_raw(self, layer, stage, chunk, q_ptr, k_ptr, v_ptr, out_ptr, stream_handle) -> int:
        """Pointer-level call (no checks in Python); returns the status code."""
        return _lib().ff_render_attn(self.handle, layer, stage, chunk, ctypes.c_void_p(q_ptr), ctypes.c_void_p(k_ptr),
                                     ctypes.c_void_p(v_ptr), ctypes.c_void_p(out_ptr), ctypes.c_void_p(stream_handle))

    def close(self):
        if self.handle:
            _lib().ff_bank_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- introspection ------------------------------------------------------
    @property
    def n_chunks(self):
        return -(-self.desc.total_frames // self.desc.chunk_frames)

    def gamma(self, chunk):
        l, r, n = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        _check(_lib().ff_bank_gamma(self.handle, chunk, ctypes.byref(l), ctypes.byref(r), ctypes.byref(n)),
               "ff_bank_gamma")
        return [l.value, r.value][:n.value]

    def slot_info(self, layer, stage, slot):
        tag, frames = ctypes.c_int(), ctypes.c_int()
        kp, vp = ctypes.c_void_p(), ctypes.c_void_p()
        _check(_lib().ff_bank_slot_info(self.handle, layer, stage, slot, ctypes.byref(tag), ctypes.byref(frames),
                                        ctypes.byref(kp), ctypes.byref(vp)), "ff_bank_slot_info")
        return tag.value, frames.value, kp.value, vp.value

    def slot_tensors(self, layer, stage, slot):
        """(tag, K, V) of a slot; K and V are uint16 (bf16 bit) views of bank memory."""
        import torch
        tag, frames, kp, vp = self.slot_info(layer, stage, slot)
        shape = (frames * self.T, self.desc.heads, self.desc.head_dim)
        if frames == 0:
            return tag, None, None
        with torch.cuda.device(self.device):
            k = torch.as_tensor(_DevView(kp, shape, self.device), device=f"cuda:{self.device}")
            v = torch.as_tensor(_DevView(vp, shape, self.device), device=f"cuda:{self.device}")
        return tag, k, v

    def bytes(self):
        n = ctypes.c_size_t()
        _check(_lib().ff_bank_bytes(self.handle, ctypes.byref(n)), "ff_bank_bytes")
        return n.value

    def error_poll(self):
        return _lib().ff_bank_error_poll(self.handle)

    def wait_probe(self, limit_ms: int, stream=None):
        """Enqueue the failure-detection self-test (a wait that times out)."""
        _check(_lib().ff_bank_wait_probe(self.handle, limit_ms, _stream(stream, self.device)), "ff_bank_wait_probe")

    def set_timing(self, enable: bool):
        _check(_lib().ff_bank_set_timing(self.handle, int(enable)), "ff_bank_set_timing")

    def read_timing(self) -> KernelTimes:
        t = KernelTimes()
        _check(_lib().ff_bank_read_timing(self.handle, ctypes.byref(t)), "ff_bank_read_timing")
        return t

    def kernel_count(self, chunk) -> int:
        c = ctypes.c_int()
        _check(_lib().ff_render_kernel_count(self.handle, chunk, ctypes.byref(c)), "ff_render_kernel_count")
        return c.value


class _Handle:
    """Owner of one libff cache: freed when neither the cache nor a view of its memory is left."""

    def __init__(self, kind, desc):
        self.handle, self._destroy = ctypes.c_void_p(), f"{kind}_destroy"
        _check(getattr(_lib(), f"{kind}_create")(ctypes.byref(desc), ctypes.byref(self.handle)), f"{kind}_create")

    def close(self):
        if self.handle:
            getattr(_lib(), self._destroy)(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _Cache:
    """What the caches share: the handle, checks of tensors, views of device memory."""

    _kind: str
    _desc: type

    def __init__(self, kw):
        import torch
        self.desc = self._desc()
        _check(getattr(_lib(), f"{self._kind}_desc_default")(ctypes.byref(self.desc)), f"{self._kind}_desc_default")
        if "heads" in kw and "kv_heads" not in kw:
            kw["kv_heads"] = kw["heads"]
        for k, v in kw.items():
            if not hasattr(self.desc, k):
                raise TypeError(f"unknown cache field {k}")
            setattr(self.desc, k, v)
        self._owner = _Handle(self._kind, self.desc)
        self.handle = self._owner.handle
        d = self.desc
        self.device, self.capacity = d.device, d.capacity
        self.heads, self.kv_heads, self.head_dim = d.heads, d.kv_heads, d.head_dim
        self._views = {}
        self._bf16, self._f32, self._i32 = torch.bfloat16, torch.float32, torch.int32
        # the current stream's handle without the Stream object around it, where torch offers that
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._current = raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)

    def _tensor(self, t, shape, dtype, name):
        # one test for the common case: these checks are most of a small call's time on the host
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == self.device:
            return t.data_ptr()
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous {dtype} CUDA tensor")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{self.device}")

    def _stream(self, stream):
        return self._current(self.device) if stream is None else stream.cuda_stream

    def _view(self, pointer, shape, kind):
        import torch
        with torch.cuda.device(self.device):
            return torch.as_tensor(_DevView(pointer.value, shape, self.device, kind, self._owner),
                                   device=f"cuda:{self.device}")

    def bytes(self):
        n = ctypes.c_size_t()
        _check(getattr(_lib(), f"{self._kind}_bytes")(self.handle, ctypes.byref(n)), f"{self._kind}_bytes")
        return n.value

    def error_poll(self):
        return getattr(_lib(), f"{self._kind}_error_poll")(self.handle)

    def close(self):
        """Free the cache now; its views must not be used any more."""
        self._views = {}
        self._owner.close()
        self.handle = self._owner.handle


class KV8Cache(_Cache):
    """Key/value cache in 8 bits with a scale for each block of 64 tokens and head (ff_kv8_* in include/ff.h).

    ``n_layers`` caches of ``batch`` sequences, up to ``capacity`` rows each.  Tensors are contiguous, on the
    cache's device: k, v, q, out bf16 [batch, n, heads, head_dim]; start, counts int32 [batch]; lse fp32
    [batch, n, heads]; weights fp32 [batch, kv_heads, capacity]."""

    _kind, _desc = "ff_kv8", KV8Desc

    def __init__(self, **kw):
        super().__init__(kw)
        self.batch = self.desc.batch

    def _per_sequence(self, t, name):
        return None if t is None else self._tensor(t, (self.batch,), self._i32, name)

    def append(self, layer, k, v, start=None, counts=None, stream=None):
        """Store rows behind those held, or at `start` (see ff_kv8_append)."""
        n = k.shape[1]
        shape = (self.batch, n, self.kv_heads, self.head_dim)
        _check(_LIB.ff_kv8_append(self.handle, layer, n, self._tensor(k, shape, self._bf16, "k"),
                                  self._tensor(v, shape, self._bf16, "v"), self._per_sequence(start, "start"),
                                  self._per_sequence(counts, "counts"), self._stream(stream)), "ff_kv8_append")

    def load(self, layer, k, v, start=None, stream=None):
        """Read k.shape[1] rows from `start` (default 0) back into k and v; rows not held read as zeros."""
        n = k.shape[1]
        shape = (self.batch, n, self.kv_heads, self.head_dim)
        _check(_LIB.ff_kv8_load(self.handle, layer, n, self._per_sequence(start, "start"),
                                self._tensor(k, shape, self._bf16, "k"), self._tensor(v, shape, self._bf16, "v"),
                                self._stream(stream)), "ff_kv8_load")

    def attn(self, layer, q, out, causal=False, counts=None, lse=None, weights=None, weights_in=None, stream=None):
        """Attention of q over the rows held, into out (see ff_kv8_attn)."""
        n = q.shape[1]
        shape = (self.batch, n, self.heads, self.head_dim)
        wshape = (self.batch, self.kv_heads, self.capacity)
        _check(_LIB.ff_kv8_attn(
            self.handle, layer, n, self._tensor(q, shape, self._bf16, "q"), self._per_sequence(counts, "counts"),
            1 if causal else 0, self._tensor(out, shape, self._bf16, "out"),
            None if lse is None else self._tensor(lse, shape[:3], self._f32, "lse"),
            None if weights_in is None else self._tensor(weights_in, wshape, self._f32, "weights_in"),
            None if weights is None else self._tensor(weights, wshape, self._f32, "weights"),
            self._stream(stream)), "ff_kv8_attn")

    def evict(self, layer, dst, dst_layer, n_keep, n_recent, weights, weights_out, kept, stream=None):
        """Keep the n_recent last and the heaviest other rows, n_keep in all, as the rows of a layer of `dst`
        (see ff_kv8_evict); kept: int32 [batch, kv_heads, n_keep]."""
        lists = (self.batch, self.kv_heads)
        _check(_LIB.ff_kv8_evict(
            self.handle, layer, dst.handle, dst_layer, n_keep, n_recent,
            self._tensor(weights, (*lists, self.capacity), self._f32, "weights"),
            self._tensor(weights_out, (*lists, dst.capacity), self._f32, "weights_out"),
            self._tensor(kept, (*lists, n_keep), self._i32, "kept"), self._stream(stream)), "ff_kv8_evict")

    # -- introspection ------------------------------------------------------
    def layer(self, layer):
        """Views of a layer: (k8, v8, k_scale, v_scale, lengths), codes as uint8 [batch, blocks, kv_heads, 64, d]."""
        if layer not in self._views:
            p = [ctypes.c_void_p() for _ in range(5)]
            _check(_lib().ff_kv8_layer_info(self.handle, layer, *[ctypes.byref(x) for x in p]), "ff_kv8_layer_info")
            tiles = (self.batch, -(-self.capacity // 64), self.kv_heads)
            codes = (*tiles, 64, self.head_dim)
            self._views[layer] = tuple(
                self._view(x, shape, kind) for x, shape, kind in
                zip(p, (codes, codes, tiles, tiles, (self.batch,)), ("|u1", "|u1", "<f4", "<f4", "<i4")))
        return self._views[layer]

    def lengths(self, layer):
        """View of the rows held by each sequence (int32)."""
        return self.layer(layer)[4]


class PagedCache(_Cache):
    """Key/value cache in pages that requests of different lengths share (ff_paged_* in include/ff.h).

    ``n_layers`` pools of ``pages`` pages of ``page_rows`` rows; up to ``requests`` requests of up to ``capacity`` rows
    each; steps of up to ``max_rows`` new rows, packed one request after the other.  Tensors are contiguous, on the
    cache's device: q, out bf16 [n, heads, head_dim]; k, v bf16 [n, kv_heads, head_dim]; start, counts int32
    [requests]; lse fp32 [n, heads]."""

    _kind, _desc = "ff_paged", PagedDesc

    def __init__(self, **kw):
        super().__init__(kw)
        d = self.desc
        self.pages, self.page_rows, self.requests, self.max_rows = d.pages, d.page_rows, d.requests, d.max_rows

    def plan(self, n, counts, start=None, stream=None):
        """Cut every request to `start` rows (default: all held), then add counts[r] new ones (see ff_paged_plan); the
        step's packed tensors have n rows."""
        each = (self.requests,)
        _check(_LIB.ff_paged_plan(self.handle, n, None if start is None else self._tensor(start, each, self._i32, "start"),
                                  self._tensor(counts, each, self._i32, "counts"), self._stream(stream)), "ff_paged_plan")

    def store(self, layer, k, v, stream=None):
        """Put the step's rows into their places (see ff_paged_store)."""
        n = k.shape[0]
        shape = (n, self.kv_heads, self.head_dim)
        _check(_LIB.ff_paged_store(self.handle, layer, n, self._tensor(k, shape, self._bf16, "k"),
                                   self._tensor(v, shape, self._bf16, "v"), self._stream(stream)), "ff_paged_store")

    def attn(self, layer, q, out, most=None, lse=None, stream=None):
        """Causal attention of the step's rows over the rows held, into out (see ff_paged_attn); most: the most new
        rows of any request of the step (default: q's rows)."""
        n = q.shape[0]
        shape = (n, self.heads, self.head_dim)
        _check(_LIB.ff_paged_attn(self.handle, layer, n, n if most is None else most, self._tensor(q, shape, self._bf16, "q"),
                                  self._tensor(out, shape, self._bf16, "out"),
                                  None if lse is None else self._tensor(lse, shape[:2], self._f32, "lse"),
                                  self._stream(stream)), "ff_paged_attn")

    # -- introspection ------------------------------------------------------
    def _table(self, name):
        if name not in self._views:
            p = [ctypes.c_void_p() for _ in range(7)]
            _check(_lib().ff_paged_info(self.handle, *[ctypes.byref(x) for x in p]), "ff_paged_info")
            shapes = dict(tables=(self.requests, -(-self.capacity // self.page_rows)), lengths=(self.requests,),
                          first=(self.requests + 1,), slots=(self.max_rows,), positions=(self.max_rows,),
                          free=(self.pages,), n_free=(1,))
            for x, (key, shape) in zip(p, shapes.items()):
                self._views[key] = self._view(x, shape, "<i4")
        return self._views[name]

    tables = property(lambda self: self._table("tables"), doc="View of the requests' pages (int32).")
    lengths = property(lambda self: self._table("lengths"), doc="View of the rows held by each request.")
    first = property(lambda self: self._table("first"), doc="View of where each request's rows begin in the packed tensors.")
    slots = property(lambda self: self._table("slots"), doc="View of the packed rows' places, -1 where there is none.")
    positions = property(lambda self: self._table("positions"), doc="View of the packed rows' indices in their requests.")
    free = property(lambda self: self._table("free"), doc="View of the stack of free pages.")
    n_free = property(lambda self: self._table("n_free"), doc="View of the number of free pages.")

    def layer(self, layer):
        """Views of a layer's pools (k, v): bf16 [pages, kv_heads, page_rows, head_dim]."""
        if layer not in self._views:
            p = [ctypes.c_void_p(), ctypes.c_void_p()]
            _check(_lib().ff_paged_layer_info(self.handle, layer, *[ctypes.byref(x) for x in p]), "ff_paged_layer_info")
            shape = (self.pages, self.kv_heads, self.page_rows, self.head_dim)
            self._views[layer] = tuple(self._view(x, shape, "<u2").view(self._bf16) for x in p)
        return self._views[layer]
