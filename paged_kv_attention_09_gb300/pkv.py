"""Python binding of libpkv.so: the C ABI of include/pkv.h, same names, argument
marshalling only.  Tensors are torch CUDA tensors (torch supplies device memory and
streams); every computation runs in the library's CUDA kernels.  There is no fallback:
if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpkv.so")

F32, BF16, INT8, FP8, INT4, INT8B, FP8B = 0, 1, 2, 3, 4, 5, 6
BLOCK_SCALED = (INT8B, FP8B)  # 8-bit codes with one FP32 scale per (page, kv head)
# stored as codes with one FP32 scale per (token, kv head), or per block of a page's tokens
CODED = (INT8, FP8, INT4) + BLOCK_SCALED
# element containers of the cache tensors (FP8 codes and INT4 code pairs as raw bytes)
# (INT8 bytes hold code + 128, offset binary)
_TORCH_DTYPE = {F32: torch.float32, BF16: torch.bfloat16, INT8: torch.uint8, FP8: torch.uint8,
                INT4: torch.uint8, INT8B: torch.uint8, FP8B: torch.uint8}
_CODE = {torch.float32: F32, torch.bfloat16: BF16}

DEV_BAD_PAGE, DEV_BAD_LEN, DEV_BAD_SLOT, DEV_BAD_CHUNK, DEV_TIMEOUT = 0x1, 0x2, 0x4, 0x8, 0x10
DEV_NO_PAGES = 0x20
STATUS = {0: "PKV_OK", 1: "PKV_ERR_NULL", 2: "PKV_ERR_SHAPE", 3: "PKV_ERR_DTYPE",
          4: "PKV_ERR_PAGE_SIZE", 5: "PKV_ERR_ALIGN", 6: "PKV_ERR_WORKSPACE",
          7: "PKV_ERR_UNSUPPORTED", 8: "PKV_ERR_LAUNCH", 9: "PKV_ERR_DEVICE"}
EXPORTS = ("pkv_append", "pkv_decode_workspace_size", "pkv_decode_attn", "pkv_decode_step",
           "pkv_decode_workspace_size_ex", "pkv_decode_attn_ex", "pkv_decode_step_ex",
           "pkv_prefill_workspace_size", "pkv_prefill_chunk_attn",
           "pkv_prefill_workspace_size_ex", "pkv_prefill_chunk_attn_ex",
           "pkv_decode_attn_noalloc", "pkv_decode_attn_noalloc_ex", "pkv_status_string",
           "pkv_decode_graph_workspace_size", "pkv_decode_graph_create",
           "pkv_decode_graph_launch", "pkv_decode_graph_bucket", "pkv_decode_graph_destroy",
           "pkv_batch_tables", "pkv_rope_plan_init", "pkv_rope")
GRAPH_MAX_BUCKETS = 16
NOALLOC_SCRATCH_BYTES = 4 << 20


class PkvError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)}")
        self.code = code


class pkv_cache(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("window", ctypes.c_int32)]


class pkv_decode_opts(ctypes.Structure):
    _fields_ = [("split_pages", ctypes.c_int32)]


class pkv_prefill_opts(ctypes.Structure):
    _fields_ = [("key_split", ctypes.c_int32)]


class pkv_graph_layer(ctypes.Structure):
    _fields_ = [("cache", pkv_cache), ("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p),
                ("v_new", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class pkv_decode_graph_desc(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("layers", ctypes.POINTER(pkv_graph_layer)),
                ("num_q_heads", ctypes.c_int32), ("q_dtype", ctypes.c_int32),
                ("new_dtype", ctypes.c_int32), ("fused", ctypes.c_int32),
                ("block_tables", ctypes.c_void_p), ("max_blocks_per_seq", ctypes.c_int32),
                ("context_lens", ctypes.c_void_p), ("slot_mapping", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("rope_theta", ctypes.c_double),
                ("scale", ctypes.c_float), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("dev_status", ctypes.c_void_p),
                ("num_buckets", ctypes.c_int32), ("buckets", ctypes.POINTER(ctypes.c_int32))]


class pkv_page_pool(ctypes.Structure):
    _fields_ = [("ring", ctypes.c_void_p), ("state", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)]


ROPE_MAX_PAIRS = 128
ROPE_LAYOUT = {"half": 0, "interleaved": 1}
ROPE_SCALING = {"none": 0, "linear": 1, "base": 2, "bands": 3}


class pkv_rope_params(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("transposed", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("original_len", ctypes.c_int32), ("attention_factor", ctypes.c_float)]


class pkv_rope_plan(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("transposed", ctypes.c_int32), ("attention_factor", ctypes.c_float),
                ("freq", ctypes.c_uint64 * ROPE_MAX_PAIRS)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libpkv.so (build it with __graft_entry__.build()); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = bind(path)
    return _lib


def bind(path: str):
    """A handle on the library at ``path`` with every entry point's argument types (a
    variant build, e.g. a test build, is used beside the product library this way)."""
    if not os.path.exists(path):
        raise RuntimeError(f"libpkv.so not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, I32, F, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    C = ctypes.POINTER(pkv_cache)
    lib.pkv_append.argtypes = [C, P, P, I32, P, I32, P, P]
    O = ctypes.POINTER(pkv_decode_opts)
    lib.pkv_decode_workspace_size.argtypes = [C, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.pkv_decode_workspace_size_ex.argtypes = [C, I32, I32, I32, O, ctypes.POINTER(SZ)]
    lib.pkv_decode_attn.argtypes = [C, P, I32, I32, I32, P, I32, P, F, P, P, SZ, P, P]
    lib.pkv_decode_attn_ex.argtypes = [C, P, I32, I32, I32, P, I32, P, F, P, P, SZ, O, P, P]
    lib.pkv_decode_step.argtypes = [C, P, I32, P, P, I32, P, P, ctypes.c_double, I32, I32, P,
                                    I32, P, F, P, P, SZ, P, P]
    lib.pkv_decode_step_ex.argtypes = [C, P, I32, P, P, I32, P, P, ctypes.c_double, I32, I32,
                                       P, I32, P, F, P, P, SZ, O, P, P]
    lib.pkv_prefill_workspace_size.argtypes = [C, I32, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.pkv_prefill_chunk_attn.argtypes = [C, P, I32, I32, I32, P, I32, P, I32, P, F, P, P, SZ,
                                           P, P]
    PO = ctypes.POINTER(pkv_prefill_opts)
    lib.pkv_prefill_workspace_size_ex.argtypes = [C, I32, I32, I32, I32, PO, ctypes.POINTER(SZ)]
    lib.pkv_prefill_chunk_attn_ex.argtypes = [C, P, I32, I32, I32, P, I32, P, I32, P, F, P, P,
                                              SZ, PO, P, P]
    for fn in ("pkv_append", "pkv_decode_workspace_size", "pkv_decode_attn", "pkv_decode_step",
               "pkv_decode_workspace_size_ex", "pkv_decode_attn_ex", "pkv_decode_step_ex",
               "pkv_prefill_workspace_size", "pkv_prefill_chunk_attn",
               "pkv_prefill_workspace_size_ex", "pkv_prefill_chunk_attn_ex"):
        getattr(lib, fn).restype = ctypes.c_int
    lib.pkv_decode_attn_noalloc.argtypes = [C, P, I32, I32, I32, P, I32, P, F, P, P, P]
    lib.pkv_decode_attn_noalloc.restype = ctypes.c_int
    lib.pkv_decode_attn_noalloc_ex.argtypes = [C, P, I32, I32, I32, P, I32, P, F, P, O, P, P]
    lib.pkv_decode_attn_noalloc_ex.restype = ctypes.c_int
    lib.pkv_status_string.argtypes = [ctypes.c_int]
    lib.pkv_status_string.restype = ctypes.c_char_p
    I64 = ctypes.c_int64
    lib.pkv_batch_tables.argtypes = [ctypes.POINTER(pkv_page_pool), P, P, I32, P, I32, P, P, P, P,
                                     I32, P, P]
    lib.pkv_rope_plan_init.argtypes = [ctypes.POINTER(pkv_rope_params),
                                       ctypes.POINTER(pkv_rope_plan)]
    lib.pkv_rope.argtypes = [ctypes.POINTER(pkv_rope_plan), P, P, I64, I64, I32, P, P, I64, I64,
                             I32, I32, I32, I32, P, P, P]
    for fn in ("pkv_batch_tables", "pkv_rope_plan_init", "pkv_rope"):
        getattr(lib, fn).restype = ctypes.c_int
    GD = ctypes.POINTER(pkv_decode_graph_desc)
    lib.pkv_decode_graph_workspace_size.argtypes = [GD, ctypes.POINTER(SZ)]
    lib.pkv_decode_graph_create.argtypes = [GD, ctypes.POINTER(ctypes.c_void_p)]
    lib.pkv_decode_graph_launch.argtypes = [P, I32, P]
    lib.pkv_decode_graph_bucket.argtypes = [P, I32]
    lib.pkv_decode_graph_destroy.argtypes = [P]
    lib.pkv_decode_graph_destroy.restype = None
    for fn in ("pkv_decode_graph_workspace_size", "pkv_decode_graph_create",
               "pkv_decode_graph_launch", "pkv_decode_graph_bucket"):
        getattr(lib, fn).restype = ctypes.c_int
    return lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without building a Stream object (a microsecond or two per
# call), where this torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _current_device() -> int:
    """torch.cuda.current_device() of a process whose CUDA is initialised."""
    return torch.cuda.current_device() if _get_device is None else _get_device()


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return ctypes.c_void_p(_raw_stream(_current_device()))
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(code: int, what: str):
    if code != 0:
        raise PkvError(code, what)


class BoundCall:
    """One library call with its arguments marshalled once: the cache struct, device
    pointers, sizes, options and stream.  Calling it issues the same C call again, with no
    Python work beyond the ctypes call itself (about a microsecond against ~10 for the
    full wrapper), for loops that repeat a launch on fixed buffers.  The caller keeps the
    tensors alive and their contents current; a non-zero status raises PkvError."""

    __slots__ = ("_fn", "_args", "_what")

    def __init__(self, fn, args, what: str):
        self._fn, self._args, self._what = fn, tuple(args), what

    def __call__(self) -> None:
        code = self._fn(*self._args)
        if code != 0:
            raise PkvError(code, self._what)


def _call(fn, args, what: str, bound: bool):
    """Issue the call now, or (bound=True) return it as a BoundCall without issuing it."""
    if bound:
        return BoundCall(fn, args, what)
    _check(fn(*args), what)
    return None


class KVCache:
    """Device tensors of one paged cache in the library's layout.

    k: [num_pages, Hkv, 16, D]; v: [num_pages, Hkv, D, 16] (page blocks transposed);
    k_scale, v_scale: float32 [num_pages, Hkv, 16] for INT8, FP8 and INT4 caches,
    [num_pages, Hkv] for INT8B and FP8B.  For
    BF16 caches the elements inside each (page, kv head) block are in tensor-core tile
    order, FP8 codes are bytes, and INT4 blocks hold two codes per byte (k: [.., 16, D/2],
    v: [.., D/2, 16] bytes); see include/pkv.h.  The tensor shapes are containers of the
    right size.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None, window=0, kv_dtype=None):
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.kv_dtype = _CODE[k.dtype] if kv_dtype is None else int(kv_dtype)
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = k.shape
        if self.kv_dtype == INT4:
            self.head_dim *= 2
        self.window = int(window)  # sliding window in tokens (0: none), read by every call
        self._struct = self._made = None

    @classmethod
    def allocate(cls, num_pages, num_kv_heads, head_dim, kv_dtype, device="cuda",
                 page_size=16):
        dt = _TORCH_DTYPE[kv_dtype]
        if kv_dtype == INT4:
            k = torch.zeros(num_pages, num_kv_heads, page_size, head_dim // 2, dtype=dt, device=device)
            v = torch.zeros(num_pages, num_kv_heads, head_dim // 2, page_size, dtype=dt, device=device)
        else:
            k = torch.zeros(num_pages, num_kv_heads, page_size, head_dim, dtype=dt, device=device)
            v = torch.zeros(num_pages, num_kv_heads, head_dim, page_size, dtype=dt, device=device)
        ks = vs = None
        if kv_dtype in CODED:
            per = () if kv_dtype in BLOCK_SCALED else (page_size,)
            ks = torch.zeros(num_pages, num_kv_heads, *per, dtype=torch.float32, device=device)
            vs = torch.zeros_like(ks)
        return cls(k, v, ks, vs, kv_dtype=kv_dtype)

    def clone(self) -> "KVCache":
        """A copy in fresh device memory (same format and window)."""
        return KVCache(self.k.clone(), self.v.clone(),
                       None if self.k_scale is None else self.k_scale.clone(),
                       None if self.v_scale is None else self.v_scale.clone(),
                       window=self.window, kv_dtype=self.kv_dtype)

    def struct(self) -> pkv_cache:
        """The C descriptor: made once and again whenever a tensor or the window changes (a
        bound call keeps the one it was made with; not to be written to)."""
        ks, vs = self.k_scale, self.v_scale
        now = (self.k.data_ptr(), self.v.data_ptr(), None if ks is None else ks.data_ptr(),
               None if vs is None else vs.data_ptr(), self.num_pages, self.page_size,
               self.num_kv_heads, self.head_dim, self.kv_dtype, self.window)
        if now != self._made:
            self._struct, self._made = pkv_cache(*now), now
        return self._struct


def pkv_status_string(code: int) -> str:
    return load().pkv_status_string(code).decode()


def _opts(split_pages: int):
    """The options argument of the _ex calls (None: every option at its default)."""
    return None if not split_pages else ctypes.byref(pkv_decode_opts(int(split_pages)))


def _rows_in(cache: KVCache, k_new, v_new, slots) -> None:
    """New rows of a block-scaled cache: dense, alike, one for each slot."""
    n = slots.shape[0] * cache.num_kv_heads * cache.head_dim
    if k_new.dtype is not v_new.dtype or k_new.numel() != n or v_new.numel() != n or \
            not (k_new.is_contiguous() and v_new.is_contiguous()):
        raise ValueError("pkv_append: contiguous k_new and v_new [tokens, kv heads, head_dim] of one "
                         "type are wanted, a row for each slot")


def _rows_out(cache: KVCache, q, out, what: str) -> None:
    """Query and output rows over a block-scaled cache: dense, of the cache's head_dim."""
    if q.shape[2] != cache.head_dim or out.dtype is not torch.float32 or out.numel() < q.numel() or \
            not (q.is_contiguous() and out.is_contiguous()):
        raise ValueError(f"{what}: contiguous q [rows, heads, head_dim] and a float32 out of its shape "
                         "are wanted")


def pkv_append(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor,
               slot_mapping: torch.Tensor, dev_status: Optional[torch.Tensor] = None,
               stream=None, bound: bool = False) -> Optional[BoundCall]:
    c = cache.struct()
    if cache.kv_dtype in BLOCK_SCALED:
        _rows_in(cache, k_new, v_new, slot_mapping)
    return _call(load().pkv_append,
                 (ctypes.byref(c), _ptr(k_new), _ptr(v_new), _CODE[k_new.dtype],
                  _ptr(slot_mapping), int(slot_mapping.shape[0]), _ptr(dev_status),
                  _stream(stream)), "pkv_append", bound)


def pkv_decode_workspace_size(cache: KVCache, num_seqs: int, num_q_heads: int,
                              max_blocks_per_seq: int, split_pages: int = 0) -> int:
    """Scratch bytes of the decode calls for this shape; ``split_pages`` as in
    pkv_decode_opts (0: automatic)."""
    c = cache.struct()
    n = ctypes.c_size_t(0)
    _check(load().pkv_decode_workspace_size_ex(ctypes.byref(c), num_seqs, num_q_heads,
                                               max_blocks_per_seq, _opts(split_pages),
                                               ctypes.byref(n)),
           "pkv_decode_workspace_size")
    return int(n.value)


def pkv_decode_attn(cache: KVCache, q: torch.Tensor, block_tables: torch.Tensor,
                    context_lens: torch.Tensor, scale: float, out: torch.Tensor,
                    workspace: Optional[torch.Tensor] = None,
                    dev_status: Optional[torch.Tensor] = None, stream=None,
                    split_pages: int = 0, bound: bool = False) -> Optional[BoundCall]:
    c = cache.struct()
    B, Hq, _ = q.shape
    if cache.kv_dtype in BLOCK_SCALED:
        _rows_out(cache, q, out, "pkv_decode_attn")
    wb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _call(load().pkv_decode_attn_ex,
                 (ctypes.byref(c), _ptr(q), _CODE[q.dtype], B, Hq, _ptr(block_tables),
                  int(block_tables.shape[1]), _ptr(context_lens), float(scale), _ptr(out),
                  _ptr(workspace), wb, _opts(split_pages), _ptr(dev_status), _stream(stream)),
                 "pkv_decode_attn", bound)


def pkv_decode_step(cache: KVCache, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                    slot_mapping: torch.Tensor, positions: Optional[torch.Tensor],
                    rope_theta: float, block_tables: torch.Tensor, context_lens: torch.Tensor,
                    scale: float, out: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                    dev_status: Optional[torch.Tensor] = None, stream=None,
                    split_pages: int = 0, bound: bool = False) -> Optional[BoundCall]:
    """One fused decode step (rotate, append the new row, attend); see include/pkv.h."""
    c = cache.struct()
    B, Hq, _ = q.shape
    wb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _call(load().pkv_decode_step_ex,
                 (ctypes.byref(c), _ptr(q), _CODE[q.dtype], _ptr(k_new), _ptr(v_new),
                  _CODE[k_new.dtype], _ptr(slot_mapping), _ptr(positions), float(rope_theta),
                  B, Hq, _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens),
                  float(scale), _ptr(out), _ptr(workspace), wb, _opts(split_pages),
                  _ptr(dev_status), _stream(stream)), "pkv_decode_step", bound)


class GraphLayer:
    """One layer of a decode-graph step: its cache, query rows, new K/V rows (or None: no
    append) and output, all sized for the largest bucket."""

    def __init__(self, cache: KVCache, q: torch.Tensor, out: torch.Tensor,
                 k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None):
        self.cache, self.q, self.out, self.k_new, self.v_new = cache, q, out, k_new, v_new


class DecodeGraph:
    """pkv_decode_graph: one captured CUDA graph per batch-size bucket (see include/pkv.h).

    The tensors are captured by address and must stay alive (and in place) for the
    executor's lifetime; rows past a launch's num_seqs up to its bucket must be inert
    (context_lens 0, slot_mapping -1).  The workspace is allocated here, zero-filled."""

    def __init__(self, layers, block_tables: torch.Tensor, context_lens: torch.Tensor,
                 scale: float, buckets, slot_mapping: Optional[torch.Tensor] = None,
                 fused: bool = False, positions: Optional[torch.Tensor] = None,
                 rope_theta: float = 10000.0, dev_status: Optional[torch.Tensor] = None):
        lib = load()
        self.layers = list(layers)
        self._keep = (block_tables, context_lens, slot_mapping, positions, dev_status)
        arr = (pkv_graph_layer * len(self.layers))()
        for i, L in enumerate(self.layers):
            arr[i] = pkv_graph_layer(L.cache.struct(), _ptr(L.q), _ptr(L.k_new), _ptr(L.v_new),
                                     _ptr(L.out))
        self._arr = arr
        self._buckets = (ctypes.c_int32 * len(buckets))(*[int(b) for b in buckets])
        q0 = self.layers[0].q
        k0 = next((L.k_new for L in self.layers if L.k_new is not None), None)
        d = pkv_decode_graph_desc()
        d.num_layers = len(self.layers)
        d.layers = ctypes.cast(arr, ctypes.POINTER(pkv_graph_layer))
        d.num_q_heads = int(q0.shape[1])
        d.q_dtype = _CODE[q0.dtype]
        d.new_dtype = _CODE[k0.dtype] if k0 is not None else F32
        d.fused = 1 if fused else 0
        d.block_tables = _ptr(block_tables)
        d.max_blocks_per_seq = int(block_tables.shape[1])
        d.context_lens = _ptr(context_lens)
        d.slot_mapping = _ptr(slot_mapping)
        d.positions = _ptr(positions)
        d.rope_theta = float(rope_theta)
        d.scale = float(scale)
        d.dev_status = _ptr(dev_status)
        d.num_buckets = len(buckets)
        d.buckets = ctypes.cast(self._buckets, ctypes.POINTER(ctypes.c_int32))
        n = ctypes.c_size_t(0)
        _check(lib.pkv_decode_graph_workspace_size(ctypes.byref(d), ctypes.byref(n)),
               "pkv_decode_graph_workspace_size")
        self.workspace = workspace_for(int(n.value), q0.device)
        d.workspace = _ptr(self.workspace)
        d.workspace_bytes = int(n.value)
        self._desc = d
        h = ctypes.c_void_p(None)
        _check(lib.pkv_decode_graph_create(ctypes.byref(d), ctypes.byref(h)),
               "pkv_decode_graph_create")
        self._h = h

    def bucket(self, num_seqs: int) -> int:
        return int(load().pkv_decode_graph_bucket(self._h, int(num_seqs)))

    def launch(self, num_seqs: int, stream=None) -> None:
        _check(load().pkv_decode_graph_launch(self._h, int(num_seqs), _stream(stream)),
               "pkv_decode_graph_launch")

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            load().pkv_decode_graph_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def pkv_decode_attn_noalloc(cache: KVCache, q: torch.Tensor, block_tables: torch.Tensor,
                            context_lens: torch.Tensor, scale: float, out: torch.Tensor,
                            dev_status: Optional[torch.Tensor] = None, stream=None,
                            split_pages: int = 0) -> None:
    """pkv_decode_attn with its split scratch in the library's fixed device array (for
    callers that cannot allocate); see include/pkv.h for the size limit and sharing."""
    c = cache.struct()
    B, Hq, _ = q.shape
    if cache.kv_dtype in BLOCK_SCALED:
        _rows_out(cache, q, out, "pkv_decode_attn_noalloc")
    _check(load().pkv_decode_attn_noalloc_ex(ctypes.byref(c), _ptr(q), _CODE[q.dtype], B, Hq,
                                             _ptr(block_tables), int(block_tables.shape[1]),
                                             _ptr(context_lens), float(scale), _ptr(out),
                                             _opts(split_pages), _ptr(dev_status),
                                             _stream(stream)),
           "pkv_decode_attn_noalloc")


def _prefill_opts(key_split: int):
    """The options argument of the prefill _ex calls (None: every option at its default)."""
    return None if not key_split else ctypes.byref(pkv_prefill_opts(int(key_split)))


def pkv_prefill_workspace_size(cache: KVCache, num_seqs: int, num_q_heads: int,
                               max_q_len: int, max_blocks_per_seq: int,
                               key_split: int = 0) -> int:
    """Scratch bytes of pkv_prefill_chunk_attn; key_split (0: automatic, 1..3) is the
    pkv_prefill_opts option."""
    c = cache.struct()
    n = ctypes.c_size_t(0)
    _check(load().pkv_prefill_workspace_size_ex(ctypes.byref(c), num_seqs, num_q_heads,
                                                max_q_len, max_blocks_per_seq,
                                                _prefill_opts(key_split), ctypes.byref(n)),
           "pkv_prefill_workspace_size")
    return int(n.value)


def pkv_prefill_chunk_attn(cache: KVCache, q: torch.Tensor, q_start_loc: torch.Tensor,
                           max_q_len: int, block_tables: torch.Tensor,
                           context_lens: torch.Tensor, scale: float, out: torch.Tensor,
                           workspace: Optional[torch.Tensor] = None,
                           dev_status: Optional[torch.Tensor] = None, stream=None,
                           key_split: int = 0, bound: bool = False) -> Optional[BoundCall]:
    c = cache.struct()
    B = int(context_lens.shape[0])
    Hq = int(q.shape[1])
    if cache.kv_dtype in BLOCK_SCALED:
        _rows_out(cache, q, out, "pkv_prefill_chunk_attn")
    wb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _call(load().pkv_prefill_chunk_attn_ex,
                 (ctypes.byref(c), _ptr(q), _CODE[q.dtype], B, Hq, _ptr(q_start_loc),
                  int(max_q_len), _ptr(block_tables), int(block_tables.shape[1]),
                  _ptr(context_lens), float(scale), _ptr(out), _ptr(workspace), wb,
                  _prefill_opts(key_split), _ptr(dev_status), _stream(stream)),
                 "pkv_prefill_chunk_attn", bound)


class PagePool:
    """A pool of page ids on the GPU, from which pkv_batch_tables takes the new pages of a
    step and to which it returns those of ended requests (see include/pkv.h).

    ring: int32 [num_pages]; state: int32 [4], the first free entry and their number."""

    def __init__(self, ring: torch.Tensor, state: torch.Tensor, page_size: int = 16):
        _int32("ring", ring, 1)
        _int32("state", state, 1, ring.device)
        if state.numel() < 4:
            raise ValueError("state: int32 [4] is wanted")
        self.ring, self.state, self.index = ring, state, ring.get_device()
        self._struct = pkv_page_pool(ring.data_ptr(), state.data_ptr(), ring.numel(), page_size)
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def allocate(cls, num_pages: int, device="cuda") -> "PagePool":
        """A pool with all its pages free."""
        return cls(torch.arange(num_pages, dtype=torch.int32, device=device),
                   torch.tensor([0, num_pages, 0, 0], dtype=torch.int32, device=device))


def _int32(name: str, t: torch.Tensor, dims: int, device=None) -> None:
    if t.dtype is not torch.int32 or t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 tensor of {dims} dimension(s) is wanted, "
                         f"got {t.dtype} {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _is_int32(t: torch.Tensor, shape: tuple, index: int) -> bool:
    """A contiguous int32 tensor of this shape on this device (get_device's number)."""
    return t.dtype is torch.int32 and t.shape == shape and t.is_contiguous() and \
        t.get_device() == index


def _issue(fn, args, what: str, bound: bool, index: int):
    """_call with the tensors' device current (a bound call is issued as the caller's
    current device stands: bind and issue it there).  index: the device's number, -1: CPU."""
    if bound:
        return BoundCall(fn, args, what)
    if index >= 0 and index != _current_device():
        with torch.cuda.device(index):
            code = fn(*args)
    else:
        code = fn(*args)
    if code != 0:
        raise PkvError(code, what)
    return None


def _stream_on(stream, index: int) -> int:
    """The stream argument: given, or the current stream of the tensors' device."""
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(index)
        return torch.cuda.current_stream(index).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def pkv_batch_tables(pool: PagePool, cached_lens: torch.Tensor, new_lens: torch.Tensor,
                     block_tables: torch.Tensor, context_lens: torch.Tensor,
                     q_start_loc: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                     slot_mapping: torch.Tensor, dev_status: Optional[torch.Tensor] = None,
                     stream=None, bound: bool = False) -> Optional[BoundCall]:
    """One step's tables from the requests' lengths; see include/pkv.h.  The row buffers
    (positions, slot_mapping) are filled to their end, padding rows with -1."""
    index = pool.index
    B, T = cached_lens.shape[0], slot_mapping.shape[0]
    rows, one = (T,), (B,)
    bt_shape = block_tables.shape
    if not (_is_int32(cached_lens, one, index) and _is_int32(new_lens, one, index)
            and _is_int32(context_lens, one, index) and _is_int32(slot_mapping, rows, index)
            and bt_shape[0] == B and _is_int32(block_tables, bt_shape, index)
            and len(bt_shape) == 2
            and (q_start_loc is None or _is_int32(q_start_loc, (B + 1,), index))
            and (positions is None or _is_int32(positions, rows, index))
            and (dev_status is None or _is_int32(dev_status, dev_status.shape, index))):
        raise ValueError("pkv_batch_tables: contiguous int32 tensors on the pool's device are wanted: "
                         "cached_lens, new_lens and context_lens [B], block_tables [B, blocks], "
                         "q_start_loc [B + 1], positions and slot_mapping [rows]")
    return _issue(load().pkv_batch_tables,
                  (pool._ref, cached_lens.data_ptr(), new_lens.data_ptr(), B,
                   block_tables.data_ptr(), bt_shape[1], context_lens.data_ptr(),
                   None if q_start_loc is None else q_start_loc.data_ptr(),
                   None if positions is None else positions.data_ptr(), slot_mapping.data_ptr(), T,
                   None if dev_status is None else dev_status.data_ptr(),
                   _stream_on(stream, index)),
                  "pkv_batch_tables", bound, index)


class RopeParams:
    """The turn that pkv_rope makes: layout "half" or "interleaved", scaling "none",
    "linear", "base" or "bands" (see include/pkv.h); its frequencies are computed here,
    once.  ``transposed`` turns by the opposite angle, which is the gradient."""

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, layout: str = "half",
                 theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 low: float = 1.0, high: float = 32.0, original_len: int = 1,
                 attention_factor: float = 1.0, transposed: bool = False):
        self.head_dim = int(head_dim)
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        p = pkv_rope_params(self.rotary_dim, ROPE_LAYOUT[layout], int(transposed),
                            ROPE_SCALING[scaling], float(theta), float(factor), float(low),
                            float(high), int(original_len), float(attention_factor))
        if self.rotary_dim > self.head_dim:
            raise PkvError(2, "pkv_rope_plan_init")
        self._plan = pkv_rope_plan()
        _check(load().pkv_rope_plan_init(ctypes.byref(p), ctypes.byref(self._plan)),
               "pkv_rope_plan_init")
        self._ref = ctypes.byref(self._plan)


def _rope_rows(name: str, x: torch.Tensor, shape: tuple, dtype, index: int) -> int:
    """Checks rows [T, heads, D] whose heads lie side by side; their token stride."""
    st = x.stride()
    if x.shape != shape or x.dtype is not dtype or x.get_device() != index:
        raise ValueError(f"{name}: {dtype} {shape} on device {index} is wanted, got {x.dtype} "
                         f"{tuple(x.shape)} on {x.device}")
    T, H, D = shape
    if (st[2] != 1 and D > 1) or (st[1] != D and H > 1):
        raise ValueError(f"{name}: the heads of a token must lie side by side (strides {st})")
    return st[0] if T > 1 else 0


def pkv_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
             params: RopeParams, q_out: Optional[torch.Tensor] = None,
             k_out: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
             stream=None, bound: bool = False) -> Optional[BoundCall]:
    """Turns the rows of q [T, Hq, D] and k [T, Hkv, D] (k may be None) at their positions,
    into q_out and k_out or, where those are None, in place; see include/pkv.h.  The rows may
    be views with any token stride."""
    shape = q.shape
    T, Hq, D = shape
    if D != params.head_dim:
        raise ValueError(f"q has heads of {D} columns, the parameters {params.head_dim}")
    index, dtype = q.get_device(), q.dtype
    if not _is_int32(positions, (T,), index):
        raise ValueError("positions: a contiguous int32 tensor with one entry for each row of q "
                         "on q's device is wanted")
    qp = qop = q.data_ptr()
    qs = qos = _rope_rows("q", q, shape, dtype, index)
    if q_out is not None:
        qop, qos = q_out.data_ptr(), _rope_rows("q_out", q_out, shape, dtype, index)
    kp = kop = None
    ks = kos = Hk = 0
    if k is not None:
        Hk = k.shape[1]
        shape = (T, Hk, D)
        kp = kop = k.data_ptr()
        ks = kos = _rope_rows("k", k, shape, dtype, index)
        if k_out is not None:
            kop, kos = k_out.data_ptr(), _rope_rows("k_out", k_out, shape, dtype, index)
    return _issue(load().pkv_rope,
                  (params._ref, qp, qop, qs, qos, Hq, kp, kop, ks, kos, Hk, _CODE[dtype], T, D,
                   positions.data_ptr(), None if dev_status is None else dev_status.data_ptr(),
                   _stream_on(stream, index)),
                  "pkv_rope", bound, index)


def workspace_for(nbytes: int, device="cuda") -> Optional[torch.Tensor]:
    """A zero-filled workspace tensor of at least nbytes (16-byte aligned), or None."""
    if nbytes == 0:
        return None
    return torch.zeros((nbytes + 15) // 16 * 4, dtype=torch.int32, device=device)
