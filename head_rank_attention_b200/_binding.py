"""ctypes binding of libhra.so (include/hra.h).  Argument marshalling only: every step of
the decode runs in the library's CUDA kernels.  There is no fallback: if the library is
missing or fails to load, importing a call raises.
"""
from __future__ import annotations

import ctypes
import math
import pathlib
from typing import Optional

LIB_PATH = pathlib.Path(__file__).resolve().with_name("libhra.so")

HRA_OK = 0
HRA_ERR_INVALID_ARG = -1
HRA_ERR_UNSUPPORTED = -2
HRA_ERR_WORKSPACE = -3
HRA_ERR_CUDA = -4
HRA_ERR_DEVICE_TIMEOUT = -5
HRA_BF16 = 0
HRA_F32 = 1
HRA_INT8 = 2
HRA_E4M3 = 3
HRA_ERR_PLAN = -6
HRA_VERSION = "0.2.0"  # of the header whose structs are mirrored below

STATUS_NAMES = {0: "HRA_OK", -1: "HRA_ERR_INVALID_ARG", -2: "HRA_ERR_UNSUPPORTED", -3: "HRA_ERR_WORKSPACE",
                -4: "HRA_ERR_CUDA", -5: "HRA_ERR_DEVICE_TIMEOUT", -6: "HRA_ERR_PLAN"}

# Symbols declared in include/hra.h.
EXPORTS = ("hra_workspace_size", "mlra_decode", "mla_decode", "mlra_decode_static", "hra_check_device_status",
           "hra_selftest_wait_timeout", "hra_last_error", "hra_version", "hra_prefill_workspace_size", "mlra_prefill",
           "hra_check_prefill_status", "hra_combine_partials", "hra_page_plan", "hra_check_plan_status",
           "hra_cache_append", "hra_cache_load")


class HraError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class HraDecodeParams(ctypes.Structure):
    """Mirror of hra_decode_params (field order and C types as in include/hra.h)."""
    _fields_ = [
        ("batch", ctypes.c_int), ("num_heads", ctypes.c_int), ("n_branch", ctypes.c_int),
        ("d_c", ctypes.c_int), ("d_rope", ctypes.c_int), ("d_nope", ctypes.c_int), ("d_v", ctypes.c_int),
        ("q", ctypes.c_void_p), ("ckv", ctypes.c_void_p), ("krope", ctypes.c_void_p),
        ("ckv_stride", ctypes.c_int64), ("krope_stride", ctypes.c_int64), ("cache_rows", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("seq_stride", ctypes.c_int64),
        ("w_uk", ctypes.c_void_p), ("w_uv", ctypes.c_void_p),
        ("alpha_q", ctypes.c_float), ("alpha_kv", ctypes.c_float), ("branch_scale", ctypes.c_float),
        ("softmax_scale", ctypes.c_float), ("rope_theta", ctypes.c_float),
        ("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("num_splits", ctypes.c_int), ("wait_limit", ctypes.c_int),
        ("stage_events", ctypes.c_void_p),
        ("out_accumulate", ctypes.c_int), ("n_out_peers", ctypes.c_int), ("out_peers", ctypes.c_void_p),
        ("cache_dtype", ctypes.c_int), ("ckv_scale", ctypes.c_void_p), ("ckv_scale_stride", ctypes.c_int64),
        ("q_positions", ctypes.c_void_p), ("part_o", ctypes.c_void_p), ("part_lse", ctypes.c_void_p),
        ("scale_block", ctypes.c_int),
    ]


class HraPrefillParams(ctypes.Structure):
    """Mirror of hra_prefill_params (field order and C types as in include/hra.h)."""
    _fields_ = [
        ("num_heads", ctypes.c_int), ("n_branch", ctypes.c_int),
        ("d_c", ctypes.c_int), ("d_rope", ctypes.c_int), ("d_nope", ctypes.c_int), ("d_v", ctypes.c_int),
        ("seq_len", ctypes.c_int), ("n_query", ctypes.c_int),
        ("q", ctypes.c_void_p), ("ckv", ctypes.c_void_p), ("krope", ctypes.c_void_p),
        ("ckv_stride", ctypes.c_int64), ("krope_stride", ctypes.c_int64),
        ("w_uk", ctypes.c_void_p), ("w_uv", ctypes.c_void_p),
        ("alpha_q", ctypes.c_float), ("alpha_kv", ctypes.c_float), ("branch_scale", ctypes.c_float),
        ("softmax_scale", ctypes.c_float), ("rope_theta", ctypes.c_float),
        ("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("wait_limit", ctypes.c_int),
    ]


class HraPlanParams(ctypes.Structure):
    """Mirror of hra_plan_params (field order and C types as in include/hra.h)."""
    _fields_ = [
        ("batch", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
        ("num_pages", ctypes.c_int), ("max_tokens", ctypes.c_int),
        ("seq_lens", ctypes.c_void_p), ("new_tokens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("free_pages", ctypes.c_void_p), ("free_range", ctypes.c_void_p), ("seq_lens_out", ctypes.c_void_p),
        ("free_range_out", ctypes.c_void_p), ("query_start", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("positions", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


class HraAppendParams(ctypes.Structure):
    """Mirror of hra_append_params (field order and C types as in include/hra.h)."""
    _fields_ = [
        ("n_tokens", ctypes.c_int), ("d_c", ctypes.c_int), ("d_rope", ctypes.c_int),
        ("latent", ctypes.c_void_p), ("krope_in", ctypes.c_void_p),
        ("latent_stride", ctypes.c_int64), ("krope_in_stride", ctypes.c_int64),
        ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rope_theta", ctypes.c_float),
        ("ckv", ctypes.c_void_p), ("krope", ctypes.c_void_p),
        ("ckv_stride", ctypes.c_int64), ("krope_stride", ctypes.c_int64), ("cache_rows", ctypes.c_int64),
        ("cache_dtype", ctypes.c_int), ("ckv_scale", ctypes.c_void_p), ("ckv_scale_stride", ctypes.c_int64),
        ("scale_block", ctypes.c_int), ("rows_out", ctypes.c_void_p), ("rows_out_stride", ctypes.c_int64),
    ]


class HraLoadParams(ctypes.Structure):
    """Mirror of hra_load_params (field order and C types as in include/hra.h)."""
    _fields_ = [
        ("batch", ctypes.c_int), ("max_tokens", ctypes.c_int), ("d_c", ctypes.c_int), ("d_rope", ctypes.c_int),
        ("ckv", ctypes.c_void_p), ("krope", ctypes.c_void_p),
        ("ckv_stride", ctypes.c_int64), ("krope_stride", ctypes.c_int64), ("cache_rows", ctypes.c_int64),
        ("cache_dtype", ctypes.c_int), ("ckv_scale", ctypes.c_void_p), ("ckv_scale_stride", ctypes.c_int64),
        ("scale_block", ctypes.c_int), ("seq_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("seq_stride", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64), ("out_seq_stride", ctypes.c_int64),
    ]


_lib: Optional[ctypes.CDLL] = None


def load_library() -> ctypes.CDLL:
    """Load libhra.so from the package directory (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not LIB_PATH.exists():
        raise ImportError(f"{LIB_PATH} is not built; run `python -m head_rank_attention_b200.build`")
    lib = ctypes.CDLL(str(LIB_PATH))
    lib.hra_version.argtypes = []
    lib.hra_version.restype = ctypes.c_char_p
    built = lib.hra_version().decode()
    if built.split()[1:2] != [HRA_VERSION]:  # it would read other fields than the structs above have
        raise ImportError(f"{LIB_PATH} is {built}, not {HRA_VERSION}; run `python -m head_rank_attention_b200.build`")
    P = ctypes.POINTER(HraDecodeParams)
    lib.hra_workspace_size.argtypes = [P]
    lib.hra_workspace_size.restype = ctypes.c_size_t
    for name in ("mlra_decode", "mla_decode", "mlra_decode_static", "hra_check_device_status"):
        getattr(lib, name).argtypes = [P, ctypes.c_void_p]
        getattr(lib, name).restype = ctypes.c_int
    PP = ctypes.POINTER(HraPrefillParams)
    lib.hra_prefill_workspace_size.argtypes = [PP]
    lib.hra_prefill_workspace_size.restype = ctypes.c_size_t
    for name in ("mlra_prefill", "hra_check_prefill_status"):
        getattr(lib, name).argtypes = [PP, ctypes.c_void_p]
        getattr(lib, name).restype = ctypes.c_int
    for name, cls in (("hra_page_plan", HraPlanParams), ("hra_check_plan_status", HraPlanParams),
                      ("hra_cache_append", HraAppendParams), ("hra_cache_load", HraLoadParams)):
        getattr(lib, name).argtypes = [ctypes.POINTER(cls), ctypes.c_void_p]
        getattr(lib, name).restype = ctypes.c_int
    lib.hra_combine_partials.argtypes = [P, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    lib.hra_combine_partials.restype = ctypes.c_int
    lib.hra_selftest_wait_timeout.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    lib.hra_selftest_wait_timeout.restype = ctypes.c_int
    lib.hra_last_error.argtypes = []
    lib.hra_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def last_error() -> str:
    return load_library().hra_last_error().decode()


def version() -> str:
    return load_library().hra_version().decode()


def _check(status: int) -> None:
    if status != HRA_OK:
        raise HraError(status, last_error())


def _stream_handle(stream) -> int:
    if stream is None:
        # the handle that torch.cuda.current_stream().cuda_stream gives, without its 5 us of
        # Python objects (more than the smallest of these kernels takes)
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return getattr(stream, "cuda_stream", stream)


def _on_one_device(p, tensors) -> None:
    """Remember which device p's tensors are on (they share one)."""
    devices = {t.device for t in tensors if t is not None}
    if len(devices) != 1:
        raise ValueError(f"the tensors lie on several devices: {sorted(map(str, devices))}")
    p._device = devices.pop()
    p._index = p._device.index if p._device.type == "cuda" else None


def _launch(name: str, p, stream) -> None:
    """Call an entry point with p on a stream (the current one by default).  p's tensors must be
    on the current device, which is the one that the kernel runs on."""
    import torch
    if p._index is None:
        raise ValueError(f"the tensors are on {p._device}, not on a CUDA device")
    current = torch._C._cuda_getDevice()  # torch.cuda.current_device() without its check that CUDA is up
    if current != p._index:
        raise ValueError(f"the tensors are on {p._device}, the current device is cuda:{current}")
    handle = torch._C._cuda_getCurrentRawStream(current) if stream is None else getattr(stream, "cuda_stream", stream)
    status = getattr(_lib or load_library(), name)(ctypes.byref(p), handle)
    if status != HRA_OK:
        _check(status)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _cache_format(p, ckv, ckv_scale, scale_block: int, rows: int) -> None:
    """The format of a cache of `rows` rows; kernels read (the append writes) a scale for each
    begun block of them and 128 columns."""
    import torch
    p.cache_dtype = {torch.int8: HRA_INT8, torch.float8_e4m3fn: HRA_E4M3}.get(ckv.dtype, HRA_BF16)
    p.scale_block = int(scale_block)
    if p.cache_dtype == HRA_BF16:
        return
    if ckv_scale is None:
        raise ValueError("an int8 cache needs ckv_scale" if p.cache_dtype == HRA_INT8 else "an e4m3 cache needs ckv_scale")
    block = max(1, int(scale_block))
    need = (-(-rows // block), int(ckv.shape[1]) // 128)
    fits = ckv_scale.dtype == torch.float32 and ckv_scale.dim() in (1, 2) and int(ckv_scale.shape[0]) >= need[0]
    if fits and ckv_scale.dim() == 2:
        fits = int(ckv_scale.shape[1]) >= need[1] and (need[1] == 1 or ckv_scale.stride(1) == 1)
    elif fits:  # a branch's column by itself
        fits = need[1] == 1
    if not fits:
        raise ValueError(f"ckv_scale must be float32 {list(need)} with adjacent columns, one scale per "
                         + (f"block of {block} rows" if block > 1 else "row") + " and 128 columns")
    p.ckv_scale, p.ckv_scale_stride = _ptr(ckv_scale), int(ckv_scale.stride(0))


def make_params(q, ckv, krope, seq_lens, w_uk, w_uv, out, workspace=None, *, n_branch: int,
                alpha_q: float = 1.0, alpha_kv: float = 1.0, branch_scale: Optional[float] = None,
                softmax_scale: float = 0.0, rope_theta: float = 10000.0, block_table=None,
                page_size: int = 0, seq_stride: int = 0, cache_rows: Optional[int] = None,
                num_splits: int = 0, wait_limit: int = 0, out_accumulate: bool = False,
                out_peers=None, ckv_scale=None, q_positions=None, part_o=None,
                part_lse=None, scale_block: int = 0) -> HraDecodeParams:
    """Fill hra_decode_params from torch tensors (shapes/dtypes as documented in hra.h).

    ckv / krope are 2-D row views of the cache (e.g. cache[:, :512], cache[:, 512:]);
    their row strides become ckv_stride / krope_stride.  An int8 ckv selects the quantised
    cache: ckv_scale is then the fp32 [rows, d_c / 128] view of its block scales; with
    scale_block (int8 or float8_e4m3fn) it is [rows / scale_block, d_c / 128].  out_peers: device addresses (ints)
    or tensors of other ranks' out buffers for out_accumulate (the array is kept alive on
    the returned object).  q_positions (int32 [B]), part_o (fp32 [B, h, d_c]) and part_lse
    (fp32 [B, h, d_c / 128]) make the call the decode of one token range of longer
    sequences (see hra.h); out may then be None.
    """
    import torch
    p = HraDecodeParams()
    p.batch, p.num_heads = int(q.shape[0]), int(q.shape[1])
    p.n_branch = int(n_branch)
    p.d_c, p.d_rope, p.d_nope, p.d_v = int(ckv.shape[1]), int(krope.shape[1]), int(q.shape[2]) - int(krope.shape[1]), int(w_uv.shape[2])
    p.q, p.ckv, p.krope = _ptr(q), _ptr(ckv), _ptr(krope)
    p.ckv_stride, p.krope_stride = int(ckv.stride(0)), int(krope.stride(0))
    p.cache_rows = int(ckv.shape[0]) if cache_rows is None else int(cache_rows)
    _cache_format(p, ckv, ckv_scale, scale_block, p.cache_rows)
    p.seq_lens = _ptr(seq_lens)
    p.block_table = _ptr(block_table)
    p.max_pages = int(block_table.shape[1]) if block_table is not None else 0
    p.page_size = int(page_size)
    p.seq_stride = int(seq_stride)
    p.w_uk, p.w_uv = _ptr(w_uk), _ptr(w_uv)
    p.alpha_q, p.alpha_kv = float(alpha_q), float(alpha_kv)
    p.branch_scale = float(1.0 / math.sqrt(n_branch) if branch_scale is None else branch_scale)
    p.softmax_scale, p.rope_theta = float(softmax_scale), float(rope_theta)
    p.out = _ptr(out)
    p.out_dtype = HRA_F32 if out is not None and out.dtype == torch.float32 else HRA_BF16
    p.workspace = _ptr(workspace)
    p.workspace_bytes = 0 if workspace is None else int(workspace.numel() * workspace.element_size())
    p.num_splits, p.wait_limit = int(num_splits), int(wait_limit)
    p.out_accumulate = int(bool(out_accumulate))
    peers = [x if isinstance(x, int) else _ptr(x) for x in (out_peers or [])]
    p._out_peers = (ctypes.c_void_p * max(1, len(peers)))(*peers)
    p.out_peers = ctypes.cast(p._out_peers, ctypes.c_void_p).value if peers else None
    p.n_out_peers = len(peers)
    p.q_positions, p.part_o, p.part_lse = _ptr(q_positions), _ptr(part_o), _ptr(part_lse)
    return p


def workspace_size(p: HraDecodeParams) -> int:
    n = load_library().hra_workspace_size(ctypes.byref(p))
    if n == 0:
        raise HraError(HRA_ERR_INVALID_ARG, last_error())
    return int(n)


def mlra_decode(p: HraDecodeParams, stream=None) -> None:
    _check(load_library().mlra_decode(ctypes.byref(p), ctypes.c_void_p(_stream_handle(stream))))


def mla_decode(p: HraDecodeParams, stream=None) -> None:
    _check(load_library().mla_decode(ctypes.byref(p), ctypes.c_void_p(_stream_handle(stream))))


def mlra_decode_static(p: HraDecodeParams, stream=None) -> None:
    """Decode without a workspace (scratch from the library's 32 MiB static device array):
    for callers that cannot allocate device memory.  p.workspace is ignored."""
    _check(load_library().mlra_decode_static(ctypes.byref(p), ctypes.c_void_p(_stream_handle(stream))))


def combine_partials(p: HraDecodeParams, parts_o, parts_lse, stream=None) -> None:
    """Merge the gathered token-range states parts_o (fp32 [n, B, h, d_c]) and parts_lse
    (fp32 [n, B, h, d_c / 128]) and finish the decode into p.out (hra_combine_partials)."""
    _check(load_library().hra_combine_partials(ctypes.byref(p), int(parts_o.shape[0]), ctypes.c_void_p(_ptr(parts_o)),
                                               ctypes.c_void_p(_ptr(parts_lse)),
                                               ctypes.c_void_p(_stream_handle(stream))))


def check_device_status(p: HraDecodeParams, stream=None) -> None:
    _check(load_library().hra_check_device_status(ctypes.byref(p), ctypes.c_void_p(_stream_handle(stream))))


def selftest_wait_timeout(workspace, limit_us: int, stream=None) -> None:
    _check(load_library().hra_selftest_wait_timeout(ctypes.c_void_p(_ptr(workspace)), int(limit_us),
                                                    ctypes.c_void_p(_stream_handle(stream))))


def alloc_workspace(p: HraDecodeParams, device=None):
    """Allocate a workspace for p with torch (256-byte aligned) and attach it to p."""
    import torch
    n = workspace_size(p)
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    p.workspace, p.workspace_bytes = ws.data_ptr(), n
    return ws


def make_prefill_params(q, ckv, krope, w_uk, w_uv, out, *, n_branch: int, alpha_q: float = 1.0,
                        alpha_kv: float = 1.0, branch_scale: Optional[float] = None, softmax_scale: float = 0.0,
                        rope_theta: float = 10000.0, wait_limit: int = 0) -> HraPrefillParams:
    """Fill hra_prefill_params from torch tensors: q [n, h, 192] bf16, ckv / krope 2-D row
    views of the sequence's L cached rows, out [n, h, 128] (bf16 or fp32)."""
    import torch
    p = HraPrefillParams()
    p.num_heads, p.n_branch = int(q.shape[1]), int(n_branch)
    p.d_c, p.d_rope, p.d_nope, p.d_v = int(ckv.shape[1]), int(krope.shape[1]), int(q.shape[2]) - int(krope.shape[1]), int(w_uv.shape[2])
    p.seq_len, p.n_query = int(ckv.shape[0]), int(q.shape[0])
    p.q, p.ckv, p.krope = _ptr(q), _ptr(ckv), _ptr(krope)
    p.ckv_stride, p.krope_stride = int(ckv.stride(0)), int(krope.stride(0))
    p.w_uk, p.w_uv = _ptr(w_uk), _ptr(w_uv)
    p.alpha_q, p.alpha_kv = float(alpha_q), float(alpha_kv)
    p.branch_scale = float(1.0 / math.sqrt(n_branch) if branch_scale is None else branch_scale)
    p.softmax_scale, p.rope_theta = float(softmax_scale), float(rope_theta)
    p.out = _ptr(out)
    p.out_dtype = HRA_F32 if out is not None and out.dtype == torch.float32 else HRA_BF16
    p.wait_limit = int(wait_limit)
    return p


def prefill_workspace_size(p: HraPrefillParams) -> int:
    n = load_library().hra_prefill_workspace_size(ctypes.byref(p))
    if n == 0:
        raise HraError(HRA_ERR_INVALID_ARG, last_error())
    return int(n)


def alloc_prefill_workspace(p: HraPrefillParams, device=None):
    """Allocate a prefill workspace with torch (256-byte aligned) and attach it to p."""
    import torch
    n = prefill_workspace_size(p)
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    p.workspace, p.workspace_bytes = ws.data_ptr(), n
    return ws


def mlra_prefill(p: HraPrefillParams, stream=None) -> None:
    _check(load_library().mlra_prefill(ctypes.byref(p), ctypes.c_void_p(_stream_handle(stream))))


def check_prefill_status(p: HraPrefillParams, stream=None) -> None:
    _check(load_library().hra_check_prefill_status(ctypes.byref(p), ctypes.c_void_p(_stream_handle(stream))))


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _vector(t, n: Optional[int], dtype, name: str) -> None:
    """t is a contiguous 1-D tensor of dtype with n elements (any number where n is None)."""
    _need(t.dtype == dtype and t.dim() == 1 and t.is_contiguous() and (n is None or int(t.shape[0]) == n),
          f"{name} must be a contiguous {dtype} vector" + ("" if n is None else f" of {n}"))


def make_plan_params(seq_lens, new_tokens, block_table, free_pages, free_range, seq_lens_out, free_range_out,
                     query_start, slots, status, *, positions=None, page_size: int) -> HraPlanParams:
    """Fill hra_plan_params (a step's page plan, see hra.h) from torch tensors: seq_lens,
    new_tokens and seq_lens_out int32 [B], block_table int32 [B, max_pages] contiguous,
    free_pages int32 [num_pages], free_range and free_range_out int64 [2], query_start
    int32 [B + 1], slots (and positions) int32 [max_tokens], status int32 [4].
    seq_lens_out and free_range_out may be seq_lens and free_range."""
    import torch
    B = int(seq_lens.shape[0])
    for t, n, name in ((seq_lens, B, "seq_lens"), (new_tokens, B, "new_tokens"), (seq_lens_out, B, "seq_lens_out"),
                       (free_pages, None, "free_pages"), (query_start, B + 1, "query_start"), (slots, None, "slots"),
                       (status, 4, "status")):
        _vector(t, n, torch.int32, name)
    for t, name in ((free_range, "free_range"), (free_range_out, "free_range_out")):
        _vector(t, 2, torch.int64, name)
    if positions is not None:
        _vector(positions, int(slots.shape[0]), torch.int32, "positions")
    _need(block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.is_contiguous()
          and int(block_table.shape[0]) == B, f"block_table must be contiguous int32 [{B}, max_pages]")
    p = HraPlanParams()
    _on_one_device(p, (seq_lens, new_tokens, block_table, free_pages, free_range, seq_lens_out, free_range_out, query_start,
                       slots, status, positions))
    p.batch, p.page_size, p.max_pages = B, int(page_size), int(block_table.shape[1])
    p.num_pages, p.max_tokens = int(free_pages.shape[0]), int(slots.shape[0])
    p.seq_lens, p.new_tokens, p.block_table = _ptr(seq_lens), _ptr(new_tokens), _ptr(block_table)
    p.free_pages, p.free_range = _ptr(free_pages), _ptr(free_range)
    p.seq_lens_out, p.free_range_out = _ptr(seq_lens_out), _ptr(free_range_out)
    p.query_start, p.slots, p.positions, p.status = _ptr(query_start), _ptr(slots), _ptr(positions), _ptr(status)
    return p


def page_plan(p: HraPlanParams, stream=None) -> None:
    """Plan a step on the device: new block table entries, slots and positions of the new
    tokens, lengths and page pool after the step.  A refused step is seen in p's status
    tensor, or with check_plan_status."""
    _launch("hra_page_plan", p, stream)


def check_plan_status(p: HraPlanParams, stream=None) -> None:
    _launch("hra_check_plan_status", p, stream)


def _rows_2d(t, cols: int, dtype, name: str) -> None:
    _need(t.dim() == 2 and t.dtype == dtype and int(t.shape[1]) == cols and t.stride(1) == 1,
          f"{name} must be {dtype} [rows, {cols}] with adjacent columns")


def _cache_rows(p, ckv, krope, ckv_scale, scale_block: int) -> None:
    import torch
    _need(ckv.dtype in (torch.bfloat16, torch.int8, torch.float8_e4m3fn), f"a cache is bfloat16, int8 or float8_e4m3fn, not {ckv.dtype}")
    _rows_2d(ckv, p.d_c, ckv.dtype, "ckv")
    _rows_2d(krope, 64, torch.bfloat16, "krope")
    _need(int(krope.shape[0]) >= int(ckv.shape[0]), "krope has fewer rows than ckv")
    _cache_format(p, ckv, ckv_scale, scale_block, int(ckv.shape[0]))
    p.ckv, p.krope = _ptr(ckv), _ptr(krope)
    p.ckv_stride, p.krope_stride, p.cache_rows = int(ckv.stride(0)), int(krope.stride(0)), int(ckv.shape[0])


def make_append_params(latent, krope_in, slots, positions, ckv, krope, *, ckv_scale=None, scale_block: int = 0,
                       rows_out=None, rope_theta: float = 10000.0) -> HraAppendParams:
    """Fill hra_append_params (new tokens into the cache, see hra.h) from torch tensors:
    latent bf16 [n, d_c] and krope_in bf16 [n, 64] (views of one projection output will do),
    slots and positions int32 [n] (a page plan's), the cache as make_params takes it, and
    optionally rows_out bf16 [n, d_c + 64] for the rows as the cache stands for them."""
    import torch
    p = HraAppendParams()
    _on_one_device(p, (latent, krope_in, slots, positions, ckv, krope, ckv_scale, rows_out))
    p.n_tokens, p.d_c, p.d_rope = int(latent.shape[0]), int(latent.shape[1]), int(krope_in.shape[1])
    _rows_2d(latent, p.d_c, torch.bfloat16, "latent")
    _rows_2d(krope_in, 64, torch.bfloat16, "krope_in")
    _need(int(krope_in.shape[0]) == p.n_tokens, "latent and krope_in differ in rows")
    _vector(slots, p.n_tokens, torch.int32, "slots")
    _vector(positions, p.n_tokens, torch.int32, "positions")
    _need(int(ckv.shape[1]) == p.d_c, f"ckv has {int(ckv.shape[1])} columns, latent {p.d_c}")
    _cache_rows(p, ckv, krope, ckv_scale, scale_block)
    p.latent, p.krope_in = _ptr(latent), _ptr(krope_in)
    p.latent_stride, p.krope_in_stride = int(latent.stride(0)), int(krope_in.stride(0))
    p.slots, p.positions, p.rope_theta = _ptr(slots), _ptr(positions), float(rope_theta)
    if rows_out is not None:
        _rows_2d(rows_out, p.d_c + 64, torch.bfloat16, "rows_out")
        _need(int(rows_out.shape[0]) == p.n_tokens, "rows_out and latent differ in rows")
        p.rows_out, p.rows_out_stride = _ptr(rows_out), int(rows_out.stride(0))
    return p


def cache_append(p: HraAppendParams, stream=None) -> None:
    """Write new tokens into the cache: latents in the cache's format, RoPE keys turned to
    their positions."""
    _launch("hra_cache_append", p, stream)


def make_load_params(ckv, krope, seq_lens, out, *, block_table=None, page_size: int = 0, seq_stride: int = 0,
                     ckv_scale=None, scale_block: int = 0) -> HraLoadParams:
    """Fill hra_load_params (cached rows back as bf16, see hra.h) from torch tensors: the
    cache as make_params takes it, seq_lens int32 [B] and out bf16 [B, max_tokens, d_c + 64]."""
    import torch
    p = HraLoadParams()
    _on_one_device(p, (ckv, krope, seq_lens, out, block_table, ckv_scale))
    p.batch, p.max_tokens, p.d_c, p.d_rope = int(seq_lens.shape[0]), int(out.shape[1]), int(ckv.shape[1]), 64
    _vector(seq_lens, None, torch.int32, "seq_lens")
    _need(out.dim() == 3 and out.dtype == torch.bfloat16 and out.stride(2) == 1
          and (int(out.shape[0]), int(out.shape[2])) == (p.batch, p.d_c + 64),
          f"out must be bfloat16 [{p.batch}, max_tokens, {p.d_c + 64}] with adjacent columns")
    _cache_rows(p, ckv, krope, ckv_scale, scale_block)
    if block_table is not None:
        _need(block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.is_contiguous()
              and int(block_table.shape[0]) == p.batch, f"block_table must be contiguous int32 [{p.batch}, max_pages]")
        p.max_pages = int(block_table.shape[1])
    p.seq_lens, p.block_table = _ptr(seq_lens), _ptr(block_table)
    p.page_size, p.seq_stride = int(page_size), int(seq_stride)
    p.out, p.out_stride, p.out_seq_stride = _ptr(out), int(out.stride(1)), int(out.stride(0))
    return p


def cache_load(p: HraLoadParams, stream=None) -> None:
    """Read cached rows back as contiguous bf16 rows [C_KV | K_RoPE], the form mlra_prefill
    takes."""
    _launch("hra_cache_load", p, stream)
