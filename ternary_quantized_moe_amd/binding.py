"""ctypes binding of libmoe_ternary.so (argument marshalling only).

Every step of the block runs in the library's HIP kernels; this module only
turns numpy arrays and torch device tensors into the pointers and sizes the C
ABI takes (include/moe_ternary.h), and raises MoeError on a non-zero status.
PyTorch provides device memory and the current stream.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import numpy as np

PQ2_0 = 142
PTQ1_0 = 143

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_ternary.so")

_ERRORS = {
    -1: "MOE_E_ARG", -2: "MOE_E_FORMAT", -3: "MOE_E_SHAPE", -4: "MOE_E_CODE",
    -5: "MOE_E_NONFINITE", -6: "MOE_E_SPACE", -7: "MOE_E_DEVICE",
}

EXPORTS = [
    "moe_block_bytes", "moe_packed_bytes", "moe_pack", "moe_unpack", "moe_unpack_device",
    "moe_quantize_device", "moe_ple_gather_q4_0", "moe_ternary_forward_q", "moe_draft_head_workspace_bytes",
    "moe_draft_head", "moe_lowrank_workspace_bytes", "moe_lowrank_apply",
    "moe_fp8_quantize", "moe_rms_norm", "moe_fp8_linear", "moe_sample_workspace_bytes", "moe_sample",
    "moe_attention_prefill_workspace_bytes", "moe_attention_prefill", "moe_attention_decode_workspace_bytes", "moe_attention_decode", "moe_kv_append",
    "moe_kv_pages_workspace_bytes", "moe_kv_reserve", "moe_kv_fork", "moe_kv_free", "moe_kv_compact",
    "moe_kv_copy_pages",
    "moe_workspace_bytes_factored", "moe_ternary_forward_factored",
    "moe_tile_container", "moe_untile_container", "moe_workspace_bytes", "moe_ternary_forward", "moe_route_workspace_bytes", "moe_route",
    "moe_route_workspace_bytes_factored", "moe_route_factored", "moe_ternary_forward_noalloc",
    "moe_set_stage_events", "moe_last_error",
]
N_STAGES = 5
STAGES = ["xproj", "routing", "gate_up", "down", "combine"]


class MoeError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{_ERRORS.get(code, code)}: {message}")
        self.code = code
        self.name = _ERRORS.get(code, str(code))


class ExpertBanksC(ctypes.Structure):
    _fields_ = [
        ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
        ("n_experts", ctypes.c_int32), ("n_shared", ctypes.c_int32),
        ("banks", ctypes.c_void_p), ("banks_bytes", ctypes.c_int64),
        ("offsets", ctypes.c_void_p), ("formats", ctypes.c_void_p),
        ("offsets_host", ctypes.c_void_p), ("formats_host", ctypes.c_void_p),
        ("layout", ctypes.c_int32),
    ]


class KvPoolC(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("planes", ctypes.c_int64), ("page_bytes", ctypes.c_int64)]


MAX_POOLS = 8
BANKS_ROW_MAJOR, BANKS_TILE_MAJOR = 1, 2


_lib = None


def lib():
    """Load the library; fails loudly if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is missing: run `python -m ternary_quantized_moe_amd.build`")
        L = ctypes.CDLL(_LIB_PATH)
        i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
        sig = {
            "moe_block_bytes": (i64, [i32]),
            "moe_packed_bytes": (i64, [i32, i64]),
            "moe_pack": (i32, [i32, vp, vp, i64, vp, i64]),
            "moe_unpack": (i32, [i32, vp, i64, vp, vp, i64]),
            "moe_unpack_device": (i32, [i32, vp, i64, vp, vp, vp]),
            "moe_quantize_device": (i32, [i32, i32, vp, i64, vp, vp, vp]),
            "moe_ple_gather_q4_0": (i32, [vp, i64, i32, vp, i64, vp, vp]),
            "moe_ternary_forward_q": (i32, [vp, i64, vp, vp, ctypes.POINTER(ExpertBanksC), vp, vp, i32,
                                            i32, vp, vp, i64, vp]),
            "moe_draft_head_workspace_bytes": (i64, [i64, i32, i32]),
            "moe_draft_head": (i32, [vp, vp, i64, i32, i32, vp, vp, vp, vp, vp, vp, i64, vp]),
            "moe_lowrank_workspace_bytes": (i64, [i64, i32, i32]),
            "moe_lowrank_apply": (i32, [vp, vp, i64, i32, vp, vp, vp, vp, i32, vp, vp, i64, vp]),
            "moe_fp8_quantize": (i32, [i32, vp, i64, i32, i32, vp, vp, vp]),
            "moe_rms_norm": (i32, [vp, vp, i64, i32, vp, ctypes.c_float, vp, vp, vp, vp, vp]),
            "moe_fp8_linear": (i32, [vp, vp, i64, vp, vp, i64, i32, i32, vp, i64, vp]),
            "moe_sample_workspace_bytes": (i64, [i64, i32]),
            "moe_sample": (i32, [i32, vp, i64, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp]),
            "moe_attention_prefill_workspace_bytes": (i64, [i64, i64, i64, i32, i32, i32]),
            "moe_attention_prefill": (i32, [i32, vp, i64, i32, i64, i64, vp, vp, i64, i32, i64, i64, i64, i64, i32, vp,
                                            vp, i64, i32, ctypes.c_float, vp, vp, vp, i64, vp]),
            "moe_attention_decode_workspace_bytes": (i64, [i64, i32, i32, i32]),
            "moe_attention_decode": (i32, [i32, vp, i64, i32, i64, i64, i32, vp, vp, vp, vp, i64, i32, i32, i32, vp, i32,
                                           vp, ctypes.c_float, vp, vp, vp, i64, vp]),
            "moe_kv_append": (i32, [i32, vp, i64, i64, i32, vp, i64, i64, vp, i64, i64, i64, i32, vp, vp, vp, vp, i64,
                                    i32, i32, i32, vp, i64, i32, vp, vp, vp, i32, i32, vp, i64, i64, vp, i64, i64,
                                    vp]),
            "moe_kv_pages_workspace_bytes": (i64, [i64, i64]),
            "moe_kv_reserve": (i32, [vp, i64, i32, vp, vp, i64, i32, vp, vp, vp, i64, vp]),
            "moe_kv_fork": (i32, [vp, i64, i32, vp, vp, i64, i32, vp, vp, i32, vp, vp, i64, vp]),
            "moe_kv_free": (i32, [vp, i64, i32, vp, vp, i64, i32, vp, vp]),
            "moe_kv_compact": (i32, [vp, i64, i32, vp, vp, i64, i32, vp, i32, vp, vp, vp, vp, i64, vp]),
            "moe_kv_copy_pages": (i32, [vp, i32, i64, vp, vp, i64, vp]),
            "moe_workspace_bytes_factored": (i64, [ctypes.POINTER(ExpertBanksC), i64, i32, i32, i32]),
            "moe_ternary_forward_factored": (i32, [vp, i64, vp, vp, vp, i32, ctypes.POINTER(ExpertBanksC), vp, vp,
                                                   i32, i32, vp, vp, i64, vp]),
            "moe_tile_container": (i32, [i32, vp, i64, i64, vp, i64]),
            "moe_untile_container": (i32, [i32, vp, i64, i64, vp, i64]),
            "moe_workspace_bytes": (i64, [ctypes.POINTER(ExpertBanksC), i64, i32, i32]),
            "moe_ternary_forward": (i32, [vp, i64, vp, vp, ctypes.POINTER(ExpertBanksC), vp, vp, i32,
                                          i32, vp, vp, i64, vp]),
            "moe_route_workspace_bytes": (i64, [i64, i32, i32, i32]),
            "moe_route": (i32, [vp, i64, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, i64, vp]),
            "moe_route_workspace_bytes_factored": (i64, [i64, i32, i32, i32, i32]),
            "moe_route_factored": (i32, [vp, i64, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, i64,
                                         vp]),
            "moe_ternary_forward_noalloc": (i32, [vp, i64, vp, vp, ctypes.POINTER(ExpertBanksC), vp, vp, i32, i32,
                                                  vp, vp]),
            "moe_set_stage_events": (i32, [ctypes.POINTER(ctypes.c_void_p), i32]),
            "moe_last_error": (ctypes.c_char_p, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc: int):
    if rc != 0:
        raise MoeError(rc, lib().moe_last_error().decode())


def _np_ptr(a: Optional[np.ndarray]):
    return None if a is None else a.ctypes.data


def _dev_ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    """The HIP stream handle: the given torch stream's, else torch's current
    stream on the current device (read through torch's C binding where it has
    one, which costs less per call than building a Stream object)."""
    import torch
    if stream is not None:
        return stream.cuda_stream
    try:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------------ host codec
def block_bytes(fmt: int) -> int:
    return lib().moe_block_bytes(fmt)


def packed_bytes(fmt: int, n_weights: int) -> int:
    return lib().moe_packed_bytes(fmt, n_weights)


def pack(fmt: int, trits: np.ndarray, scale_bits: np.ndarray) -> np.ndarray:
    trits = np.ascontiguousarray(trits, dtype=np.int8).reshape(-1)
    scale_bits = np.ascontiguousarray(scale_bits, dtype=np.uint16).reshape(-1)
    n = trits.size
    nbytes = lib().moe_packed_bytes(fmt, n)
    if nbytes < 0:
        # let the library produce the error message
        _check(lib().moe_pack(fmt, _np_ptr(trits), _np_ptr(scale_bits), n, None, 0))
    if scale_bits.size != n // 128:
        raise MoeError(-1, f"need {n // 128} scales, got {scale_bits.size}")
    out = np.empty(nbytes, dtype=np.uint8)
    _check(lib().moe_pack(fmt, _np_ptr(trits), _np_ptr(scale_bits), n, _np_ptr(out), nbytes))
    return out


def unpack(fmt: int, data: np.ndarray, n_weights: int):
    data = np.ascontiguousarray(data, dtype=np.uint8).reshape(-1)
    trits = np.empty(n_weights, dtype=np.int8)
    scales = np.empty(max(n_weights // 128, 1), dtype=np.uint16)
    _check(lib().moe_unpack(fmt, _np_ptr(data), data.size, _np_ptr(trits), _np_ptr(scales), n_weights))
    return trits, scales[: n_weights // 128]


def tile_container(fmt: int, data: np.ndarray, rows: int, cols: int) -> np.ndarray:
    """Row-major container -> the tile-major block order the expert kernels read."""
    data = np.ascontiguousarray(data, dtype=np.uint8).reshape(-1)
    out = np.empty(data.size, dtype=np.uint8)
    _check(lib().moe_tile_container(fmt, _np_ptr(data), rows, cols, _np_ptr(out), out.size))
    return out


def untile_container(fmt: int, data: np.ndarray, rows: int, cols: int) -> np.ndarray:
    """Inverse of tile_container."""
    data = np.ascontiguousarray(data, dtype=np.uint8).reshape(-1)
    out = np.empty(data.size, dtype=np.uint8)
    _check(lib().moe_untile_container(fmt, _np_ptr(data), rows, cols, _np_ptr(out), out.size))
    return out


# ------------------------------------------------------------------ device
def unpack_device(fmt: int, d_src, n_weights: int, stream=None):
    import torch
    trits = torch.empty(n_weights, dtype=torch.int8, device=d_src.device)
    scales = torch.empty(max(n_weights // 128, 1), dtype=torch.int16, device=d_src.device)
    _check(lib().moe_unpack_device(fmt, _dev_ptr(d_src), n_weights, _dev_ptr(trits), _dev_ptr(scales),
                                   _stream(stream)))
    return trits, scales[: n_weights // 128]


QUANT_ABSMEAN = 0
QUANT_LLOYD = 1


def quantize_device(fmt: int, method: int, d_w, out=None, rounds=None, stream=None):
    """bfloat16 weights (a contiguous device tensor, size a multiple of 128;
    bf16 or int16 bit patterns) -> container bytes (uint8 device tensor).
    rounds: None, or a uint8 device tensor of n/128 entries that receives the
    Lloyd rounds per group."""
    import torch
    n = d_w.numel()
    nbytes = lib().moe_packed_bytes(fmt, n)
    if nbytes < 0:
        _check(lib().moe_quantize_device(fmt, method, None, n, None, None, _stream(stream)))
    if out is None:
        out = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=d_w.device)
    elif out.numel() < nbytes:
        raise MoeError(-6, f"out holds {out.numel()} bytes, {nbytes} needed")
    if rounds is not None and rounds.numel() < n // 128:
        raise MoeError(-6, f"rounds holds {rounds.numel()} entries, {n // 128} needed")
    _check(lib().moe_quantize_device(fmt, method, _dev_ptr(d_w), n, _dev_ptr(out), _dev_ptr(rounds),
                                     _stream(stream)))
    return out[:nbytes]


def ple_gather(d_table, n_rows: int, row_len: int, d_idx, out=None, stream=None):
    """Rows d_idx (int64 device tensor) of a Q4_0 table (uint8 device tensor of
    n_rows rows of row_len values) -> fp32 device tensor [len(d_idx), row_len]."""
    import torch
    n = d_idx.numel()
    if out is None:
        out = torch.empty((n, row_len), dtype=torch.float32, device=d_idx.device)
    elif out.numel() < n * row_len:
        raise MoeError(-6, f"out holds {out.numel()} values, {n * row_len} needed")
    _check(lib().moe_ple_gather_q4_0(_dev_ptr(d_table), n_rows, row_len, _dev_ptr(d_idx), n, _dev_ptr(out),
                                     _stream(stream)))
    return out


class ExpertBanks:
    """One layer's expert containers in device memory plus the host copies the
    library validates against.  `data` is the concatenation of every bank's
    [gate | up | down] containers, each in the tile-major block order of
    tile_container (layers.build_banks writes that order); bank e starts at
    offsets[e]."""

    def __init__(self, data: np.ndarray, offsets: np.ndarray, formats: np.ndarray, d_model: int,
                 d_ff: int, n_experts: int, n_shared: int, device="cuda"):
        import torch
        self.d_model, self.d_ff, self.n_experts, self.n_shared = d_model, d_ff, n_experts, n_shared
        self.offsets_host = np.ascontiguousarray(offsets, dtype=np.int64)
        self.formats_host = np.ascontiguousarray(formats, dtype=np.uint8)
        self.data = torch.from_numpy(np.ascontiguousarray(data, dtype=np.uint8)).to(device)
        self.offsets = torch.from_numpy(self.offsets_host).to(device)
        self.formats = torch.from_numpy(self.formats_host).to(device)
        self.nbytes = int(data.size)
        self._c = ExpertBanksC(d_model, d_ff, n_experts, n_shared, self.data.data_ptr(), self.nbytes,
                               self.offsets.data_ptr(), self.formats.data_ptr(),
                               self.offsets_host.ctypes.data, self.formats_host.ctypes.data, BANKS_TILE_MAJOR)

    @classmethod
    def from_tensors(cls, data_dev, offsets_host, formats_host, d_model, d_ff, n_experts, n_shared):
        """Wrap a device byte tensor that already holds the containers."""
        import torch
        self = cls.__new__(cls)
        self.d_model, self.d_ff, self.n_experts, self.n_shared = d_model, d_ff, n_experts, n_shared
        self.offsets_host = np.ascontiguousarray(offsets_host, dtype=np.int64)
        self.formats_host = np.ascontiguousarray(formats_host, dtype=np.uint8)
        self.data = data_dev
        self.offsets = torch.from_numpy(self.offsets_host).to(data_dev.device)
        self.formats = torch.from_numpy(self.formats_host).to(data_dev.device)
        self.nbytes = int(data_dev.numel())
        self._c = ExpertBanksC(d_model, d_ff, n_experts, n_shared, data_dev.data_ptr(), self.nbytes,
                               self.offsets.data_ptr(), self.formats.data_ptr(),
                               self.offsets_host.ctypes.data, self.formats_host.ctypes.data, BANKS_TILE_MAJOR)
        return self

    @property
    def c(self):
        return ctypes.byref(self._c)


def workspace_bytes(banks: ExpertBanks, n_tokens: int, top_k: int, corr_rank: int) -> int:
    return lib().moe_workspace_bytes(banks.c, n_tokens, top_k, corr_rank)


def alloc_workspace(nbytes: int, device="cuda"):
    import torch
    return torch.empty(max(int(nbytes), 256) + 256, dtype=torch.uint8, device=device)


def _aligned(ws):
    p = ws.data_ptr()
    off = (-p) % 256
    return p + off, ws.numel() - off


def forward(x, router, router_delta, banks: ExpertBanks, corr_a, corr_b, top_k: int, y=None,
            workspace=None, stream=None):
    """x: bf16 [T, d] (torch.bfloat16 or int16 bits) on the GPU; returns y (same dtype as x)."""
    import torch
    T = x.shape[0]
    r = 0 if corr_a is None else corr_a.shape[0]
    if y is None:
        y = torch.empty_like(x)
    if workspace is None:
        need = workspace_bytes(banks, T, top_k, r)
        if need < 0:
            raise MoeError(-1, "invalid arguments for the workspace size")
        workspace = alloc_workspace(need, x.device)
    wp, wn = _aligned(workspace)
    _check(lib().moe_ternary_forward(_dev_ptr(x), T, _dev_ptr(router), _dev_ptr(router_delta), banks.c,
                                     _dev_ptr(corr_a), _dev_ptr(corr_b), r, top_k, _dev_ptr(y), wp, wn,
                                     _stream(stream)))
    return y


NOALLOC_SCRATCH_BYTES = 64 << 20


def forward_noalloc(x, router, router_delta, banks: ExpertBanks, corr_a, corr_b, top_k: int, y, stream=None):
    """forward() with the library's own scratch as workspace (nothing is
    allocated, by the library or here: the caller passes y).  Calls that overlap
    on one GPU share that scratch and race."""
    T = x.shape[0]
    r = 0 if corr_a is None else corr_a.shape[0]
    _check(lib().moe_ternary_forward_noalloc(_dev_ptr(x), T, _dev_ptr(router), _dev_ptr(router_delta), banks.c,
                                             _dev_ptr(corr_a), _dev_ptr(corr_b), r, top_k, _dev_ptr(y),
                                             _stream(stream)))
    return y


def forward_q(x, router, router_delta_q, banks: ExpertBanks, corr_a_q, corr_b_q, corr_rank: int, top_k: int,
              y=None, workspace=None, stream=None):
    """forward() with the router delta and the correction given as ternary PQ2_0
    containers (uint8 device tensors in moe_pack's row-major order, or None)."""
    import torch
    T = x.shape[0]
    r = 0 if corr_a_q is None else corr_rank
    if y is None:
        y = torch.empty_like(x)
    if workspace is None:
        need = workspace_bytes(banks, T, top_k, r)
        if need < 0:
            raise MoeError(-1, "invalid arguments for the workspace size")
        workspace = alloc_workspace(need, x.device)
    wp, wn = _aligned(workspace)
    _check(lib().moe_ternary_forward_q(_dev_ptr(x), T, _dev_ptr(router), _dev_ptr(router_delta_q), banks.c,
                                       _dev_ptr(corr_a_q), _dev_ptr(corr_b_q), r, top_k, _dev_ptr(y), wp, wn,
                                       _stream(stream)))
    return y


def forward_factored(x, router, delta_u, delta_v, banks: ExpertBanks, corr_a, corr_b, top_k: int, y=None,
                     workspace=None, stream=None):
    """forward() with the router delta as fp16 factors U [E, rd] and V [rd, d]."""
    import torch
    T = x.shape[0]
    rd = delta_u.shape[1]
    r = 0 if corr_a is None else corr_a.shape[0]
    if y is None:
        y = torch.empty_like(x)
    if workspace is None:
        need = lib().moe_workspace_bytes_factored(banks.c, T, top_k, r, rd)
        if need < 0:
            raise MoeError(-1, "invalid arguments for the workspace size")
        workspace = alloc_workspace(need, x.device)
    wp, wn = _aligned(workspace)
    _check(lib().moe_ternary_forward_factored(_dev_ptr(x), T, _dev_ptr(router), _dev_ptr(delta_u), _dev_ptr(delta_v),
                                              rd, banks.c, _dev_ptr(corr_a), _dev_ptr(corr_b), r, top_k,
                                              _dev_ptr(y), wp, wn, _stream(stream)))
    return y


def draft_head(hidden, emb, w1, b1, w2, b2, y=None, workspace=None, stream=None):
    """The k=1 draft head: bf16 hidden and emb [T, h] (bf16 or int16 bits),
    fp16 w1 [m, 2h], w2 [h, m], optional fp16 biases -> y [T, h]."""
    T, h = hidden.shape
    m = w1.shape[0]
    if y is None:
        import torch
        y = torch.empty_like(hidden)
    if workspace is None:
        need = lib().moe_draft_head_workspace_bytes(T, h, m)
        if need < 0:
            raise MoeError(-3, f"invalid draft head shape T={T} h={h} m={m}")
        workspace = alloc_workspace(need, hidden.device)
    wp, wn = _aligned(workspace)
    _check(lib().moe_draft_head(_dev_ptr(hidden), _dev_ptr(emb), T, h, m, _dev_ptr(w1), _dev_ptr(b1), _dev_ptr(w2),
                                _dev_ptr(b2), _dev_ptr(y), wp, wn, _stream(stream)))
    return y


def lowrank_apply(x, y_in, a, b, rank: int, a_q=None, b_q=None, y=None, workspace=None, stream=None):
    """y = y_in + B (A x): x, y_in bf16 [T, d] (y_in may be None, y may be y_in);
    A fp16 [r, d] or a_q its PQ2_0 container, B fp16 [d, r] or b_q."""
    import torch
    T, d = x.shape
    if y is None:
        y = torch.empty_like(x)
    if workspace is None:
        need = lib().moe_lowrank_workspace_bytes(T, d, rank)
        if need < 0:
            raise MoeError(-3, f"invalid low-rank shape T={T} d={d} r={rank}")
        workspace = alloc_workspace(need, x.device)
    wp, wn = _aligned(workspace)
    _check(lib().moe_lowrank_apply(_dev_ptr(x), _dev_ptr(y_in), T, d, _dev_ptr(a), _dev_ptr(a_q), _dev_ptr(b),
                                   _dev_ptr(b_q), rank, _dev_ptr(y), wp, wn, _stream(stream)))
    return y


def _wrong(name, t, device, dtypes, shape):
    """The refusal of an operand that _operand found wrong."""
    if t.get_device() != device:
        return MoeError(-1, f"{name} is on {t.device}, not on the current device cuda:{device}")
    if t.dtype not in dtypes:
        return MoeError(-2, f"{name} has type {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        return MoeError(-3, f"{name} has shape {tuple(t.shape)}, {tuple(shape)} wanted")
    return MoeError(-1, f"{name} is not contiguous")


def _operand(name, t, device, dtypes, shape):
    """Pointer of a contiguous tensor of one of these types and this shape on the
    device with this index; anything else is refused.  (One expression on the
    good path: these calls are a few microseconds long.)"""
    if t.get_device() == device and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise _wrong(name, t, device, dtypes, shape)


def _current(t, T):
    """Index of the current device, which has to be the tensor's."""
    d = t.get_device()
    if d < 0:
        raise MoeError(-1, f"a device tensor is wanted, got one on {t.device}")
    now = T["device"]()
    if d != now:
        raise MoeError(-1, f"the tensor is on cuda:{d}, the current device is cuda:{now}")
    return d


def _rows(name, t, dtypes):
    """(pointer, rows, columns, row stride) of a matrix with contiguous rows."""
    if t.dtype not in dtypes:
        raise MoeError(-2, f"{name} has type {t.dtype}")
    if t.dim() != 2:
        raise MoeError(-3, f"{name} has {t.dim()} dimensions, 2 wanted")
    rows, cols = t.shape
    stride, step = t.stride()
    if cols > 1 and step != 1 and rows:
        raise MoeError(-1, f"the rows of {name} are not contiguous")
    return t.data_ptr(), rows, cols, stride if rows > 1 else max(cols, 1)


def _on(stream, device, *made):
    """Handle of a given stream of this device.  What is made for the call goes to no
    other use before the stream is done with it; the caller orders the stream behind
    the work that the current one still has (wait_stream), as for any input."""
    if stream.device.index != device:
        raise MoeError(-1, f"the stream is on {stream.device}, the tensors on cuda:{device}")
    for t in made:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


BF16, F16, F32, E4M3 = 0, 1, 2, 3
_TYPES = {}


def _types():
    """torch types by role, looked up once (torch is imported with the first call)."""
    if not _TYPES:
        import torch
        # the C bindings where torch has them: they cost less per call
        device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _TYPES.update(
            device=device, stream=raw or (lambda d: torch.cuda.current_stream(d).cuda_stream), like=torch.empty_like,
            u8=torch.uint8, f8=torch.float8_e4m3fn, bf16=torch.bfloat16, f32=torch.float32, i32=torch.int32,
            codes=(torch.float8_e4m3fn, torch.uint8), half=(torch.bfloat16, torch.int16), f32s=(torch.float32,),
            i32s=(torch.int32,),
            quant={torch.bfloat16: BF16, torch.int16: BF16, torch.float16: F16},
            out={torch.bfloat16: BF16, torch.float32: F32},
            heads={torch.bfloat16: BF16, torch.float16: F16},
            logits={torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32})
    return _TYPES


def fp8_quantize(x, block_rows: int, q=None, scales=None, stream=None):
    """bf16 (torch.bfloat16 or int16 bits) or fp16 matrix [rows, cols] -> e4m3 codes
    and fp32 scales [ceil(rows / block_rows), cols / 128]: block_rows 1 for
    activations, 128 for weights."""
    T = _types()
    dev = _current(x, T)
    xp, rows, cols, stride = _rows("x", x, T["quant"])
    if stride != cols and rows > 1:
        raise MoeError(-1, "x is not contiguous")
    fn = lib().moe_fp8_quantize
    if block_rows < 1 or cols % 128:
        _check(fn(BF16, None, rows, cols, block_rows, None, None, None))
    size = (-(-rows // block_rows), cols // 128)
    if q is None:
        q = T["like"](x, dtype=T["f8"])
        qp = q.data_ptr()
    else:
        qp = _operand("q", q, dev, T["codes"], (rows, cols))
    if scales is None:
        scales = x.new_empty(size, dtype=T["f32"])
        sp = scales.data_ptr()
    else:
        sp = _operand("scales", scales, dev, T["f32s"], size)
    rc = fn(T["quant"][x.dtype], xp, rows, cols, block_rows, qp, sp,
            T["stream"](dev) if stream is None else _on(stream, dev, q, scales))
    if rc:
        _check(rc)
    return q, scales


def rms_norm(x, weight, eps: float, residual=None, bf16: bool = True, fp8: bool = False, sum=None, y=None, q=None,
             scales=None, stream=None):
    """RMS norm of x (+ residual), bf16 [T, d] (torch.bfloat16 or int16 bits), with
    fp32 weight [d].  Returns a dict: "sum" (x + residual, with a residual only),
    "y" (bf16=True), "q" and "scales" (fp8=True: e4m3 with one scale per 128).
    sum, y, q, scales: buffers for them; sum and y may be x or residual."""
    T = _types()
    dev = _current(x, T)
    half, like = T["half"], T["like"]
    xp, n, d, stride = _rows("x", x, half)
    if stride != d and n > 1:
        raise MoeError(-1, "x is not contiguous")
    wp = _operand("weight", weight, dev, T["f32s"], (d,))
    shape = (n, d)
    rp = sump = yp = qp = sp = None
    out = {}
    if residual is not None:
        rp = _operand("residual", residual, dev, half, shape)
        if sum is None:
            sum = like(x)
            sump = sum.data_ptr()
        else:
            sump = _operand("sum", sum, dev, half, shape)
        out["sum"] = sum
    elif sum is not None:
        raise MoeError(-1, "sum needs a residual")
    if bf16:
        if y is None:
            y = like(x)
            yp = y.data_ptr()
        else:
            yp = _operand("y", y, dev, half, shape)
        out["y"] = y
    elif y is not None:
        raise MoeError(-1, "y is given, but bf16 is off")
    if fp8:
        if q is None:
            q = like(x, dtype=T["f8"])
            qp = q.data_ptr()
        else:
            qp = _operand("q", q, dev, T["codes"], shape)
        if scales is None:
            scales = x.new_empty((n, d // 128), dtype=T["f32"])
            sp = scales.data_ptr()
        else:
            sp = _operand("scales", scales, dev, T["f32s"], (n, d // 128))
        out["q"] = q
        out["scales"] = scales
    elif q is not None or scales is not None:
        raise MoeError(-1, "q or scales is given, but fp8 is off")
    rc = lib().moe_rms_norm(xp, rp, n, d, wp, eps, sump, yp, qp, sp,
                            T["stream"](dev) if stream is None else _on(stream, dev, *out.values()))
    if rc:
        _check(rc)
    return out


def fp8_linear(a, a_scales, w, w_scales, y=None, out_dtype=None, stream=None):
    """a [m, K] times w [n, K] transposed, both e4m3 (torch.float8_e4m3fn or uint8
    codes) with the scales of fp8_quantize (block_rows 1 and 128) -> y [m, n],
    torch.bfloat16 (default) or torch.float32.  A given y may be padded: its rows
    are contiguous and its row stride is at least n.  For bfloat16 the matrix cores
    cut eight neighbouring products at 2^-13 of the largest of them before they add
    them; for float32 products are exact and sums fp32, at half the matrix rate."""
    T = _types()
    dev = _current(a, T)
    ap, m, K, stride = _rows("a", a, T["codes"])
    if stride != K and m > 1:
        raise MoeError(-1, "a is not contiguous")
    n = w.shape[0] if w.dim() == 2 else -1
    wp = _operand("w", w, dev, T["codes"], (n, K))
    asp = _operand("a_scales", a_scales, dev, T["f32s"], (m, K // 128))
    wsp = _operand("w_scales", w_scales, dev, T["f32s"], (-(-n // 128), K // 128))
    if y is None:
        y = a_scales.new_empty((m, n), dtype=out_dtype or T["bf16"])
    elif y.get_device() != dev:
        raise _wrong("y", y, dev, T["out"], (m, n))
    elif out_dtype is not None and out_dtype != y.dtype:
        raise MoeError(-2, f"y has type {y.dtype}, {out_dtype} wanted")
    yp, ym, yn, ldy = _rows("y", y, T["out"])
    if ym != m or yn != n:
        raise MoeError(-3, f"y has shape {(ym, yn)}, {(m, n)} wanted")
    rc = lib().moe_fp8_linear(ap, asp, m, wp, wsp, n, K, T["out"][y.dtype], yp, ldy,
                              T["stream"](dev) if stream is None else _on(stream, dev, y))
    if rc:
        _check(rc)
    return y


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, probs=None, workspace=None,
           stream=None):
    """One token per row of logits [batch, vocab] (fp32, bf16 or fp16; rows may be
    padded) from uniform numbers u [batch]; temperature, top_p, min_p: fp32 [batch]
    or None, top_k: int32 [batch] or None.  Returns (tokens int32, probs fp32)."""
    T = _types()
    dev = _current(logits, T)
    lp, B, V, ld = _rows("logits", logits, T["logits"])
    f32s, size = T["f32s"], (B,)
    up = _operand("u", u, dev, f32s, size)
    tp = None if temperature is None else _operand("temperature", temperature, dev, f32s, size)
    kp = None if top_k is None else _operand("top_k", top_k, dev, T["i32s"], size)
    pp = None if top_p is None else _operand("top_p", top_p, dev, f32s, size)
    mp = None if min_p is None else _operand("min_p", min_p, dev, f32s, size)
    if tokens is None:
        tokens = logits.new_empty(size, dtype=T["i32"])
    if probs is None:
        probs = T["like"](u)
    tokp = _operand("tokens", tokens, dev, T["i32s"], size)
    prp = _operand("probs", probs, dev, f32s, size)
    L = lib()
    if workspace is None:
        need = L.moe_sample_workspace_bytes(B, V)
        if need < 0:
            raise MoeError(-3, f"invalid sampler shape batch={B} vocab={V}")
        workspace = logits.new_empty(need + 256, dtype=T["u8"])
    elif workspace.get_device() != dev:
        raise MoeError(-1, f"the workspace is on {workspace.device}, not on the current device cuda:{dev}")
    ws, wn = _aligned(workspace)
    rc = L.moe_sample(T["logits"][logits.dtype], lp, B, V, ld, tp, kp, pp, mp, up, tokp, prp, ws, wn,
                      T["stream"](dev) if stream is None else _on(stream, dev, tokens, probs, workspace))
    if rc:
        _check(rc)
    return tokens, probs


def _wrong_heads(name, t, device, dtype, shape):
    """The refusal of a matrix of heads that _heads found wrong."""
    if t.get_device() != device:
        return MoeError(-1, f"{name} is on {t.device}, not on the current device cuda:{device}")
    if t.dtype != dtype:
        return MoeError(-2, f"{name} has type {t.dtype}, {dtype} wanted")
    if t.dim() != 3 or any(x is not None and x != n for x, n in zip(shape, t.shape)):
        want = tuple("any" if x is None else x for x in shape)
        return MoeError(-3, f"{name} has shape {tuple(t.shape)}, {want} wanted")
    return MoeError(-1, f"the heads of {name} are not contiguous")


def _heads(name, t, device, dtype, tokens=None, heads=None, dim=None):
    """(pointer, token stride, head stride, tokens, heads, dim) of [tokens, heads, dim] with
    contiguous heads.  (The good path is kept short: these calls are a few microseconds long.)"""
    if t.dtype == dtype and t.dim() == 3 and t.get_device() == device:
        n, h, d = t.shape
        token, head, step = t.stride()
        if (step == 1 or d < 2 or not n or not h) and (heads is None or h == heads) and (dim is None or d == dim) and (
                tokens is None or n == tokens):
            return t.data_ptr(), token if n > 1 else h * d, head if h > 1 else d, n, h, d
    raise _wrong_heads(name, t, device, dtype, (tokens, heads, dim))


def _cache(k, v, k_scales, v_scales, device, dtype, T):
    """(cache type, k, v, k_scales, v_scales, n_pages, kv_heads, page_size, dim) of a layer's cache."""
    shape, kind = k.shape, k.dtype
    if len(shape) != 4:
        raise MoeError(-3, f"k_cache has {len(shape)} dimensions, 4 wanted")
    if kind == dtype:
        if k_scales is not None or v_scales is not None:
            raise MoeError(-1, "k_scales and v_scales go with e4m3 caches only")
        kinds = (dtype,)
        return (T["heads"][dtype], _operand("k_cache", k, device, kinds, shape), _operand("v_cache", v, device, kinds, shape),
                None, None, *shape)
    kinds = T["codes"]
    if kind in kinds and (k_scales is None or v_scales is None):
        raise MoeError(-1, "an e4m3 cache needs k_scales and v_scales")
    kp, vp = _operand("k_cache", k, device, kinds, shape), _operand("v_cache", v, device, kinds, shape)
    rows, f32s = shape[:3], T["f32s"]
    return (E4M3, kp, vp, _operand("k_scales", k_scales, device, f32s, rows), _operand("v_scales", v_scales, device, f32s, rows),
            *shape)


def _scale(dim, scale):
    """The scale of the scores; heads without channels, which the call refuses, have none."""
    return scale if scale is not None else dim ** -0.5 if dim else 1.0


def attention_prefill(q, k, v, starts, k_starts=None, causal: bool = True, scale: Optional[float] = None, y=None,
                      lse=None, workspace=None, stream=None):
    """Attention of packed sequences: q [tokens, heads, dim], k and v [k tokens, kv heads,
    dim], bf16 or fp16, dim 64, 128 or 256; heads are contiguous, tokens and heads may be
    strided (parts of one projection's rows).  starts int32 [sequences + 1]: where each
    sequence's queries begin; k_starts likewise for its keys (None: starts).  causal: query
    i of lq sees the keys up to i + lk - lq of lk.  scale None: dim ** -0.5.  lse: an fp32
    buffer [tokens, heads] for the logarithms of the softmax sums.  -> y [tokens, heads,
    dim]; tokens outside every sequence are not written."""
    T = _types()
    dev = _current(q, T)
    kind = T["heads"].get(q.dtype)
    if kind is None:
        raise MoeError(-2, f"q has type {q.dtype}")
    dtype = q.dtype
    qp, q_token, q_head, n, H, D = _heads("q", q, dev, dtype)
    kp, k_token, k_head, m, Hk, _ = _heads("k", k, dev, dtype, None, None, D)
    vp, v_token, v_head, _, _, _ = _heads("v", v, dev, dtype, m, Hk, D)
    size, i32s = starts.shape, T["i32s"]
    if len(size) != 1 or size[0] < 1:
        raise MoeError(-3, f"starts has shape {tuple(size)}, one more than the sequences wanted")
    sp = _operand("starts", starts, dev, i32s, size)
    ksp = None if k_starts is None else _operand("k_starts", k_starts, dev, i32s, size)
    if y is None:
        y = q.new_empty((n, H, D))
        yp = y.data_ptr()
    else:
        yp = _operand("y", y, dev, (q.dtype,), (n, H, D))
    lp = None if lse is None else _operand("lse", lse, dev, T["f32s"], (n, H))
    L = lib()
    ws, wn = None, 0
    if workspace is None:
        need = L.moe_attention_prefill_workspace_bytes(n, m, size[0] - 1, H, Hk, D)
        if need > 0:
            workspace = q.new_empty(need + 256, dtype=T["u8"])
    elif workspace.get_device() != dev:
        raise MoeError(-1, f"the workspace is on {workspace.device}, not on the current device cuda:{dev}")
    if workspace is not None:
        ws, wn = _aligned(workspace)
    rc = L.moe_attention_prefill(kind, qp, n, H, q_token, q_head, kp, vp, m, Hk, k_token, k_head, v_token, v_head, D, sp,
                                 ksp, size[0] - 1, causal, _scale(D, scale), yp, lp, ws, wn,
                                 T["stream"](dev) if stream is None else _on(stream, dev, y, workspace))
    if rc:
        _check(rc)
    return y


def attention_decode(q, k_cache, v_cache, tables, lengths, k_scales=None, v_scales=None, scale: Optional[float] = None,
                     y=None, lse=None, workspace=None, stream=None):
    """Attention of one new token of every sequence over its cached ones: q [batch, heads,
    dim] (strided as attention_prefill's), a layer's cache k_cache, v_cache [pages, kv heads,
    page, dim] of q's type or e4m3 with fp32 scales [pages, kv heads, page], tables int32
    [batch, width] of page numbers, lengths int32 [batch] (the new token included).
    -> y [batch, heads, dim]."""
    T = _types()
    dev = _current(q, T)
    kind = T["heads"].get(q.dtype)
    if kind is None:
        raise MoeError(-2, f"q has type {q.dtype}")
    dtype, i32s = q.dtype, T["i32s"]
    qp, q_row, q_head, B, H, D = _heads("q", q, dev, dtype)
    ck, kp, vp, ksp, vsp, pages, Hk, P, cd = _cache(k_cache, v_cache, k_scales, v_scales, dev, dtype, T)
    if cd != D:
        raise MoeError(-3, f"the cache has dim {cd}, q has {D}")
    width = tables.shape[1] if tables.dim() == 2 else -1
    tp = _operand("tables", tables, dev, i32s, (B, width))
    lenp = _operand("lengths", lengths, dev, i32s, (B,))
    if y is None:
        y = q.new_empty((B, H, D))
        yp = y.data_ptr()
    else:
        yp = _operand("y", y, dev, (q.dtype,), (B, H, D))
    lp = None if lse is None else _operand("lse", lse, dev, T["f32s"], (B, H))
    L = lib()
    if workspace is None:
        need = L.moe_attention_decode_workspace_bytes(B, H, Hk, D)
        if need < 0:
            raise MoeError(-3, f"invalid attention shape batch={B} heads={H} kv_heads={Hk} dim={D}")
        workspace = q.new_empty(need + 256, dtype=T["u8"])
    elif workspace.get_device() != dev:
        raise MoeError(-1, f"the workspace is on {workspace.device}, not on the current device cuda:{dev}")
    ws, wn = _aligned(workspace)
    rc = L.moe_attention_decode(kind, qp, B, H, q_row, q_head, ck, kp, vp, ksp, vsp, pages, Hk, P, D, tp, width, lenp,
                                _scale(D, scale), yp, lp, ws, wn,
                                T["stream"](dev) if stream is None else _on(stream, dev, y, workspace))
    if rc:
        _check(rc)
    return y


def kv_append(k, v, k_cache, v_cache, tables, rows, positions, k_scales=None, v_scales=None, q=None, inv_freq=None,
              interleaved: bool = False, rotated_k: bool = False, q_out=None, k_out=None, stream=None):
    """New keys and values k, v [tokens, kv heads, dim] (strided as attention_prefill's) into
    the pages of a layer's cache (attention_decode's), token t at place positions[t] of row
    rows[t] of tables (int32; a row below 0 is padding and left alone).  With inv_freq (fp32
    [n]) the first 2 n channels of every head of k, and of q [tokens, heads, dim] if given, are
    turned by positions * inv_freq first: channels i and i + n, or 2 i and 2 i + 1
    (interleaved).  Returns a dict: "q" (turned q; with q) and "k" (turned k; rotated_k=True or
    a k_out).  q_out, k_out: buffers for them, which may be q and k themselves."""
    T = _types()
    dev = _current(k, T)
    kind = T["heads"].get(k.dtype)
    if kind is None:
        raise MoeError(-2, f"k has type {k.dtype}")
    dtype, i32s = k.dtype, T["i32s"]
    kp, k_token, k_head, n, Hk, D = _heads("k", k, dev, dtype)
    vp, v_token, v_head, _, _, _ = _heads("v", v, dev, dtype, n, Hk, D)
    ck, kcp, vcp, ksp, vsp, pages, ch, P, cd = _cache(k_cache, v_cache, k_scales, v_scales, dev, dtype, T)
    if ch != Hk or cd != D:
        raise MoeError(-3, f"the cache has {ch} heads of {cd}, k has {Hk} of {D}")
    if tables.dim() != 2:
        raise MoeError(-3, f"tables has {tables.dim()} dimensions, 2 wanted")
    tp = _operand("tables", tables, dev, i32s, tables.shape)
    R, width = tables.shape
    rp = _operand("rows", rows, dev, i32s, (n,))
    pp = _operand("positions", positions, dev, i32s, (n,))
    out = {}
    fp = qp = qop = kop = None
    H = rotary = q_token = q_head = qo_token = qo_head = ko_token = ko_head = 0
    if inv_freq is not None:
        half = inv_freq.numel()
        rotary = 2 * half
        fp = _operand("inv_freq", inv_freq, dev, T["f32s"], (half,))
    if q is not None:
        qp, q_token, q_head, _, H, _ = _heads("q", q, dev, dtype, n, None, D)
        if q_out is None:
            q_out = q.new_empty((n, H, D))
            qop, qo_token, qo_head = q_out.data_ptr(), H * D, D
        else:
            qop, qo_token, qo_head, _, _, _ = _heads("q_out", q_out, dev, dtype, n, H, D)
        out["q"] = q_out
    elif q_out is not None:
        raise MoeError(-1, "q_out needs a q")
    if k_out is not None:
        kop, ko_token, ko_head, _, _, _ = _heads("k_out", k_out, dev, dtype, n, Hk, D)
        out["k"] = k_out
    elif rotated_k:
        k_out = out["k"] = k.new_empty((n, Hk, D))
        kop, ko_token, ko_head = k_out.data_ptr(), Hk * D, D
    rc = lib().moe_kv_append(kind, qp, q_token, q_head, H, kp, k_token, k_head, vp, v_token, v_head, n, ck, kcp, vcp, ksp,
                             vsp, pages, Hk, P, D, tp, R, width, rp, pp, fp, rotary, interleaved,
                             qop, qo_token, qo_head, kop, ko_token, ko_head,
                             T["stream"](dev) if stream is None else _on(stream, dev, *out.values()))
    if rc:
        _check(rc)
    return out


def _pools(pools, device, n_pages):
    """(moe_kv_pool array, count) of cache tensors [layers, pages, ...] or a list of them."""
    c = (KvPoolC * MAX_POOLS)()
    if len(pools) > MAX_POOLS:
        raise MoeError(-1, f"{len(pools)} pools, at most {MAX_POOLS} wanted")
    for i, p in enumerate(pools):
        if p.get_device() != device:
            raise MoeError(-1, f"pool {i} is on {p.device}, not on the current device cuda:{device}")
        if p.dim() < 3 or p.shape[1] != n_pages:
            raise MoeError(-3, f"pool {i} has shape {tuple(p.shape)}, (layers, {n_pages}, ...) wanted")
        if not p.is_contiguous():
            raise MoeError(-1, f"pool {i} is not contiguous")
        c[i].base, c[i].planes = p.data_ptr(), p.shape[0]
        # (not the stride of the pages, which means nothing where there is one page)
        c[i].page_bytes = math.prod(p.shape[2:]) * p.element_size()
    return c, len(pools)


def _pages(tables, lengths, refs, T):
    """(device, leading arguments) of a call on the pages of a cache."""
    dev = _current(tables, T)
    if tables.dim() != 2 or refs.dim() != 1:
        raise MoeError(-3, f"tables has {tables.dim()} dimensions and refs {refs.dim()}, 2 and 1 wanted")
    R, W = tables.shape
    n = refs.shape[0]
    i32s = T["i32s"]
    return dev, R, n, (_operand("tables", tables, dev, i32s, (R, W)), R, W, _operand("lengths", lengths, dev, i32s, (R,)),
                       _operand("refs", refs, dev, i32s, (n,)), n)


def _pages_space(workspace, like, R, n, T):
    if workspace is None:
        need = lib().moe_kv_pages_workspace_bytes(R, n)
        if need < 0:
            raise MoeError(-3, f"invalid cache shape rows={R} pages={n}")
        workspace = like.new_empty(need + 256, dtype=T["u8"])
    elif workspace.get_device() != like.get_device():
        raise MoeError(-1, f"the workspace is on {workspace.device}, not on {like.device}")
    return (workspace, *_aligned(workspace))


def _status(status, like, dev, R, T):
    if status is None:
        status = T["like"](like)
        return status, status.data_ptr()
    return status, _operand("status", status, dev, T["i32s"], (R,))


def kv_reserve(tables, lengths, refs, grow, page_size: int, status=None, workspace=None, stream=None):
    """Room for grow[r] more tokens in row r of tables (int32 [rows, width]): new pages, the
    lowest free ones, where the row's last does not hold them, and lengths[r] += grow[r].
    refs int32 [pages] counts the rows that hold a page.  -> status int32 [rows]: new pages, -1
    for a negative grow or a table too narrow, -2 where the free pages did not reach."""
    T = _types()
    dev, R, n, head = _pages(tables, lengths, refs, T)
    gp = _operand("grow", grow, dev, T["i32s"], (R,))
    status, sp = _status(status, lengths, dev, R, T)
    workspace, ws, wn = _pages_space(workspace, tables, R, n, T)
    rc = lib().moe_kv_reserve(*head, page_size, gp, sp, ws, wn,
                              T["stream"](dev) if stream is None else _on(stream, dev, status, workspace))
    if rc:
        _check(rc)
    return status


def kv_fork(tables, lengths, refs, parents, page_size: int, pools, status=None, workspace=None, stream=None):
    """Every row r with parents[r] >= 0 (int32 [rows]), which has to be empty, becomes a copy of
    that row: full pages are shared, a partly filled last one is copied in every pool
    (cache tensors [layers, pages, ...]).  -> status int32 [rows]: new pages (0 or 1), -1 for a
    row or parent that does not do, -2 where the free pages did not reach."""
    T = _types()
    dev, R, n, head = _pages(tables, lengths, refs, T)
    pp = _operand("parents", parents, dev, T["i32s"], (R,))
    status, sp = _status(status, lengths, dev, R, T)
    c, count = _pools(pools, dev, n)
    workspace, ws, wn = _pages_space(workspace, tables, R, n, T)
    rc = lib().moe_kv_fork(*head, page_size, pp, c, count, sp, ws, wn,
                           T["stream"](dev) if stream is None else _on(stream, dev, status, workspace))
    if rc:
        _check(rc)
    return status


def kv_free(tables, lengths, refs, drop, page_size: int, stream=None):
    """The rows with drop[r] != 0 (int32 [rows]) give their pages back and get length 0."""
    T = _types()
    dev, R, n, head = _pages(tables, lengths, refs, T)
    dp = _operand("drop", drop, dev, T["i32s"], (R,))
    rc = lib().moe_kv_free(*head, page_size, dp, T["stream"](dev) if stream is None else _on(stream, dev))
    if rc:
        _check(rc)


def kv_compact(tables, lengths, refs, page_size: int, pools, new_tables=None, new_refs=None, live=None, workspace=None,
               stream=None):
    """The n pages in use become pages 0 .. n - 1 of every pool (cache tensors [layers, pages,
    ...]); those above move to the free ones below.  -> (new_tables, new_refs, live), live
    int32 [1] = n; new_tables and new_refs may be tables and refs themselves.  Without rows the
    pages in use move all the same."""
    T = _types()
    dev, R, n, head = _pages(tables, lengths, refs, T)
    if new_tables is None:
        new_tables = T["like"](tables)
    if new_refs is None:
        new_refs = T["like"](refs)
    if live is None:
        live = refs.new_empty((1,))
    tp = _operand("new_tables", new_tables, dev, T["i32s"], tables.shape)
    rp = _operand("new_refs", new_refs, dev, T["i32s"], (n,))
    lp = _operand("live", live, dev, T["i32s"], (1,))
    c, count = _pools(pools, dev, n)
    row = None
    if R == 0:  # without rows the call does nothing: one whose content does not matter stands in
        W = tables.shape[1]
        row = refs.new_empty((W + 1,))
        tp = row.data_ptr()
        head = (tp, 1, W, tp + 4 * W, *head[4:])
    workspace, ws, wn = _pages_space(workspace, tables, max(R, 1), n, T)
    rc = lib().moe_kv_compact(*head, page_size, c, count, tp, rp, lp, ws, wn,
                              T["stream"](dev) if stream is None else _on(stream, dev, new_tables, new_refs, live,
                                                                          workspace, row))
    if rc:
        _check(rc)
    return new_tables, new_refs, live


def kv_copy_pages(pools, src, dst, stream=None):
    """Page dst[i] becomes a copy of page src[i] (int32) in every pool [layers, pages, ...]."""
    T = _types()
    dev = _current(src, T)
    size = src.shape
    if len(size) != 1:
        raise MoeError(-3, f"src has shape {tuple(size)}, one dimension wanted")
    sp, dp = _operand("src", src, dev, T["i32s"], size), _operand("dst", dst, dev, T["i32s"], size)
    if not pools:
        return
    n = pools[0].shape[1] if pools[0].dim() > 1 else 0
    c, count = _pools(pools, dev, n)
    rc = lib().moe_kv_copy_pages(c, count, n, sp, dp, size[0],
                                 T["stream"](dev) if stream is None else _on(stream, dev))
    if rc:
        _check(rc)


def _route_outputs(T, n_experts, top_k, dev):
    import torch
    return dict(
        logits=torch.empty((T, n_experts), dtype=torch.float32, device=dev),
        idx=torch.empty((T, top_k), dtype=torch.int32, device=dev),
        w=torch.empty((T, top_k), dtype=torch.float32, device=dev),
        counts=torch.empty(n_experts, dtype=torch.int32, device=dev),
        offsets=torch.empty(n_experts + 1, dtype=torch.int32, device=dev),
        perm=torch.empty(max(T * top_k, 1), dtype=torch.int32, device=dev),
    )


def route_factored(x, router, delta_u, delta_v, n_experts: int, top_k: int, workspace=None, stream=None):
    """Routing half of forward_factored (router delta as fp16 factors U [E, rd],
    V [rd, d]); returns the same dict as route()."""
    T, d = x.shape
    rd = delta_u.shape[1]
    out = _route_outputs(T, n_experts, top_k, x.device)
    if workspace is None:
        need = lib().moe_route_workspace_bytes_factored(T, d, n_experts, top_k, rd)
        if need < 0:
            raise MoeError(-1, "invalid arguments for the routing workspace size")
        workspace = alloc_workspace(need, x.device)
    wp, wn = _aligned(workspace)
    _check(lib().moe_route_factored(_dev_ptr(x), T, d, n_experts, _dev_ptr(router), _dev_ptr(delta_u),
                                    _dev_ptr(delta_v), rd, top_k, _dev_ptr(out["logits"]), _dev_ptr(out["idx"]),
                                    _dev_ptr(out["w"]), _dev_ptr(out["counts"]), _dev_ptr(out["offsets"]),
                                    _dev_ptr(out["perm"]), wp, wn, _stream(stream)))
    out["perm"] = out["perm"][: T * top_k]
    return out


def route(x, router, router_delta, n_experts: int, top_k: int, workspace=None, stream=None):
    """Routing half of the block; returns dict of device tensors
    (logits, idx, w, counts, offsets, perm)."""
    import torch
    T, d = x.shape
    dev = x.device
    out = dict(
        logits=torch.empty((T, n_experts), dtype=torch.float32, device=dev),
        idx=torch.empty((T, top_k), dtype=torch.int32, device=dev),
        w=torch.empty((T, top_k), dtype=torch.float32, device=dev),
        counts=torch.empty(n_experts, dtype=torch.int32, device=dev),
        offsets=torch.empty(n_experts + 1, dtype=torch.int32, device=dev),
        perm=torch.empty(max(T * top_k, 1), dtype=torch.int32, device=dev),
    )
    if workspace is None:
        need = lib().moe_route_workspace_bytes(T, d, n_experts, top_k)
        if need < 0:
            raise MoeError(-1, "invalid arguments for the routing workspace size")
        workspace = alloc_workspace(need, dev)
    wp, wn = _aligned(workspace)
    _check(lib().moe_route(_dev_ptr(x), T, d, n_experts, _dev_ptr(router), _dev_ptr(router_delta), top_k,
                           _dev_ptr(out["logits"]), _dev_ptr(out["idx"]), _dev_ptr(out["w"]),
                           _dev_ptr(out["counts"]), _dev_ptr(out["offsets"]), _dev_ptr(out["perm"]),
                           wp, wn, _stream(stream)))
    out["perm"] = out["perm"][: T * top_k]
    return out


class StageTimer:
    """Per-stage device time of forward calls, from the library's stage events.

    Create once, then `with timer.step():` around each forward call; events are
    recorded on the call's stream.  `ms()` synchronises and returns the mean
    duration per stage over the recorded steps."""

    def __init__(self, n_steps: int, stages=None):
        """stages: indices of the stages to time (default: all); the others
        record nothing, which keeps the timed stream free of extra markers."""
        import torch
        self.stages = list(range(N_STAGES)) if stages is None else list(stages)
        self._ev = [[torch.cuda.Event(enable_timing=True) if (i // 2) in self.stages else None
                     for i in range(2 * N_STAGES)] for _ in range(n_steps)]
        for evs in self._ev:          # torch creates the HIP event on first record
            for e in evs:
                if e is not None:
                    e.record()
        torch.cuda.synchronize()
        self._arr = [(ctypes.c_void_p * (2 * N_STAGES))(*[e.cuda_event if e is not None else None for e in evs])
                     for evs in self._ev]
        self._i = 0

    def step(self):
        timer = self

        class _Ctx:
            def __enter__(self_inner):
                _check(lib().moe_set_stage_events(timer._arr[timer._i], 2 * N_STAGES))

            def __exit__(self_inner, *exc):
                _check(lib().moe_set_stage_events(None, 0))
                timer._i += 1
        return _Ctx()

    def ms(self):
        import torch
        torch.cuda.synchronize()
        out = np.full(N_STAGES, np.nan)
        for s in self.stages:
            out[s] = sum(evs[2 * s].elapsed_time(evs[2 * s + 1]) for evs in self._ev[: self._i])
        return out / max(self._i, 1)
