"""Python binding of libr9k.so: block-scaled fp8 GEMMs on one MI355X (gfx950).

Argument marshalling only.  Every step of the path runs in the HIP kernels of
libr9k.so; this module takes torch tensors (device memory and streams are all
torch provides here), checks dtypes, allocates outputs and workspaces with
torch when the caller does not pass them, and calls the C ABI declared in
include/r9k.h under the same names.  There is no fallback: if the library is
not built, or a call returns an error, an exception is raised.

Tensor conventions (all contiguous, on the current CUDA/HIP device):
  bf16 values      torch.bfloat16 (or int16/uint16 holding the bits)
  fp8 e4m3 codes   torch.uint8 (or torch.float8_e4m3fn)
  scales, weights  torch.float32;  expert ids torch.int32
  4-bit weights    torch.uint8, two codes to a byte; their scales torch.bfloat16
                   (int4) or torch.uint8 (mxfp4), their zero points torch.uint8
  8-bit integers   torch.int8; a float32 scale per row (token or output channel)
"""
from __future__ import annotations

import ctypes
import functools
import os
from ctypes import POINTER, c_char_p, c_int, c_int64, c_size_t, c_void_p

import torch

ABI_VERSION = 12
ENGINE_AUTO, ENGINE_SKINNY, ENGINE_TILED, ENGINE_SPLITK = 0, 1, 2, 3
TILE_AUTO, TILE_256X256, TILE_256X128, TILE_128X64, TILE_256X64 = 0, 1, 2, 3, 4

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libr9k.so")
_lib = None


class R9kError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: r9k error {code} ({strerror(code)})")


def lib() -> ctypes.CDLL:
    """Load libr9k.so (once).  Raises if it is missing or its ABI differs."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run `python -m block_scaled_fp8_r9k_amd.build` "
                              "(or __graft_entry__.build()) first")
        L = ctypes.CDLL(LIB_PATH)
        L.r9k_abi_version.restype = c_int
        L.r9k_strerror.argtypes = [c_int]
        L.r9k_strerror.restype = c_char_p
        L.r9k_quant_act.argtypes = [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_void_p]
        L.r9k_quant_weight.argtypes = [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_void_p]
        L.r9k_encode_e4m3.argtypes = [c_void_p, c_int64, c_void_p, c_void_p]
        L.r9k_gemm_fp8_block_workspace.argtypes = [c_int64, c_int64, c_int64, POINTER(c_size_t)]
        L.r9k_gemm_fp8_block.argtypes = [c_void_p, c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_int64,
                                         c_void_p, c_void_p, c_size_t, c_void_p]
        L.r9k_gemm_fp8_block_qa.argtypes = [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_int64, c_void_p,
                                            c_void_p, c_size_t, c_void_p]
        L.r9k_gemm_fp8_block_packed.argtypes = L.r9k_gemm_fp8_block.argtypes
        L.r9k_gemm_fp8_block_qa_packed.argtypes = L.r9k_gemm_fp8_block_qa.argtypes
        L.r9k_pack_weight.argtypes = [c_void_p, c_int64, c_int64, c_void_p, c_void_p]
        L.r9k_set_dispatch.argtypes = [c_int, c_int]
        L.r9k_set_tiled_plan.argtypes = [c_int, c_int]
        L.r9k_get_tiled_plan.argtypes = [POINTER(c_int), POINTER(c_int)]
        L.r9k_get_dispatch.argtypes = [POINTER(c_int), POINTER(c_int)]
        L.r9k_gemm_fp8_block_plan.argtypes = [c_int64, c_int64, c_int64, c_int, POINTER(c_int), POINTER(c_int)]
        L.r9k_moe_fp8_decode_workspace.argtypes = [c_int64] * 5 + [POINTER(c_size_t)]
        L.r9k_moe_ws_offset.argtypes = [c_int64] * 5 + [c_int, POINTER(c_size_t)]
        L.r9k_moe_fp8_decode.argtypes = [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_int64, c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_void_p, c_void_p,
                                         c_size_t, c_int, c_void_p]
        L.r9k_moe_fp8_decode_packed.argtypes = L.r9k_moe_fp8_decode.argtypes
        L.r9k_moe_fp8_decode_ex.argtypes = L.r9k_moe_fp8_decode.argtypes[:15] + [POINTER(MoeOpts), c_void_p]
        L.r9k_moe_route.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_void_p, c_void_p]
        L.r9k_gemm_fp8_block_bf16a.argtypes = [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_int64, c_void_p,
                                               c_void_p]
        L.r9k_gemm_fp8_block_bf16a_packed.argtypes = L.r9k_gemm_fp8_block_bf16a.argtypes
        L.r9k_gemm_fp8_block_qa_noalloc.argtypes = [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_int64,
                                                    c_void_p, c_int, c_void_p]
        L.r9k_quant_weight_w4.argtypes = [c_void_p, c_int64, c_int64, c_int, c_int] + [c_void_p] * 4
        L.r9k_pack_weight_w4.argtypes = [c_void_p] * 3 + [c_int64, c_int64, c_int, c_int] + [c_void_p] * 4
        L.r9k_gemm_w4_workspace.argtypes = [c_int64, c_int64, c_int64, POINTER(c_size_t)]
        L.r9k_gemm_w4.argtypes = [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int64,
                                  c_void_p, c_void_p, c_size_t, c_void_p]
        L.r9k_moe_gemm_w4.argtypes = [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_int64, c_int64,
                                      c_void_p, c_void_p, c_void_p, c_int, c_int, c_int64, c_int, c_void_p, c_void_p]
        L.r9k_w4_plan.argtypes = [c_int64] * 4 + [c_int] * 3 + [POINTER(c_int)]
        L.r9k_set_w4_plan.argtypes = [c_int] * 5
        L.r9k_moe_permute_workspace.argtypes = [c_int64, c_int64, c_int64, POINTER(c_size_t)]
        L.r9k_moe_permute.argtypes = [c_void_p, c_int, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p,
                                      c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
        L.r9k_moe_permute_backward.argtypes = [c_void_p, c_int, c_int64, c_int64, c_void_p, c_int64, c_void_p,
                                               c_void_p]
        L.r9k_moe_unpermute.argtypes = [c_void_p, c_int, c_int64, c_int64, c_void_p, c_void_p, c_int64, c_void_p,
                                        c_void_p]
        L.r9k_moe_unpermute_backward.argtypes = [c_void_p, c_void_p, c_int, c_int64, c_int64, c_void_p, c_void_p,
                                                 c_int64, c_void_p, c_void_p, c_void_p]
        L.r9k_quant_i8.argtypes = [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_void_p]
        L.r9k_pack_weight_i8.argtypes = [c_void_p, c_int64, c_int64, c_void_p, c_void_p]
        L.r9k_gemm_i8_workspace.argtypes = [c_int64, c_int64, c_int64, POINTER(c_size_t)]
        L.r9k_gemm_i8_codes_workspace.argtypes = L.r9k_gemm_i8_workspace.argtypes
        L.r9k_gemm_i8.argtypes = L.r9k_gemm_fp8_block.argtypes
        L.r9k_gemm_i8_qa.argtypes = L.r9k_gemm_fp8_block_qa.argtypes
        L.r9k_moe_gemm_i8.argtypes = [c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_int64, c_int64,
                                      c_void_p, c_void_p, c_int64, c_int, c_void_p, c_void_p]
        L.r9k_i8_plan.argtypes = [c_int64] * 4 + [c_int, c_int, POINTER(c_int)]
        L.r9k_set_i8_plan.argtypes = [c_int] * 6
        L.r9k_moe_balance_loss_workspace.argtypes = [c_int64, c_int64, c_int64, POINTER(c_size_t)]
        L.r9k_moe_balance_loss.argtypes = [c_void_p, c_int, c_int64, c_int64, c_void_p, c_int64] + [c_void_p] * 5 + [
            c_size_t, c_void_p]
        L.r9k_moe_balance_loss_backward.argtypes = [c_void_p, c_void_p, c_int, c_int64, c_int64, c_int64] + [c_void_p] * 7
        L.r9k_moe_route_backward.argtypes = [c_void_p] * 3 + [c_int64] * 3 + [c_void_p] * 2
        v = L.r9k_abi_version()
        if v != ABI_VERSION:
            raise ImportError(f"libr9k.so has ABI version {v}, this binding needs {ABI_VERSION}")
        _lib = L
    return _lib


def abi_version() -> int:
    return lib().r9k_abi_version()


def strerror(code: int) -> str:
    return lib().r9k_strerror(code).decode()


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise R9kError(rc, what)


# torch's handle of the current stream as a plain integer: about 0.15 us a call,
# where torch.cuda.current_stream() builds a Stream object (about 2.7 us), which
# was the largest host cost of an eager call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> c_void_p:
    if stream is None:
        if _raw_stream is not None:
            return c_void_p(_raw_stream(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t: torch.Tensor | None, dtypes, name: str) -> c_void_p:
    if t is None:
        return c_void_p(None)
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return c_void_p(t.data_ptr())


BF16 = (torch.bfloat16, torch.int16, torch.uint16)
FP8 = (torch.uint8, torch.float8_e4m3fn)
F32 = (torch.float32,)
I32 = (torch.int32,)


class Workspace:
    """A device workspace that grows on demand (each growth is a fresh
    allocation, zero-filled, though the library needs no initialisation: every
    call writes what it reads).  Not shared between streams that run
    concurrently."""

    def __init__(self, device=None):
        self.device = device
        self.buf: torch.Tensor | None = None

    def get(self, nbytes: int) -> torch.Tensor:
        nbytes = max(int(nbytes), 256)
        if self.buf is None or self.buf.numel() < nbytes:
            dev = self.device if self.device is not None else torch.device("cuda", torch.cuda.current_device())
            self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        return self.buf


_default_ws: dict[int, Workspace] = {}


def _workspace(ws: torch.Tensor | None, nbytes: int) -> torch.Tensor:
    if ws is not None:
        return ws
    dev = torch.cuda.current_device()
    if dev not in _default_ws:
        _default_ws[dev] = Workspace(torch.device("cuda", dev))
    return _default_ws[dev].get(nbytes)


# ------------------------------------------------------------------ quant ----

def quant_act(a: torch.Tensor, aq: torch.Tensor | None = None, as_: torch.Tensor | None = None, stream=None):
    """Per-token group-128 activation quant: a [M,K] bf16 -> (codes [M,K] u8, scales [M,K/128] f32)."""
    M, K = a.shape
    if aq is None:
        aq = torch.empty((M, K), dtype=torch.uint8, device=a.device)
    if as_ is None:
        as_ = torch.empty((M, K // 128 if K % 128 == 0 else 1), dtype=torch.float32, device=a.device)
    _check(lib().r9k_quant_act(_ptr(a, BF16, "a"), M, K, _ptr(aq, FP8, "aq"), _ptr(as_, F32, "as"),
                               _stream(stream)), "r9k_quant_act")
    return aq, as_


def quant_weight(w: torch.Tensor, wq: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """128x128 block weight quant: w [N,K] bf16 -> (codes [N,K] u8, scales [N/128,K/128] f32)."""
    N, K = w.shape
    if wq is None:
        wq = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    if ws is None:
        ws = torch.empty((max(N // 128, 1), max(K // 128, 1)), dtype=torch.float32, device=w.device)
    _check(lib().r9k_quant_weight(_ptr(w, BF16, "w"), N, K, _ptr(wq, FP8, "wq"), _ptr(ws, F32, "ws"),
                                  _stream(stream)), "r9k_quant_weight")
    return wq, ws


def encode_e4m3(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Elementwise fp32 -> e4m3fn codes with the library's device encoder."""
    n = x.numel()
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(lib().r9k_encode_e4m3(_ptr(x, F32, "x"), n, _ptr(out, FP8, "codes"), _stream(stream)),
           "r9k_encode_e4m3")
    return out


# ------------------------------------------------------------------- gemm ----

@functools.lru_cache(maxsize=4096)
def gemm_fp8_block_workspace(M: int, K: int, N: int) -> int:
    """Workspace bytes for a GEMM of this shape (r9k_gemm_fp8_block_workspace).  The answer depends on the
    shape (it covers every dispatch setting, and the library reads its tuning variables once) and on a
    forced tiled plan, which set_tiled_plan changes and then clears this cache; so it is cached: an eager
    call then pays no query."""
    b = c_size_t(0)
    _check(lib().r9k_gemm_fp8_block_workspace(M, K, N, ctypes.byref(b)), "r9k_gemm_fp8_block_workspace")
    return b.value


def gemm_fp8_block(aq, as_, w, ws, c=None, workspace=None, stream=None) -> torch.Tensor:
    """Block GEMM on pre-quantised activations (the split form) -> C [M,N] bf16."""
    M, K = aq.shape
    N = w.shape[0]
    if c is None:
        c = torch.empty((M, N), dtype=torch.bfloat16, device=aq.device)
    if M == 0:  # an empty batch: nothing to compute (an empty tensor has no device address to pass)
        return c
    nbytes = gemm_fp8_block_workspace(M, K, N)
    wsb = _workspace(workspace, nbytes)
    _check(lib().r9k_gemm_fp8_block(_ptr(aq, FP8, "aq"), _ptr(as_, F32, "as"), M, K, _ptr(w, FP8, "w"),
                                    _ptr(ws, F32, "ws"), N, _ptr(c, BF16, "c"), _ptr(wsb, FP8, "workspace"),
                                    wsb.numel(), _stream(stream)), "r9k_gemm_fp8_block")
    return c


def gemm_fp8_block_qa(a, w, ws, c=None, workspace=None, stream=None) -> torch.Tensor:
    """The fused form: bf16 activations quantised inside the GEMM -> C [M,N] bf16."""
    M, K = a.shape
    N = w.shape[0]
    if c is None:
        c = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if M == 0:  # an empty batch: nothing to compute (an empty tensor has no device address to pass)
        return c
    nbytes = gemm_fp8_block_workspace(M, K, N)
    wsb = _workspace(workspace, nbytes)
    _check(lib().r9k_gemm_fp8_block_qa(_ptr(a, BF16, "a"), M, K, _ptr(w, FP8, "w"), _ptr(ws, F32, "ws"), N,
                                       _ptr(c, BF16, "c"), _ptr(wsb, FP8, "workspace"), wsb.numel(),
                                       _stream(stream)), "r9k_gemm_fp8_block_qa")
    return c


NOALLOC_SCRATCH_BYTES = 64 << 20


def gemm_fp8_block_qa_noalloc(a, w, ws, c=None, packed: bool = False, stream=None) -> torch.Tensor:
    """The fused GEMM without a workspace (r9k_gemm_fp8_block_qa_noalloc): the library's own scratch on
    this GPU, no device allocation in the call (pass c to avoid torch's output allocation too).  Calls on
    one GPU must not overlap in time."""
    M, K = a.shape
    N = w.shape[0]
    if c is None:
        c = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if M == 0:  # an empty batch: nothing to compute (an empty tensor has no device address to pass)
        return c
    _check(lib().r9k_gemm_fp8_block_qa_noalloc(_ptr(a, BF16, "a"), M, K, _ptr(w, FP8, "w"), _ptr(ws, F32, "ws"), N,
                                               _ptr(c, BF16, "c"), 1 if packed else 0, _stream(stream)),
           "r9k_gemm_fp8_block_qa_noalloc")
    return c


def gemm_fp8_block_bf16a(a, w, ws, c=None, stream=None, packed: bool = False) -> torch.Tensor:
    """The bf16-activation variant at decode widths (M <= 16): a [M,K] bf16 (not quantised), w [N,K] fp8 codes
    (or their pack_weight copy when packed), ws [N/128,K/128] -> C [M,N] bf16."""
    M, K = a.shape
    N = w.shape[0]
    if c is None:
        c = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    fn = lib().r9k_gemm_fp8_block_bf16a_packed if packed else lib().r9k_gemm_fp8_block_bf16a
    _check(fn(_ptr(a, BF16, "a"), M, K, _ptr(w, FP8, "w"), _ptr(ws, F32, "ws"), N, _ptr(c, BF16, "c"),
              _stream(stream)), "r9k_gemm_fp8_block_bf16a_packed" if packed else "r9k_gemm_fp8_block_bf16a")
    return c


def pack_weight(wq: torch.Tensor, wp: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Fragment-order copy of the weight codes (r9k_pack_weight): wq [N,K] u8
    row-major -> wp, also [N,K] u8 in shape, bytes in fragment order."""
    N, K = wq.shape
    if wp is None:
        wp = torch.empty((N, K), dtype=torch.uint8, device=wq.device)
    _check(lib().r9k_pack_weight(_ptr(wq, FP8, "wq"), N, K, _ptr(wp, FP8, "wp"), _stream(stream)),
           "r9k_pack_weight")
    return wp


def gemm_fp8_block_packed(aq, as_, wp, ws, c=None, workspace=None, stream=None) -> torch.Tensor:
    """gemm_fp8_block on fragment-order weights (pack_weight)."""
    M, K = aq.shape
    N = wp.shape[0]
    if c is None:
        c = torch.empty((M, N), dtype=torch.bfloat16, device=aq.device)
    if M == 0:  # an empty batch: nothing to compute (an empty tensor has no device address to pass)
        return c
    nbytes = gemm_fp8_block_workspace(M, K, N)
    wsb = _workspace(workspace, nbytes)
    _check(lib().r9k_gemm_fp8_block_packed(_ptr(aq, FP8, "aq"), _ptr(as_, F32, "as"), M, K, _ptr(wp, FP8, "wp"),
                                           _ptr(ws, F32, "ws"), N, _ptr(c, BF16, "c"),
                                           _ptr(wsb, FP8, "workspace"), wsb.numel(), _stream(stream)),
           "r9k_gemm_fp8_block_packed")
    return c


def gemm_fp8_block_qa_packed(a, wp, ws, c=None, workspace=None, stream=None) -> torch.Tensor:
    """gemm_fp8_block_qa on fragment-order weights (pack_weight)."""
    M, K = a.shape
    N = wp.shape[0]
    if c is None:
        c = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if M == 0:  # an empty batch: nothing to compute (an empty tensor has no device address to pass)
        return c
    nbytes = gemm_fp8_block_workspace(M, K, N)
    wsb = _workspace(workspace, nbytes)
    _check(lib().r9k_gemm_fp8_block_qa_packed(_ptr(a, BF16, "a"), M, K, _ptr(wp, FP8, "wp"), _ptr(ws, F32, "ws"),
                                              N, _ptr(c, BF16, "c"), _ptr(wsb, FP8, "workspace"), wsb.numel(),
                                              _stream(stream)), "r9k_gemm_fp8_block_qa_packed")
    return c


def set_dispatch(skinny_max_m: int = 255, engine: int = ENGINE_AUTO) -> None:
    _check(lib().r9k_set_dispatch(skinny_max_m, engine), "r9k_set_dispatch")


def set_tiled_plan(shape: int = TILE_AUTO, ksplit: int = 0) -> None:
    """Force the tiled engine's tile shape (TILE_*) and K split (0: the planner's) for later calls
    (r9k_set_tiled_plan).  A forced split changes the workspace a shape needs, so the cached
    workspace sizes are dropped."""
    _check(lib().r9k_set_tiled_plan(shape, ksplit), "r9k_set_tiled_plan")
    gemm_fp8_block_workspace.cache_clear()


def get_tiled_plan() -> tuple[int, int]:
    sh, ks = c_int(0), c_int(0)
    _check(lib().r9k_get_tiled_plan(ctypes.byref(sh), ctypes.byref(ks)), "r9k_get_tiled_plan")
    return sh.value, ks.value


def get_dispatch() -> tuple[int, int]:
    m, e = c_int(0), c_int(0)
    _check(lib().r9k_get_dispatch(ctypes.byref(m), ctypes.byref(e)), "r9k_get_dispatch")
    return m.value, e.value


KERNEL_NONE, KERNEL_DECODE, KERNEL_SKINNY, KERNEL_TILED, KERNEL_MID = 0, 1, 2, 3, 4


def gemm_fp8_block_plan(M: int, K: int, N: int, packed: bool = False) -> tuple[int, int]:
    """(kernel, ksplit) that a GEMM call of this shape runs (host only)."""
    k, s = c_int(0), c_int(0)
    _check(lib().r9k_gemm_fp8_block_plan(M, K, N, int(bool(packed)), ctypes.byref(k), ctypes.byref(s)),
           "r9k_gemm_fp8_block_plan")
    return k.value, s.value


# -------------------------------------------------------------------- moe ----

@functools.lru_cache(maxsize=1024)
def moe_fp8_decode_workspace(T: int, H: int, E: int, I: int, topk: int) -> int:
    b = c_size_t(0)
    _check(lib().r9k_moe_fp8_decode_workspace(T, H, E, I, topk, ctypes.byref(b)), "r9k_moe_fp8_decode_workspace")
    return b.value


def moe_ws_offset(T: int, H: int, E: int, I: int, topk: int, which: str) -> int:
    b = c_size_t(0)
    w = {"gu": 0, "h": 1, "y": 2, "hq": 3, "hs": 4}[which]
    _check(lib().r9k_moe_ws_offset(T, H, E, I, topk, w, ctypes.byref(b)), "r9k_moe_ws_offset")
    return b.value


class MoeOpts(ctypes.Structure):
    """r9k_moe_opts."""
    _fields_ = [("fused", c_int), ("packed", c_int), ("shared", c_void_p), ("shared_w", c_void_p)]


def moe_route(logits, topk: int, ids=None, w=None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """One-launch routing: logits [T,E] fp32 -> (topk ids [T,topk] int32, renormalised weights [T,topk] fp32)."""
    T, E = logits.shape
    if ids is None:
        ids = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
    _check(lib().r9k_moe_route(_ptr(logits, F32, "logits"), T, E, topk, _ptr(ids, I32, "ids"), _ptr(w, F32, "w"),
                               _stream(stream)), "r9k_moe_route")
    return ids, w


def moe_fp8_decode(x, topk_ids, topk_w, w13, w13_s, w2, w2_s, out=None, workspace=None, fused: bool = True,
                   stream=None, packed: bool = False, shared=None, shared_w=None) -> torch.Tensor:
    """Routed MoE decode: x [T,H] bf16, ids/weights [T,topk], experts w13 [E,2I,H], w2 [E,H,I] (fp8 +
    block scales) -> out [T,H] bf16.  packed: w13 and w2 are pack_weight copies (same shapes).
    shared [T,H] bf16 (and its per-token weight shared_w [T] fp32): the shared expert's output, added in the
    combine (r9k_moe_fp8_decode_ex)."""
    T, H = x.shape
    topk = topk_ids.shape[1]
    E, twoI, _ = w13.shape
    I = twoI // 2
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    nbytes = moe_fp8_decode_workspace(T, H, E, I, topk)
    wsb = _workspace(workspace, nbytes)
    if shared is not None or shared_w is not None:
        opts = MoeOpts(1 if fused else 0, 1 if packed else 0, _ptr(shared, BF16, "shared"),
                       _ptr(shared_w, F32, "shared_w"))
        _check(lib().r9k_moe_fp8_decode_ex(
            _ptr(x, BF16, "x"), T, H, _ptr(topk_ids, I32, "topk_ids"), _ptr(topk_w, F32, "topk_w"), topk,
            _ptr(w13, FP8, "w13"), _ptr(w13_s, F32, "w13_s"), _ptr(w2, FP8, "w2"), _ptr(w2_s, F32, "w2_s"), E, I,
            _ptr(out, BF16, "out"), _ptr(wsb, FP8, "workspace"), wsb.numel(), ctypes.byref(opts), _stream(stream)),
            "r9k_moe_fp8_decode_ex")
        return out
    fn = lib().r9k_moe_fp8_decode_packed if packed else lib().r9k_moe_fp8_decode
    _check(fn(_ptr(x, BF16, "x"), T, H, _ptr(topk_ids, I32, "topk_ids"), _ptr(topk_w, F32, "topk_w"), topk,
              _ptr(w13, FP8, "w13"), _ptr(w13_s, F32, "w13_s"), _ptr(w2, FP8, "w2"), _ptr(w2_s, F32, "w2_s"), E, I,
              _ptr(out, BF16, "out"), _ptr(wsb, FP8, "workspace"), wsb.numel(), 1 if fused else 0, _stream(stream)),
           "r9k_moe_fp8_decode_packed" if packed else "r9k_moe_fp8_decode")
    return out


# ------------------------------------------------------ 4-bit weights ----

W4_INT, W4_MXFP4 = 0, 1
ACT_NONE, ACT_SILU_MUL = 0, 1
U8 = (torch.uint8,)
_ROWS = {torch.bfloat16: 0, torch.float32: 1}  # R9K_BF16, R9K_F32


# the current device's index without torch.cuda's lazy-initialisation check (a device
# tensor is in hand when these are called)
_cur_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _dev(t: torch.Tensor, name: str) -> int:
    """The current device's index; the call's first tensor has to be there."""
    if t.is_cuda:
        cur = _cur_device()
        if t.get_device() == cur:
            return cur
    raise ValueError(f"{name} must be a tensor of the current device")


def _addr(t: torch.Tensor, dtypes, name: str, dev: int, shape=None) -> int:
    """Device address of a contiguous tensor of device `dev`, checked (0 for an empty one)."""
    if t.dtype in dtypes and t.get_device() == dev and t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor of the current device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name}: shape {tuple(t.shape)}, needs {tuple(shape)}")


def _raw(stream, dev: int) -> int:
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(shape, dtype, dev: int, stream, like: torch.Tensor | None = None) -> torch.Tensor:
    """A fresh tensor for a call on `stream`, owned by that stream in torch's allocator.  `like`: a tensor of that
    type and device, from which torch makes one in less time."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev) if like is None else like.new_empty(shape)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _scratch(ws: torch.Tensor | None, nbytes: int, dev: int, stream):
    """(address, bytes, tensor) of a call's workspace: the caller's, or a fresh one, which torch keeps for
    this stream (or the graph being captured) until the call's work is done."""
    if nbytes == 0:
        return None, 0, None
    if ws is None:
        ws = _new((nbytes,), torch.uint8, dev, stream)
    return _addr(ws, U8, "workspace", dev) or None, ws.numel(), ws


_W4_SCALES = {torch.bfloat16: W4_INT, torch.uint8: W4_MXFP4}


def _w4_format(wp, sp, zp, dev: int, dims: int = 0):
    """Addresses, format, rows (all leading sizes), K and group of a 4-bit weight [..., N, K/2] with its scales and
    zeros [..., N, K/group] (`dims`: the number of sizes it must have)."""
    ws, ss = wp.shape, sp.shape
    nd = len(ws)
    if nd < 2 or (dims and nd != dims) or len(ss) != nd or ss[-2] != ws[-2] or (nd > 2 and ss[:-2] != ws[:-2]):
        raise ValueError(f"scales {tuple(ss)} do not go with 4-bit codes {tuple(ws)}"
                         + (f" of {dims} sizes" if dims else ""))
    K, groups = 2 * ws[-1], ss[-1]
    if not K or not groups or K % groups:
        raise ValueError(f"{groups} scales a row do not divide K = {K}")
    return (_addr(wp, U8, "codes", dev), _addr(sp, _W4_SCALES, "scales", dev),
            None if zp is None else _addr(zp, U8, "zeros", dev, ss), _W4_SCALES[sp.dtype], K, K // groups)


def quant_weight_w4(w: torch.Tensor, group: int = 128, fmt: int = W4_INT, zeros: bool = False, stream=None):
    """4-bit group quant: w [..., N, K] bf16 -> (codes [..., N, K/2] u8, scales [..., N, K/group], zeros or None).
    W4_INT: scales bf16, zero points u8 when `zeros` (else 8 is meant); W4_MXFP4: group 32, scales u8 (e8m0)."""
    dev = _dev(w, "w")
    K, rows = w.shape[-1], w.numel() // max(w.shape[-1], 1)
    if not K or group <= 0 or K % group:
        raise ValueError(f"K = {K} is not whole groups of {group}")
    lead = w.shape[:-1]
    wq = _new((*lead, K // 2), torch.uint8, dev, stream)
    s = _new((*lead, K // group), torch.bfloat16 if fmt == W4_INT else torch.uint8, dev, stream)
    z = _new((*lead, K // group), torch.uint8, dev, stream) if zeros else None
    _check(lib().r9k_quant_weight_w4(_addr(w, BF16, "w", dev), rows, K, fmt, group, wq.data_ptr(), s.data_ptr(),
                                     None if z is None else z.data_ptr(), _raw(stream, dev)), "r9k_quant_weight_w4")
    return wq, s, z


def pack_weight_w4(wq, s, z=None, stream=None):
    """The packed copy that the products read (r9k_pack_weight_w4): codes [..., N, K/2], scales [..., N, K/group],
    zeros or None -> the same shapes.  Experts' weights [E, N, K/2] pack as one.  Once, at load time."""
    dev = _dev(wq, "wq")
    a, b, c, fmt, K, group = _w4_format(wq, s, z, dev)
    wp, sp = _new(wq.shape, torch.uint8, dev, stream), _new(s.shape, s.dtype, dev, stream)
    zp = None if z is None else _new(z.shape, torch.uint8, dev, stream)
    if wq.shape[-2] % 16:
        raise ValueError(f"wq: {wq.shape[-2]} rows are not a multiple of 16")
    _check(lib().r9k_pack_weight_w4(a, b, c, 2 * wq.numel() // K, K, fmt, group, wp.data_ptr(), sp.data_ptr(),
                                    None if zp is None else zp.data_ptr(), _raw(stream, dev)), "r9k_pack_weight_w4")
    return wp, sp, zp


@functools.lru_cache(maxsize=4096)
def gemm_w4_workspace(M: int, K: int, N: int) -> int:
    """Workspace bytes for gemm_w4 of this shape (r9k_gemm_w4_workspace); 0 for many shapes.  Cached; set_w4_plan,
    which changes the answer, clears the cache."""
    b = c_size_t(0)
    _check(lib().r9k_gemm_w4_workspace(M, K, N, ctypes.byref(b)), "r9k_gemm_w4_workspace")
    return b.value


def gemm_w4(a, wp, sp, zp=None, c=None, workspace=None, stream=None) -> torch.Tensor:
    """Product with a packed 4-bit weight (r9k_gemm_w4): a [M,K] bf16, (wp, sp, zp) from pack_weight_w4 -> C [M,N]
    bf16.  The format and the group follow from sp's type and shape."""
    # The checks of a well-formed call with its output and workspace given, in one
    # expression (a decode call's host time counts: 1.2 us less than one by one); any
    # other call goes through the checks that name what is wrong.
    dev = _dev(a, "a")  # a host tensor's index is -1: never compared with another's
    if c is not None and a.dtype in BF16 and c.dtype in BF16 and wp.dtype in U8 and len(a.shape) == len(sp.shape) == 2:
        M, K = a.shape
        N, groups = sp.shape
        if (wp.shape == (N, K // 2) and c.shape == (M, N) and M and groups and K % (2 * groups) == 0
                and sp.dtype in _W4_SCALES and a.is_contiguous() and wp.is_contiguous() and sp.is_contiguous()
                and c.is_contiguous()
                and wp.get_device() == sp.get_device() == c.get_device() == dev
                and (zp is None or (zp.dtype in U8 and zp.shape == (N, groups) and zp.is_contiguous()
                                    and zp.get_device() == dev))):
            need = gemm_w4_workspace(M, K, N)
            pw, nb, _keep = (None, 0, None) if need == 0 else _scratch(workspace, need, dev, stream)
            rc = lib().r9k_gemm_w4(a.data_ptr(), M, K, wp.data_ptr(), sp.data_ptr(),
                                   None if zp is None else zp.data_ptr(), _W4_SCALES[sp.dtype], K // groups, N,
                                   c.data_ptr(), pw, nb, _raw(stream, dev))
            if rc:
                _check(rc, "r9k_gemm_w4")
            return c
    w, s, z, fmt, K, group = _w4_format(wp, sp, zp, dev, 2)
    M, N = a.shape[0], wp.shape[0]
    pa = _addr(a, BF16, "a", dev, (M, K))
    if c is None:
        c = _new((M, N), torch.bfloat16, dev, stream)
    pc = _addr(c, BF16, "c", dev, (M, N))
    if M == 0:  # an empty batch: nothing to compute (an empty tensor has no device address to pass)
        return c
    pw, nb, _keep = _scratch(workspace, gemm_w4_workspace(M, K, N), dev, stream)
    _check(lib().r9k_gemm_w4(pa, M, K, w, s, z, fmt, group, N, pc, pw, nb, _raw(stream, dev)), "r9k_gemm_w4")
    return c


_ACTS = {"none": ACT_NONE, "silu_mul": ACT_SILU_MUL}


def moe_gemm_w4(x, offsets, wp, sp, zp=None, src=None, topk: int = 1, act: str = "none", c=None,
                stream=None) -> torch.Tensor:
    """The experts' products on sorted rows (r9k_moe_gemm_w4): offsets [E+1] and src [R] from moe_permute, (wp, sp,
    zp) the packed weights [E,N,K/2] -> [R,N] bf16, or with act="silu_mul" [R,N/2].  Without src, x [R,K] holds the
    sorted rows; with it, x [T,K] the tokens' rows and row r reads x[src[r] // topk], topk as in the sort (R more than
    T * topk is refused).  Rows from offsets[E] on are not written."""
    dev = _dev(x, "x")
    w, s, z, fmt, K, group = _w4_format(wp, sp, zp, dev, 3)
    if act not in _ACTS:
        raise ValueError(f"act {act!r} not in {tuple(_ACTS)}")
    rows, E, N = x.shape[0], wp.shape[0], wp.shape[1]
    R = rows if src is None else src.numel()
    out = (R, N if act == "none" else N // 2)
    px = _addr(x, BF16, "x", dev, (rows, K))
    po = _addr(offsets, I32, "offsets", dev, (E + 1,))
    ps = None if src is None else _addr(src, I32, "src", dev)
    if c is None:
        c = _new(out, torch.bfloat16, dev, stream)
    pc = _addr(c, BF16, "c", dev, out)
    if R == 0:
        return c
    rc = lib().r9k_moe_gemm_w4(px, rows, ps, topk, po, E, R, K, w, s, z, fmt, group, N, _ACTS[act], pc,
                               _raw(stream, dev))
    if rc:
        _check(rc, "r9k_moe_gemm_w4")
    return c


W4_AUTO, W4_STREAM, W4_TILED = 0, 1, 2


def w4_plan(M: int, K: int, N: int, E: int = 0, act: str = "none", fmt: int = W4_INT, group: int = 128) -> tuple:
    """The launch of a 4-bit product (r9k_w4_plan): (kernel W4_STREAM or W4_TILED, column tiles a wave, waves along
    the columns, waves along K, CTAs along K, LDS segments or 0).  E = 0: gemm_w4; else moe_gemm_w4 of M rows."""
    plan = (c_int * 6)()
    _check(lib().r9k_w4_plan(M, K, N, E, _ACTS[act], fmt, group, plan), "r9k_w4_plan")
    return tuple(plan)


def set_w4_plan(kernel: int = W4_AUTO, tiles: int = 0, waves: int = 0, slices: int = 0, ksplit: int = 0) -> None:
    """Force the launch of later 4-bit products (r9k_set_w4_plan; 0: the planner's).  A forced split changes the
    workspace a shape needs, so the cached workspace sizes are dropped."""
    _check(lib().r9k_set_w4_plan(kernel, tiles, waves, slices, ksplit), "r9k_set_w4_plan")
    gemm_w4_workspace.cache_clear()


# ------------------------------------------- rows sorted by expert ----

@functools.lru_cache(maxsize=1024)
def moe_permute_workspace(T: int, E: int, topk: int) -> int:
    b = c_size_t(0)
    _check(lib().r9k_moe_permute_workspace(T, E, topk, ctypes.byref(b)), "r9k_moe_permute_workspace")
    return b.value


def moe_permute(x, topk_ids, E: int, xs=None, src=None, pos=None, offsets=None, workspace=None, stream=None):
    """Token rows sorted by expert (r9k_moe_permute): x [T,H] bf16 or fp32, ids [T,topk] int32 -> (xs [T*topk,H],
    src [T*topk], pos [T,topk], offsets [E+1]).  x None: the sort alone, and xs is None.  Rows of xs from
    offsets[E] on (slots whose id lies outside [0,E)) are not written."""
    dev = _dev(topk_ids, "topk_ids")
    T, topk = topk_ids.shape
    R = T * topk
    need = moe_permute_workspace(T, E, topk)  # refuses counts that no output could be made for
    pi = _addr(topk_ids, I32, "topk_ids", dev)
    px = pxs = None
    H = dt = 0
    if x is not None:
        px = _addr(x, _ROWS, "x", dev)
        if x.dim() != 2 or x.shape[0] != T:
            raise ValueError(f"x: shape {tuple(x.shape)} does not go with {T} tokens")
        H, dt = x.shape[1], _ROWS[x.dtype]
        if xs is None:
            xs = _new((R, H), x.dtype, dev, stream)
        pxs = _addr(xs, (x.dtype,), "xs", dev, (R, H))
    elif xs is not None:
        raise ValueError("xs without x")
    if src is None:
        src = _new(R, torch.int32, dev, stream, topk_ids)
        psrc = src.data_ptr()
    else:
        psrc = _addr(src, I32, "src", dev, (R,))
    if pos is None:
        pos = _new((T, topk), torch.int32, dev, stream, topk_ids)
        ppos = pos.data_ptr()
    else:
        ppos = _addr(pos, I32, "pos", dev, (T, topk))
    if offsets is None:
        offsets = _new(E + 1, torch.int32, dev, stream, topk_ids)
        poff = offsets.data_ptr()
    else:
        poff = _addr(offsets, I32, "offsets", dev, (E + 1,))
    if T == 0:  # no slots (empty tensors have no device address to pass): the call sees only the offsets
        px = pxs = None
        pi = psrc = ppos = poff
    pw, nb, _keep = _scratch(workspace, need, dev, stream)
    rc = lib().r9k_moe_permute(px, dt, T, H, pi, topk, E, pxs, psrc, ppos, poff, pw, nb, _raw(stream, dev))
    if rc:
        _check(rc, "r9k_moe_permute")
    return xs, src, pos, offsets


def _sorted_rows(y, pos, dev: int, name: str):
    T, topk = pos.shape
    ppos = _addr(pos, I32, "pos", dev)
    py = _addr(y, _ROWS, name, dev)
    ys = y.shape
    if len(ys) != 2 or ys[0] != T * topk:
        raise ValueError(f"{name}: shape {tuple(ys)} does not go with {T} x {topk} slots")
    return T, topk, ys[1], ppos, py


def _out(t, shape, like, name: str, dev: int, stream):
    """(tensor, address) of an output of `like`'s type: the caller's, checked, or a fresh one."""
    if t is None:
        t = _new(shape, like.dtype, dev, stream, like)
        return t, t.data_ptr()
    return t, _addr(t, (like.dtype,), name, dev, shape)


def moe_permute_backward(gxs, pos, gx=None, stream=None) -> torch.Tensor:
    """Gradient of moe_permute: gxs [T*topk,H], pos [T,topk] -> gx [T,H], the sum over a token's kept slots."""
    dev = _dev(gxs, "gxs")
    T, topk, H, ppos, pg = _sorted_rows(gxs, pos, dev, "gxs")
    gx, po = _out(gx, (T, H), gxs, "gx", dev, stream)
    if T:
        rc = lib().r9k_moe_permute_backward(pg, _ROWS[gxs.dtype], T, H, ppos, topk, po, _raw(stream, dev))
        if rc:
            _check(rc, "r9k_moe_permute_backward")
    return gx


def moe_unpermute(y, pos, w=None, out=None, stream=None) -> torch.Tensor:
    """Sorted rows back to their tokens (r9k_moe_unpermute): y [T*topk,H], pos [T,topk], weights w [T,topk] fp32 (None: 1)
    -> out [T,H] = sum_j w[t,j] * y[pos[t,j]]."""
    dev = _dev(y, "y")
    T, topk, H, ppos, py = _sorted_rows(y, pos, dev, "y")
    pw = None if w is None else _addr(w, F32, "w", dev, (T, topk))
    out, po = _out(out, (T, H), y, "out", dev, stream)
    if T:
        rc = lib().r9k_moe_unpermute(py, _ROWS[y.dtype], T, H, ppos, pw, topk, po, _raw(stream, dev))
        if rc:
            _check(rc, "r9k_moe_unpermute")
    return out


def moe_unpermute_backward(gout, y, pos, w, gy=None, gw=None, stream=None):
    """Gradient of moe_unpermute: gout [T,H], y [T*topk,H], pos and w [T,topk] -> (gy [T*topk,H], gw [T,topk] fp32).
    Rows of gy that no slot fills are not written.  The gradient of moe_unpermute without weights takes ones."""
    dev = _dev(y, "y")
    if w is None:
        raise TypeError("w: the weights are needed (ones for a moe_unpermute without them)")
    T, topk, H, ppos, py = _sorted_rows(y, pos, dev, "y")
    pg = _addr(gout, (y.dtype,), "gout", dev, (T, H))
    pw = _addr(w, F32, "w", dev, (T, topk))
    gy, pgy = _out(gy, y.shape, y, "gy", dev, stream)
    gw, pgw = _out(gw, (T, topk), w, "gw", dev, stream)
    if T:
        rc = lib().r9k_moe_unpermute_backward(pg, py, _ROWS[y.dtype], T, H, ppos, pw, topk, pgy, pgw,
                                              _raw(stream, dev))
        if rc:
            _check(rc, "r9k_moe_unpermute_backward")
    return gy, gw


# ------------------------------------------ products in 8-bit integers ----

I8 = (torch.int8,)


def quant_i8(x: torch.Tensor, q=None, s=None, stream=None):
    """Rows to signed bytes with a scale each (r9k_quant_i8): x [..., K] bf16 -> (codes [..., K] int8, scales [...] fp32).
    Activations per token; a weight [..., N, K] per output channel, at load time."""
    dev = _dev(x, "x")
    if (q is not None and s is not None and x.dtype in BF16 and q.dtype in I8 and s.dtype in F32 and q.shape == x.shape
            and len(x.shape) and s.shape == x.shape[:-1] and x.is_contiguous() and q.is_contiguous() and s.is_contiguous()
            and q.get_device() == s.get_device() == dev):  # as in gemm_i8
        rows = s.numel()
        rc = lib().r9k_quant_i8(x.data_ptr(), rows, x.shape[-1], q.data_ptr(), s.data_ptr(), _raw(stream, dev)) if rows else 0
        if rc:
            _check(rc, "r9k_quant_i8")
        return q, s
    px = _addr(x, BF16, "x", dev)
    if x.dim() < 1:
        raise ValueError("x has no rows")
    if q is None:
        q = _new(x.shape, torch.int8, dev, stream)
    if s is None:
        s = _new(x.shape[:-1], torch.float32, dev, stream)
    pq, ps = _addr(q, I8, "q", dev, x.shape), _addr(s, F32, "s", dev, x.shape[:-1])
    if s.numel():
        rc = lib().r9k_quant_i8(px, s.numel(), x.shape[-1], pq, ps, _raw(stream, dev))
        if rc:
            _check(rc, "r9k_quant_i8")
    return q, s


def pack_weight_i8(wq: torch.Tensor, stream=None) -> torch.Tensor:
    """The packed copy that the products read (r9k_pack_weight_i8): codes [..., N, K] int8 -> the same shape.  Experts'
    weights [E, N, K] pack as one.  Once, at load time; the scales stay as they are."""
    dev = _dev(wq, "wq")
    if wq.dim() < 2 or wq.shape[-2] % 16 or not wq.numel():
        raise ValueError(f"wq: shape {tuple(wq.shape)}; its rows must be a multiple of 16")
    p = _addr(wq, I8, "wq", dev)
    wp = _new(wq.shape, torch.int8, dev, stream)
    K = wq.shape[-1]
    _check(lib().r9k_pack_weight_i8(p, wq.numel() // K, K, wp.data_ptr(), _raw(stream, dev)), "r9k_pack_weight_i8")
    return wp


@functools.lru_cache(maxsize=4096)
def gemm_i8_workspace(M: int, K: int, N: int, quant: bool = True) -> int:
    """Workspace bytes for gemm_i8 and gemm_i8_qa of this shape (r9k_gemm_i8_workspace); with quant=False for gemm_i8
    alone (r9k_gemm_i8_codes_workspace), which has no codes to keep: 0 unless K is split."""
    b = c_size_t(0)
    if quant:
        _check(lib().r9k_gemm_i8_workspace(M, K, N, ctypes.byref(b)), "r9k_gemm_i8_workspace")
    else:
        _check(lib().r9k_gemm_i8_codes_workspace(M, K, N, ctypes.byref(b)), "r9k_gemm_i8_codes_workspace")
    return b.value


def _i8_product(x, wp, ws, c, dev: int, stream):
    if x.dim() != 2 or wp.dim() != 2 or not wp.numel():
        raise ValueError(f"activations {tuple(x.shape)} and weight {tuple(wp.shape)} need two sizes each, the weight some values")
    (M, K), N = x.shape, wp.shape[0]
    pw, ps = _addr(wp, I8, "wp", dev, (N, K)), _addr(ws, F32, "ws", dev, (N,))
    if c is None:
        c = _new((M, N), torch.bfloat16, dev, stream)
    return M, K, N, pw, ps, c, _addr(c, BF16, "c", dev, (M, N))


def gemm_i8(aq, as_, wp, ws, c=None, workspace=None, stream=None) -> torch.Tensor:
    """The product of int8 codes (r9k_gemm_i8): aq [M,K], as_ [M], wp [N,K] from pack_weight_i8, ws [N] -> C [M,N] bf16."""
    dev = _dev(aq, "aq")
    # A well-formed call with its output given, checked in one expression (0.8 us less than one by one); any other goes
    # through the checks that name what is wrong.
    if (c is not None and aq.dtype in I8 and as_.dtype in F32 and wp.dtype in I8 and ws.dtype in F32 and c.dtype in BF16
            and len(aq.shape) == len(wp.shape) == 2):
        M, K = aq.shape
        N = wp.shape[0]
        if (M and N and wp.shape == (N, K) and as_.shape == (M,) and ws.shape == (N,) and c.shape == (M, N)
                and aq.is_contiguous() and as_.is_contiguous() and wp.is_contiguous() and ws.is_contiguous()
                and c.is_contiguous()
                and as_.get_device() == wp.get_device() == ws.get_device() == c.get_device() == dev):
            need = gemm_i8_workspace(M, K, N, False)
            pws, nb, _keep = (None, 0, None) if need == 0 else _scratch(workspace, need, dev, stream)
            rc = lib().r9k_gemm_i8(aq.data_ptr(), as_.data_ptr(), M, K, wp.data_ptr(), ws.data_ptr(), N, c.data_ptr(),
                                   pws, nb, _raw(stream, dev))
            if rc:
                _check(rc, "r9k_gemm_i8")
            return c
    M, K, N, pw, ps, c, pc = _i8_product(aq, wp, ws, c, dev, stream)
    pa, pas = _addr(aq, I8, "aq", dev), _addr(as_, F32, "as", dev, (M,))
    if M == 0:  # an empty batch: nothing to compute (an empty tensor has no device address to pass)
        return c
    pws, nb, _keep = _scratch(workspace, gemm_i8_workspace(M, K, N, False), dev, stream)
    rc = lib().r9k_gemm_i8(pa, pas, M, K, pw, ps, N, pc, pws, nb, _raw(stream, dev))
    if rc:
        _check(rc, "r9k_gemm_i8")
    return c


def gemm_i8_qa(a, wp, ws, c=None, workspace=None, stream=None) -> torch.Tensor:
    """The product with the activations quantised in the call (r9k_gemm_i8_qa): a [M,K] bf16, (wp, ws) as for gemm_i8
    -> C [M,N] bf16, the bits of quant_i8 and gemm_i8."""
    dev = _dev(a, "a")
    if (c is not None and a.dtype in BF16 and wp.dtype in I8 and ws.dtype in F32 and c.dtype in BF16
            and len(a.shape) == len(wp.shape) == 2):  # as in gemm_i8
        M, K = a.shape
        N = wp.shape[0]
        if (M and N and wp.shape == (N, K) and ws.shape == (N,) and c.shape == (M, N) and a.is_contiguous()
                and wp.is_contiguous() and ws.is_contiguous() and c.is_contiguous()
                and wp.get_device() == ws.get_device() == c.get_device() == dev):
            need = gemm_i8_workspace(M, K, N)
            pws, nb, _keep = (None, 0, None) if need == 0 else _scratch(workspace, need, dev, stream)
            rc = lib().r9k_gemm_i8_qa(a.data_ptr(), M, K, wp.data_ptr(), ws.data_ptr(), N, c.data_ptr(), pws, nb,
                                      _raw(stream, dev))
            if rc:
                _check(rc, "r9k_gemm_i8_qa")
            return c
    M, K, N, pw, ps, c, pc = _i8_product(a, wp, ws, c, dev, stream)
    pa = _addr(a, BF16, "a", dev)
    if M == 0:
        return c
    pws, nb, _keep = _scratch(workspace, gemm_i8_workspace(M, K, N), dev, stream)
    rc = lib().r9k_gemm_i8_qa(pa, M, K, pw, ps, N, pc, pws, nb, _raw(stream, dev))
    if rc:
        _check(rc, "r9k_gemm_i8_qa")
    return c


def moe_gemm_i8(xq, xs, offsets, wp, ws, src=None, topk: int = 1, act: str = "none", c=None,
                stream=None) -> torch.Tensor:
    """The experts' products on sorted rows, in int8 codes (r9k_moe_gemm_i8): xq [rows,K] and xs [rows] from quant_i8,
    offsets [E+1] and src [R] from moe_permute, wp [E,N,K] from pack_weight_i8, ws [E,N] -> [R,N] bf16, or with
    act="silu_mul" [R,N/2].  Without src, xq holds the sorted rows; with it the tokens' rows, and row r reads
    xq[src[r] // topk], topk as in the sort.  Rows from offsets[E] on are not written."""
    dev = _dev(xq, "xq")
    if act not in _ACTS:
        raise ValueError(f"act {act!r} not in {tuple(_ACTS)}")
    if xq.dim() != 2 or wp.dim() != 3 or not wp.numel():
        raise ValueError(f"activations {tuple(xq.shape)} need two sizes, the experts' weight {tuple(wp.shape)} three and "
                         "some values")
    (rows, K), (E, N) = xq.shape, wp.shape[:2]
    if (c is not None and xq.dtype in I8 and xs.dtype in F32 and wp.dtype in I8 and ws.dtype in F32 and offsets.dtype in I32
            and c.dtype in BF16 and wp.shape[2] == K and xs.shape == (rows,) and ws.shape == (E, N) and offsets.shape == (E + 1,)
            and xq.is_contiguous() and xs.is_contiguous() and wp.is_contiguous() and ws.is_contiguous()
            and offsets.is_contiguous() and c.is_contiguous()
            and xs.get_device() == wp.get_device() == ws.get_device() == offsets.get_device() == c.get_device() == dev
            and (src is None or (src.dtype in I32 and src.is_contiguous() and src.get_device() == dev))):  # as in gemm_i8
        R = rows if src is None else src.numel()
        if R and c.shape == (R, N if act == "none" else N // 2):
            rc = lib().r9k_moe_gemm_i8(xq.data_ptr(), xs.data_ptr(), rows, None if src is None else src.data_ptr(), topk,
                                       offsets.data_ptr(), E, R, K, wp.data_ptr(), ws.data_ptr(), N, _ACTS[act], c.data_ptr(),
                                       _raw(stream, dev))
            if rc:
                _check(rc, "r9k_moe_gemm_i8")
            return c
    px, pxs = _addr(xq, I8, "xq", dev), _addr(xs, F32, "xs", dev, (rows,))
    pw, ps = _addr(wp, I8, "wp", dev, (E, N, K)), _addr(ws, F32, "ws", dev, (E, N))
    po = _addr(offsets, I32, "offsets", dev, (E + 1,))
    pi = None if src is None else _addr(src, I32, "src", dev)
    R = rows if src is None else src.numel()
    out = (R, N if act == "none" else N // 2)
    if c is None:
        c = _new(out, torch.bfloat16, dev, stream)
    pc = _addr(c, BF16, "c", dev, out)
    if R == 0:
        return c
    rc = lib().r9k_moe_gemm_i8(px, pxs, rows, pi, topk, po, E, R, K, pw, ps, N, _ACTS[act], pc, _raw(stream, dev))
    if rc:
        _check(rc, "r9k_moe_gemm_i8")
    return c


I8_AUTO, I8_STREAM, I8_TILED = 0, 1, 2


def i8_plan(M: int, K: int, N: int, E: int = 0, act: str = "none", quant: bool = False) -> tuple:
    """The launch of an 8-bit product (r9k_i8_plan): (I8_STREAM, column tiles a wave, waves along the columns, waves along
    K, CTAs along K, row tiles a CTA, whether the activations are quantised inside) or (I8_TILED, columns, rows, 0, CTAs
    along K, 0, 0).  E = 0: gemm_i8, with quant gemm_i8_qa; else moe_gemm_i8 of M rows."""
    plan = (c_int * 7)()
    _check(lib().r9k_i8_plan(M, K, N, E, _ACTS[act], int(quant), plan), "r9k_i8_plan")
    return tuple(plan)


def set_i8_plan(kernel: int = I8_AUTO, a: int = 0, b: int = 0, c: int = 0, ksplit: int = 0, rows: int = 0) -> None:
    """Force the launch of later 8-bit products (r9k_set_i8_plan; 0: the planner's).  A forced plan changes the workspace
    a shape needs, so the cached workspace sizes are dropped."""
    _check(lib().r9k_set_i8_plan(kernel, a, b, c, ksplit, rows), "r9k_set_i8_plan")
    gemm_i8_workspace.cache_clear()


# --------------------------------------------------- the router in training ----

MASK = (torch.bool, torch.uint8)


@functools.lru_cache(maxsize=1024)
def moe_balance_loss_workspace(T: int, E: int, topk: int) -> int:
    b = c_size_t(0)
    _check(lib().r9k_moe_balance_loss_workspace(T, E, topk, ctypes.byref(b)), "r9k_moe_balance_loss_workspace")
    return b.value


def moe_balance_loss(logits, topk_ids, mask=None, loss=None, counts=None, psum=None, workspace=None, stream=None):
    """The load balance loss of a routed batch (r9k_moe_balance_loss): logits [T,E] fp32 or bf16, ids [T,topk] int32, mask
    [T] bool (None: every token counts) -> (loss [] fp32, counts [E+1] int32: the slots of each expert and last the tokens
    counted, psum [E] fp32)."""
    dev = _dev(logits, "logits")
    if logits.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError(f"logits {tuple(logits.shape)} and ids {tuple(topk_ids.shape)} need two sizes each")
    (T, E), topk = logits.shape, topk_ids.shape[1]
    need = moe_balance_loss_workspace(T, E, topk)  # refuses sizes that no output could be made for
    pl = _addr(logits, _ROWS, "logits", dev)
    pi = _addr(topk_ids, I32, "topk_ids", dev, (T, topk))
    pm = None if mask is None else _addr(mask, MASK, "mask", dev, (T,))
    like = logits if logits.dtype in F32 else None
    if loss is None:
        loss = _new((), torch.float32, dev, stream, like)
        po = loss.data_ptr()
    else:
        po = _addr(loss, F32, "loss", dev, ())
    if counts is None:
        counts = _new((E + 1,), torch.int32, dev, stream, topk_ids)
        pc = counts.data_ptr()
    else:
        pc = _addr(counts, I32, "counts", dev, (E + 1,))
    if psum is None:
        psum = _new((E,), torch.float32, dev, stream, like)
        pp = psum.data_ptr()
    else:
        pp = _addr(psum, F32, "psum", dev, (E,))
    pw, nb, keep = _scratch(workspace, need, dev, stream)
    if T == 0:  # no rows to read (empty tensors have no device address to pass)
        pl = pi = po
        pm = None
    rc = lib().r9k_moe_balance_loss(pl, _ROWS[logits.dtype], T, E, pi, topk, pm, po, pc, pp, pw, nb, _raw(stream, dev))
    if rc:
        _check(rc, "r9k_moe_balance_loss")
    return loss, counts, psum


def moe_balance_loss_backward(gloss, logits, counts, topk: int, mask=None, route=None, glogits=None,
                              stream=None) -> torch.Tensor:
    """The gradient of moe_balance_loss for the logits (r9k_moe_balance_loss_backward): gloss [] fp32, logits and mask as in
    the forward call, counts [E+1] from it (or their sum over ranks) -> glogits [T,E] of the logits' type.  route = (gw, ids,
    w), each [T,topk]: the gradient of moe_route_backward is added in the same pass."""
    dev = _dev(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits {tuple(logits.shape)} need two sizes")
    T, E = logits.shape
    pl = _addr(logits, _ROWS, "logits", dev)
    pg, pc = _addr(gloss, F32, "gloss", dev, ()), _addr(counts, I32, "counts", dev, (E + 1,))
    pm = None if mask is None else _addr(mask, MASK, "mask", dev, (T,))
    pgw = pi = pw = None
    if route is not None:
        gw, ids, w = route
        pgw, pi = _addr(gw, F32, "gw", dev, (T, topk)), _addr(ids, I32, "ids", dev, (T, topk))
        pw = _addr(w, F32, "w", dev, (T, topk))
    glogits, po = _out(glogits, (T, E), logits, "glogits", dev, stream)
    if T:
        rc = lib().r9k_moe_balance_loss_backward(pg, pl, _ROWS[logits.dtype], T, E, topk, pc, pm, pgw, pi, pw, po,
                                                 _raw(stream, dev))
        if rc:
            _check(rc, "r9k_moe_balance_loss_backward")
    return glogits


def moe_route_backward(gw, topk_ids, topk_w, E: int, glogits=None, stream=None) -> torch.Tensor:
    """The gradient of moe_route for the logits (r9k_moe_route_backward): gw, ids and weights [T,topk] -> glogits [T,E] fp32,
    zero outside a token's experts."""
    dev = _dev(gw, "gw")
    if gw.dim() != 2:
        raise ValueError(f"gw {tuple(gw.shape)} needs two sizes")
    T, topk = gw.shape
    if not 1 <= E <= 65536:  # before an output of that many columns is made
        _check(-2, "r9k_moe_route_backward")
    if (gw.dtype in F32 and topk_ids.dtype in I32 and topk_w.dtype in F32 and topk_ids.shape == gw.shape == topk_w.shape
            and topk_ids.get_device() == topk_w.get_device() == dev and gw.is_contiguous() and topk_ids.is_contiguous()
            and topk_w.is_contiguous()):
        pg, pi, pw = gw.data_ptr(), topk_ids.data_ptr(), topk_w.data_ptr()
    else:  # name what is wrong
        pg, pi, pw = _addr(gw, F32, "gw", dev), _addr(topk_ids, I32, "ids", dev, gw.shape), _addr(topk_w, F32, "w", dev, gw.shape)
    glogits, po = _out(glogits, (T, E), gw, "glogits", dev, stream)
    if T:
        rc = lib().r9k_moe_route_backward(pg, pi, pw, T, E, topk, po, _raw(stream, dev))
        if rc:
            _check(rc, "r9k_moe_route_backward")
    return glogits
