"""Python binding of the C ABI in include/fp8gemm.h (ctypes; marshalling only).

Every function takes torch CUDA tensors in the library's layouts, passes their
device pointers and the current CUDA stream to libfp8gemm.so, and raises if the
library returns an error.  No step of the GEMM runs in Python or on the CPU; if
the shared library is missing, importing this module raises.
"""
from __future__ import annotations

import ctypes as C
import math
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8gemm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m fp8_block_scaled_x128_b200.build` "
        "(the library has no CPU fallback)")

_P, _I, _U32, _F = C.c_void_p, C.c_int, C.c_uint32, C.c_float

lib = C.CDLL(LIB_PATH)
lib.fp8_gemm_nt.restype = _I
lib.fp8_gemm_nt.argtypes = [_P, _P, _I, _P, _P, _P, _I, _I, _I, _P]
lib.m_grouped_fp8_gemm_nt_contiguous.restype = _I
lib.m_grouped_fp8_gemm_nt_contiguous.argtypes = [_P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P]
lib.m_grouped_fp8_gemm_nt_masked.restype = _I
lib.m_grouped_fp8_gemm_nt_masked.argtypes = [_P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]
lib.fp8_gemm_nt_no_alloc.restype = _I
lib.fp8_gemm_nt_no_alloc.argtypes = [_P, _P, _I, _P, _P, _P, _I, _I, _I, _P]
lib.fp8g_sa_to_mn_major.restype = _I
lib.fp8g_sa_to_mn_major.argtypes = [_P, _P, _I, _I, _I, _I]
lib.fp8g_quantize_1x128.restype = _I
lib.fp8g_quantize_1x128.argtypes = [_P, _I, _I, _I, _P, _P, _I, _P]
lib.fp8g_quantize_128x128.restype = _I
lib.fp8g_quantize_128x128.argtypes = [_P, _I, _I, _I, _P, _P, _P]
lib.fp8g_testing_withhold_stage.restype = _I
lib.fp8g_testing_withhold_stage.argtypes = [_I, C.c_uint]
lib.fp8g_testing_withhold_sum.restype = _I
lib.fp8g_testing_withhold_sum.argtypes = [_I, C.c_uint]
lib.fp8g_moe_dispatch_workspace_bytes.restype = C.c_size_t
lib.fp8g_moe_dispatch_workspace_bytes.argtypes = [_I, _I]
lib.fp8g_moe_dispatch.restype = _I
lib.fp8g_moe_dispatch.argtypes = [_P, _I, _I, _I, _P, _I, _I, _I, _P, _P, _I, _P, _P, _P, C.c_size_t, _P]
lib.fp8g_moe_combine.restype = _I
lib.fp8g_moe_combine.argtypes = [_P, _I, _P, _P, _I, _I, _P, _P]
lib.fp8g_moe_dispatch_masked.restype = _I
lib.fp8g_moe_dispatch_masked.argtypes = [_P, _I, _I, _I, _P, _I, _I, _I, _P, _P, _I, _P, _P, _P]
lib.fp8g_moe_permute.restype = _I
lib.fp8g_moe_permute.argtypes = [_P, _I, _I, _I, _P, _I, _I, _I, _P, _P, _P, _P]
lib.fp8g_moe_permute_backward.restype = _I
lib.fp8g_moe_permute_backward.argtypes = [_P, _I, _I, _I, _P, _I, _I, _P, _P]
lib.fp8g_moe_combine_backward.restype = _I
lib.fp8g_moe_combine_backward.argtypes = [_P, _P, _I, _P, _P, _I, _I, _I, _P, _P, _P, _I, _P, _P]
lib.fp8g_norm_residual.restype = _I
lib.fp8g_norm_residual.argtypes = [_P, _P, _I, _I, _I, _P, _P, _I, _F, _P, _F, _P, _P, _P, _P, _I, _P]
lib.fp8g_norm_residual_backward_workspace_bytes.restype = C.c_size_t
lib.fp8g_norm_residual_backward_workspace_bytes.argtypes = [_I, _I]
lib.fp8g_norm_residual_backward.restype = _I
lib.fp8g_norm_residual_backward.argtypes = [_P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _F, _P, _F, _P, _P, _P, _P, _P, _P,
                                            C.c_size_t, _P]
lib.bf16_gemm_nt.restype = _I
lib.bf16_gemm_nt.argtypes = [_P, _P, _P, _I, _I, _I, _P]
lib.fp8_gemm_nt_ue8m0.restype = _I
lib.fp8_gemm_nt_ue8m0.argtypes = [_P, _P, _I, _P, _P, _P, _I, _I, _I, _P]
lib.fp8g_status_string.restype = C.c_char_p
lib.fp8g_status_string.argtypes = [_I]
lib.fp8g_get_device_error.restype = _I
lib.fp8g_get_device_error.argtypes = [_I, C.POINTER(_U32), _I]
lib.fp8g_set_variant_override.restype = _I
lib.fp8g_set_variant_override.argtypes = [_I]
lib.fp8g_num_variants.restype = _I
lib.fp8g_num_variants.argtypes = []
lib.fp8g_variant_name.restype = C.c_char_p
lib.fp8g_variant_name.argtypes = [_I]
lib.fp8g_last_variant.restype = _I
lib.fp8g_last_variant.argtypes = []
lib.fp8g_version.restype = _I
lib.fp8g_version.argtypes = []

DEVERR_TIMEOUT, DEVERR_BAD_M_INDEX, DEVERR_MASKED_OVER, DEVERR_BAD_EXPERT = 0x1, 0x2, 0x4, 0x8
DEVERR_BAD_POS = 0x10


class Fp8GemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib.fp8g_status_string(status).decode()} (status {status})")


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise Fp8GemmError(rc, what)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream, device):
    s = torch.cuda.current_stream(device) if stream is None else stream
    if s.device != device:
        raise ValueError(f"stream is on {s.device}, the operands on {device}")
    return C.c_void_p(s.cuda_stream)


def _dev(t, dt, name):
    if not t.is_cuda or t.dtype != dt or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous CUDA tensor of {dt}, got {t.dtype} on {t.device}")
    return t


def _one_device(**tensors):
    """The device every operand lives on.  The library encodes its tensor maps
    and launches on the current device, so the call runs under this device and
    operands on different devices are refused before anything is launched."""
    devs = {name: t.device for name, t in tensors.items()}
    first = next(iter(devs.values()))
    for name, d in devs.items():
        if d != first:
            raise ValueError(f"all operands must be on one device: {name} is on {d}, "
                             f"{next(iter(devs))} on {first}")
    return first


def variant_names():
    return [lib.fp8g_variant_name(i).decode() for i in range(lib.fp8g_num_variants())]


def set_variant_override(v: int | None) -> None:
    _check(lib.fp8g_set_variant_override(-1 if v is None else int(v)), "fp8g_set_variant_override")


def testing_withhold_stage(iteration: int | None, wait_limit_us: int = 2000) -> None:
    """Test hook (include/fp8gemm_testing.h): from the next call on, the
    single-CTA kernels skip the loads of pipeline iteration `iteration` and
    give up on any wait after `wait_limit_us`; None turns it off."""
    _check(lib.fp8g_testing_withhold_stage(-1 if iteration is None else int(iteration), int(wait_limit_us)),
           "fp8g_testing_withhold_stage")


def testing_withhold_sum(call: int | None, wait_limit_us: int = 2000) -> None:
    """Test hook (include/fp8gemm_testing.h): from the next call on, the last CTA
    of a norm's cluster waits in exchange `call` (0 or 1) for an arrival that never
    comes, and waits for sums give up after `wait_limit_us`; None turns it off."""
    _check(lib.fp8g_testing_withhold_sum(-1 if call is None else int(call), int(wait_limit_us)),
           "fp8g_testing_withhold_sum")


def last_variant() -> int:
    return lib.fp8g_last_variant()


def device_error(clear: bool = True, device: int | None = None) -> int:
    """The device error word (FP8G_DEVERR_* bits); synchronises the device."""
    bits = _U32(0)
    d = torch.cuda.current_device() if device is None else device
    rc = lib.fp8g_get_device_error(int(d), C.byref(bits), int(clear))
    if rc not in (0, 5):
        raise Fp8GemmError(rc, "fp8g_get_device_error")
    return bits.value


def fp8_gemm_nt(A, sa, B, sb, D=None, stream=None):
    """Dense: A [M,K] uint8 (e4m3 codes), sa [K/128, ld_sa] float32, B [N,K] uint8,
    sb [ceil(N/128), K/128] float32 -> D [M,N] bfloat16."""
    M, K = A.shape
    N = B.shape[0]
    _dev(A, torch.uint8, "A"), _dev(B, torch.uint8, "B")
    _dev(sa, torch.float32, "sa"), _dev(sb, torch.float32, "sb")
    if D is None:
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _dev(D, torch.bfloat16, "D")
    dev = _one_device(A=A, sa=sa, B=B, sb=sb, D=D)
    with torch.cuda.device(dev):
        _check(lib.fp8_gemm_nt(_ptr(A), _ptr(sa), sa.shape[1], _ptr(B), _ptr(sb), _ptr(D), M, N, K,
                               _stream(stream, dev)), "fp8_gemm_nt")
    return D


def m_grouped_fp8_gemm_nt_contiguous(A, sa, B, sb, m_indices, D=None, stream=None):
    """Contiguous: A [M,K], sa [K/128, ld_sa], B [G,N,K], sb [G, ceil(N/128), K/128],
    m_indices [M/128] int32 -> D [M,N] bfloat16 (rows of -1 blocks untouched)."""
    M, K = A.shape
    G, N, _ = B.shape
    _dev(A, torch.uint8, "A"), _dev(B, torch.uint8, "B"), _dev(m_indices, torch.int32, "m_indices")
    _dev(sa, torch.float32, "sa"), _dev(sb, torch.float32, "sb")
    if D is None:
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _dev(D, torch.bfloat16, "D")
    dev = _one_device(A=A, sa=sa, B=B, sb=sb, D=D, m_indices=m_indices)
    with torch.cuda.device(dev):
        _check(lib.m_grouped_fp8_gemm_nt_contiguous(_ptr(A), _ptr(sa), sa.shape[1], _ptr(B), _ptr(sb), _ptr(D),
                                                    _ptr(m_indices), M, N, K, G, _stream(stream, dev)),
               "m_grouped_fp8_gemm_nt_contiguous")
    return D


def m_grouped_fp8_gemm_nt_masked(A, sa, B, sb, masked_m, expected_m, D=None, stream=None):
    """Masked: A [G,Mmax,K], sa [G, K/128, ld_sa], B [G,N,K], sb [G, ceil(N/128), K/128],
    masked_m [G] int32 (device) -> D [G,Mmax,N] bfloat16 (rows >= masked_m[g] untouched)."""
    G, Mmax, K = A.shape
    N = B.shape[1]
    _dev(A, torch.uint8, "A"), _dev(B, torch.uint8, "B"), _dev(masked_m, torch.int32, "masked_m")
    _dev(sa, torch.float32, "sa"), _dev(sb, torch.float32, "sb")
    if D is None:
        D = torch.empty((G, Mmax, N), dtype=torch.bfloat16, device=A.device)
    _dev(D, torch.bfloat16, "D")
    dev = _one_device(A=A, sa=sa, B=B, sb=sb, D=D, masked_m=masked_m)
    with torch.cuda.device(dev):
        _check(lib.m_grouped_fp8_gemm_nt_masked(_ptr(A), _ptr(sa), sa.shape[2], _ptr(B), _ptr(sb), _ptr(D),
                                                _ptr(masked_m), G, Mmax, N, K, int(expected_m),
                                                _stream(stream, dev)), "m_grouped_fp8_gemm_nt_masked")
    return D


def fp8_gemm_nt_no_alloc(A, sa, B, sb, D=None, stream=None):
    """Dense GEMM like fp8_gemm_nt, for callers that must not allocate device
    memory while they run it (the library keeps this path's split-K scratch in
    a fixed array of its own).  Decode shapes only: at most 160 tiles of 128
    rows of B by 64 rows of A.  Pass D to avoid the output allocation here;
    calls that overlap on the GPU share the scratch and must be ordered."""
    M, K = A.shape
    N = B.shape[0]
    _dev(A, torch.uint8, "A"), _dev(B, torch.uint8, "B")
    _dev(sa, torch.float32, "sa"), _dev(sb, torch.float32, "sb")
    if D is None:
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _dev(D, torch.bfloat16, "D")
    dev = _one_device(A=A, sa=sa, B=B, sb=sb, D=D)
    with torch.cuda.device(dev):
        _check(lib.fp8_gemm_nt_no_alloc(_ptr(A), _ptr(sa), sa.shape[1], _ptr(B), _ptr(sb), _ptr(D), M, N, K,
                                        _stream(stream, dev)), "fp8_gemm_nt_no_alloc")
    return D


def sa_to_mn_major(sa_rows, ld_sa=None):
    """Host helper: A's scales from [rows, KB] (or [G, rows, KB]) float32 to the
    library's MN-major [KB, ld_sa] (or [G, KB, ld_sa]) layout, as a numpy array.
    ld_sa defaults to rows rounded up to a multiple of 4."""
    import numpy as np
    src = np.ascontiguousarray(sa_rows, dtype=np.float32)
    grouped = src.ndim == 3
    if not grouped:
        src = src[None]
    G, rows, KB = src.shape
    ld = max(4, (rows + 3) // 4 * 4) if ld_sa is None else int(ld_sa)
    dst = np.empty((G, KB, ld), np.float32)
    _check(lib.fp8g_sa_to_mn_major(src.ctypes.data_as(_P), dst.ctypes.data_as(_P), G, rows, KB, ld),
           "fp8g_sa_to_mn_major")
    return dst if grouped else dst[0]


_IN_DTYPE = {torch.bfloat16: 0, torch.float32: 1}


def _quant_input(x):
    if not x.is_cuda or x.dtype not in _IN_DTYPE or not x.is_contiguous() or x.dim() != 2:
        raise TypeError(f"x: expected a contiguous 2-D CUDA tensor of bfloat16 or float32, got {x.dtype} "
                        f"{tuple(x.shape)} on {x.device}")
    return x


def quantize_1x128(x, q=None, sa=None, ld_sa=None, stream=None):
    """Activations x [rows, K] (bfloat16 or float32) -> (q [rows, K] uint8 e4m3
    codes, sa [K/128, ld_sa] float32 scales, one per 1x128 group), the GEMM's
    A-side inputs.  ld_sa defaults to rows rounded up to a multiple of 4."""
    _quant_input(x)
    rows, K = x.shape
    ld = max(4, (rows + 3) // 4 * 4) if ld_sa is None else int(ld_sa)
    if q is None:
        q = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
    if sa is None:
        sa = torch.zeros((max(1, K // 128), ld), dtype=torch.float32, device=x.device)
    _dev(q, torch.uint8, "q"), _dev(sa, torch.float32, "sa")
    dev = _one_device(x=x, q=q, sa=sa)
    with torch.cuda.device(dev):
        _check(lib.fp8g_quantize_1x128(_ptr(x), _IN_DTYPE[x.dtype], rows, K, _ptr(q), _ptr(sa), sa.shape[-1],
                                       _stream(stream, dev)), "fp8g_quantize_1x128")
    return q, sa


def quantize_128x128(x, q=None, sb=None, stream=None):
    """Weights x [N, K] (bfloat16 or float32) -> (q [N, K] uint8 e4m3 codes,
    sb [ceil(N/128), K/128] float32 scales, one per 128x128 block)."""
    _quant_input(x)
    N, K = x.shape
    if q is None:
        q = torch.empty((N, K), dtype=torch.uint8, device=x.device)
    if sb is None:
        sb = torch.empty(((N + 127) // 128, max(1, K // 128)), dtype=torch.float32, device=x.device)
    _dev(q, torch.uint8, "q"), _dev(sb, torch.float32, "sb")
    dev = _one_device(x=x, q=q, sb=sb)
    with torch.cuda.device(dev):
        _check(lib.fp8g_quantize_128x128(_ptr(x), _IN_DTYPE[x.dtype], N, K, _ptr(q), _ptr(sb),
                                         _stream(stream, dev)), "fp8g_quantize_128x128")
    return q, sb


def moe_blocks(T: int, topk: int, G: int) -> int:
    """128-row blocks of A that fit any routing of T*topk rows to G experts."""
    return (T * topk + 127) // 128 + G


def moe_dispatch(x, expert, topk, G, blocks=None, out=None, stream=None):
    """Expert dispatch before the contiguous GEMM: x [T, K] (bfloat16 or float32),
    expert [T*topk] int32 (-1 = dropped) -> (A [blocks*128, K] uint8, sa [K/128,
    blocks*128] float32, pos [T*topk] int32, m_indices [blocks] int32).  `out`
    may pass those four tensors (and a workspace as a fifth) to reuse them."""
    _quant_input(x)
    T, K = x.shape
    R = T * topk
    _dev(expert, torch.int32, "expert")
    if expert.numel() != R:
        raise ValueError(f"expert: {expert.numel()} entries for {T} tokens x topk {topk}")
    nb = moe_blocks(T, topk, G) if blocks is None else int(blocks)
    ws_bytes = lib.fp8g_moe_dispatch_workspace_bytes(R, G)
    if ws_bytes == 0:
        raise ValueError(f"moe_dispatch: unsupported R={R}, G={G} (1 <= G <= 256)")
    if out is None:
        A = torch.empty((nb * 128, K), dtype=torch.uint8, device=x.device)
        sa = torch.empty((K // 128, nb * 128), dtype=torch.float32, device=x.device)
        pos = torch.empty(max(R, 1), dtype=torch.int32, device=x.device)
        mi = torch.empty(nb, dtype=torch.int32, device=x.device)
        ws = torch.empty((ws_bytes + 3) // 4, dtype=torch.int32, device=x.device)
    else:
        A, sa, pos, mi, ws = out
    dev = _one_device(x=x, expert=expert, A=A, sa=sa, pos=pos, m_indices=mi, workspace=ws)
    with torch.cuda.device(dev):
        _check(lib.fp8g_moe_dispatch(_ptr(x), _IN_DTYPE[x.dtype], T, K, _ptr(expert), int(topk), int(G), nb,
                                     _ptr(A), _ptr(sa), sa.shape[-1], _ptr(pos), _ptr(mi), _ptr(ws),
                                     ws.numel() * 4, _stream(stream, dev)), "fp8g_moe_dispatch")
    return A, sa, pos[:R], mi


def moe_combine(D, pos, w, T, topk, out=None, stream=None):
    """Combine after the GEMM: out [T, N] bfloat16 = sum over slots of w * D[pos]
    (FP32, one fused multiply-add per slot in slot order); w may be None."""
    _dev(D, torch.bfloat16, "D"), _dev(pos, torch.int32, "pos")
    N = D.shape[-1]
    if w is not None:
        _dev(w, torch.float32, "w")
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=D.device)
    _dev(out, torch.bfloat16, "out")
    tensors = dict(D=D, pos=pos, out=out)
    if w is not None:
        tensors["w"] = w
    dev = _one_device(**tensors)
    with torch.cuda.device(dev):
        _check(lib.fp8g_moe_combine(_ptr(D), N, _ptr(pos), _ptr(w), int(T), int(topk), _ptr(out),
                                    _stream(stream, dev)), "fp8g_moe_combine")
    return out


def _operand(t, dt, shape, index, name):
    """t, if it is a contiguous CUDA tensor of this type and shape (a tuple) on
    device `index`.  One short check per operand: these calls are made per layer
    and decoded token."""
    if t.dtype != dt or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        if t.is_cuda and t.get_device() != index:
            raise ValueError(f"all operands must be on one device: {name} is on {t.device}, expected cuda:{index}")
        raise TypeError(f"{name}: expected a contiguous CUDA tensor of {dt} {tuple(shape)}, got {t.dtype} "
                        f"{tuple(t.shape)} on {t.device}")
    return t


def _slots(t, R, index, name):
    """t, if it is a contiguous int32 CUDA tensor of R routed slots, flat or [T, topk]."""
    return _operand(t, torch.int32, (R,) if t.dim() == 1 or math.prod(t.shape) != R else t.shape, index, name)


def _rows(t, name):
    """The device index of t, if it is a contiguous 2-D CUDA tensor of activations."""
    if t.dtype not in _IN_DTYPE or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous 2-D CUDA tensor of bfloat16 or float32, got {t.dtype} "
                        f"{tuple(t.shape)} on {t.device}")
    return t.get_device()


# the current device and the raw handle of its current stream, without torch.cuda's
# Stream object and initialisation check where torch has the short way
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(index, stream):
    """What to enter before a call whose operands are on device `index`, or None
    if that is the current device and no stream is given.  Under a given stream,
    what the call allocates belongs to the stream it runs on."""
    if stream is None:
        return None if index == _current_device() else torch.cuda.device(index)
    if stream.device != torch.device("cuda", index):
        raise ValueError(f"stream is on {stream.device}, the operands on cuda:{index}")
    return torch.cuda.stream(stream)


def _addr(t):
    return None if t is None else t.data_ptr()


def moe_dispatch_masked(x, expert, topk, G, Mmax, out=None, stream=None):
    """Expert dispatch before the masked GEMM: x [T, K] (bfloat16 or float32),
    expert [T*topk] or [T, topk] int32 (-1 = dropped) -> (A [G, Mmax, K] uint8,
    sa [G, K/128, ld_sa] float32, pos [T*topk] int32, masked_m [G] int32).  pos
    is the slot's row of D seen as [G*Mmax, N], for moe_combine; slots past an
    expert's Mmax rows are dropped and flagged (DEVERR_MASKED_OVER).  Rows behind
    masked_m are not written.  `out` may pass those four tensors to reuse them."""
    dev = _rows(x, "x")
    T, K = x.shape
    topk, G, Mmax = int(topk), int(G), int(Mmax)
    R = T * topk
    _slots(expert, R, dev, "expert")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_dispatch_masked(x, expert, topk, G, Mmax, out)
    raw = _current_raw(dev)
    if out is None:
        ld = (Mmax + 3) // 4 * 4
        out = (torch.empty((G, Mmax, K), dtype=torch.uint8, device=x.device),
               torch.empty((G, K // 128, ld), dtype=torch.float32, device=x.device),
               torch.empty(R, dtype=torch.int32, device=x.device), torch.empty(G, dtype=torch.int32, device=x.device))
        A, sa, pos, masked_m = out
    else:
        A, sa, pos, masked_m = out
        _operand(A, torch.uint8, (G, Mmax, K), dev, "A")
        _operand(sa, torch.float32, (G, K // 128, sa.shape[-1]), dev, "sa")
        _operand(pos, torch.int32, (R,), dev, "pos"), _operand(masked_m, torch.int32, (G,), dev, "masked_m")
    _check(lib.fp8g_moe_dispatch_masked(x.data_ptr(), _IN_DTYPE[x.dtype], T, K, expert.data_ptr(), topk, G, Mmax,
                                        A.data_ptr(), sa.data_ptr(), sa.shape[-1], pos.data_ptr(),
                                        masked_m.data_ptr(), raw), "fp8g_moe_dispatch_masked")
    return A, sa, pos, masked_m


def moe_permute(x, expert, topk, G, blocks=None, out=None, stream=None):
    """Expert sort without quantisation, in moe_dispatch's contiguous layout: x
    [T, N] (bfloat16 or float32), expert [T*topk] or [T, topk] int32 (-1 =
    dropped) -> (xs [blocks*128, N] of x's type, pos [T*topk] int32, m_indices
    [blocks] int32).
    Padding rows of a segment are zero; unused blocks are not written.  `out`
    may pass those three tensors to reuse them."""
    dev = _rows(x, "x")
    T, N = x.shape
    topk, G = int(topk), int(G)
    R = T * topk
    _slots(expert, R, dev, "expert")
    nb = moe_blocks(T, topk, G) if blocks is None else int(blocks)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_permute(x, expert, topk, G, blocks, out)
    raw = _current_raw(dev)
    if out is None:
        out = (torch.empty((nb * 128, N), dtype=x.dtype, device=x.device),
               torch.empty(R, dtype=torch.int32, device=x.device), torch.empty(nb, dtype=torch.int32, device=x.device))
    xs, pos, mi = out
    _operand(xs, x.dtype, (nb * 128, N), dev, "xs")
    _operand(pos, torch.int32, (R,), dev, "pos"), _operand(mi, torch.int32, (nb,), dev, "m_indices")
    _check(lib.fp8g_moe_permute(x.data_ptr(), _IN_DTYPE[x.dtype], T, N, expert.data_ptr(), topk, G, nb,
                                xs.data_ptr(), pos.data_ptr(), mi.data_ptr(), raw), "fp8g_moe_permute")
    return xs, pos, mi


def moe_permute_backward(dxs, pos, T, topk, out=None, stream=None):
    """Gradient of moe_permute (and of moe_dispatch, its quantisation taken as
    the identity): dx [T, N] = sum over a token's slots of dxs[pos] (FP32 in
    slot order, rounded once).  dxs [blocks*128, N] bfloat16 or float32; pos
    [T*topk] or [T, topk]."""
    dev = _rows(dxs, "dxs")
    M, N = dxs.shape
    T, topk = int(T), int(topk)
    _layout_rows(M, "dxs")
    _slots(pos, T * topk, dev, "pos")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_permute_backward(dxs, pos, T, topk, out)
    raw = _current_raw(dev)
    if out is None:
        dx = torch.empty_strided((T, N), (N, 1), dtype=dxs.dtype, device=dxs.device)
    else:
        dx = _operand(out, dxs.dtype, (T, N), dev, "out")
    _check(lib.fp8g_moe_permute_backward(dxs.data_ptr(), _IN_DTYPE[dxs.dtype], M // 128, N, pos.data_ptr(), T,
                                         topk, dx.data_ptr(), raw), "fp8g_moe_permute_backward")
    return dx


def _layout_rows(M, name):
    if M % 128 != 0:
        raise ValueError(f"{name}: {M} rows are not whole 128-row blocks")


def moe_combine_backward(dout, D, pos, w, T, topk, quantize=False, out=None, stream=None):
    """Gradient of moe_combine: dout [T, N], D [blocks*128, N] bfloat16, pos
    [T*topk] or [T, topk], w [T*topk] float32 or None -> (dD, dw), dD [blocks*128, N] bfloat16 with
    dD[pos] = w * dout, dw [T*topk] float32 = <dout, D[pos]> (0 for dropped
    slots; None if w is None).  quantize=True gives (q, sa, dw) instead: e4m3
    codes and [N/128, ld_sa] scales, the A side of the grouped GEMM that
    follows.  Unfilled rows of used blocks are zero, unused blocks are not
    written.  `out` may pass the returned tensors to reuse them."""
    T, topk = int(T), int(topk)
    _dev(D, torch.bfloat16, "D")
    M, N = D.shape
    _layout_rows(M, "D")
    dev = D.get_device()
    _operand(dout, torch.bfloat16, (T, N), dev, "dout"), _slots(pos, T * topk, dev, "pos")
    if w is not None:
        _operand(w, torch.float32, (T * topk,), dev, "w")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_combine_backward(dout, D, pos, w, T, topk, quantize, out)
    raw = _current_raw(dev)
    if out is None:
        dw = None if w is None else torch.empty(T * topk, dtype=torch.float32, device=D.device)
        if quantize:
            out = (torch.empty((M, N), dtype=torch.uint8, device=D.device),
                   torch.empty((N // 128, max(M, 4)), dtype=torch.float32, device=D.device), dw)
        else:
            out = (torch.empty((M, N), dtype=torch.bfloat16, device=D.device), dw)
    q = sa = dD = None
    if quantize:
        q, sa, dw = out
        _operand(q, torch.uint8, (M, N), dev, "q"), _operand(sa, torch.float32, (N // 128, sa.shape[-1]), dev, "sa")
    else:
        dD, dw = out
        _operand(dD, torch.bfloat16, (M, N), dev, "dD")
    if (dw is None) != (w is None):
        raise ValueError("dw: an output exactly if w is given")
    if dw is not None:
        _operand(dw, torch.float32, (T * topk,), dev, "dw")
    _check(lib.fp8g_moe_combine_backward(dout.data_ptr(), D.data_ptr(), N, pos.data_ptr(), _addr(w), T, topk,
                                         M // 128, _addr(dD), _addr(q), _addr(sa),
                                         0 if sa is None else sa.shape[-1], _addr(dw), raw),
           "fp8g_moe_combine_backward")
    return out


def _norm_params(y, post_weight, gate, pre_weight):
    """Checks the parameters of rows y; the kind of the gate."""
    (rows, H), dev = y.shape, y.get_device()
    if post_weight is not None:
        _operand(post_weight, torch.float32, (H,), dev, "post_weight")
    if pre_weight is not None:
        _operand(pre_weight, torch.float32, (H,), dev, "pre_weight")
    if gate is None:
        return 0
    if gate.dim() == 1:
        _operand(gate, torch.float32, (H,), dev, "gate")
        return 1
    _operand(gate, torch.float32, (rows, 1), dev, "gate")
    return 2


def norm_residual(y, h=None, post_weight=None, gate=None, scale=1.0, pre_weight=None, eps=1e-6, quantize=False,
                  out=None, stream=None):
    """The norms around a block with its gate, residual scale and residual sum:
    h_out = h + scale * gate * post_weight * y / rms(y), z = pre_weight * h_out /
    rms(h_out), rms(x) = sqrt(mean(x^2) + eps) -> (h_out, z), or (h_out, q, sa)
    with quantize=True: z's e4m3 codes and [H/128, ld_sa] scales, the GEMM's
    A-side inputs.  y, h [rows, H] bfloat16 or float32 (h None: no residual);
    post_weight, pre_weight [H] float32 (post_weight None: no post-norm,
    pre_weight None: ones); gate float32 [H] (per channel) or [rows, 1] (per
    token).  `out` may pass the returned tensors; h_out may be h, z may be y."""
    dev = _rows(y, "y")
    rows, H = y.shape
    if h is not None:
        _operand(h, y.dtype, (rows, H), dev, "h")
    kind = _norm_params(y, post_weight, gate, pre_weight)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return norm_residual(y, h, post_weight, gate, scale, pre_weight, eps, quantize, out)
    raw = _current_raw(dev)
    z = q = sa = None
    if out is None:
        h_out = torch.empty_like(y)
        if quantize:
            q = torch.empty_like(y, dtype=torch.uint8)
            sa = torch.zeros((max(1, H // 128), max(4, (rows + 3) // 4 * 4)), dtype=torch.float32, device=y.device)
        else:
            z = torch.empty_like(y)
    else:
        if quantize:
            h_out, q, sa = out
            _operand(q, torch.uint8, (rows, H), dev, "q")
            _operand(sa, torch.float32, (H // 128, sa.shape[-1]), dev, "sa")
        else:
            h_out, z = out
            _operand(z, y.dtype, (rows, H), dev, "z")
        _operand(h_out, y.dtype, (rows, H), dev, "h_out")
    _check(lib.fp8g_norm_residual(y.data_ptr(), _addr(h), _IN_DTYPE[y.dtype], rows, H, _addr(post_weight),
                                  _addr(gate), kind, float(scale), _addr(pre_weight), float(eps), h_out.data_ptr(), _addr(z),
                                  _addr(q), _addr(sa), 0 if sa is None else sa.shape[-1], raw),
           "fp8g_norm_residual")
    return (h_out, q, sa) if quantize else (h_out, z)


def norm_residual_backward(dz, dh_out, h_out, y, post_weight=None, gate=None, scale=1.0, pre_weight=None, eps=1e-6,
                           out=None, workspace=None, stream=None):
    """Gradients of norm_residual from those of z and h_out (either may be None):
    (dh, dy, dpre_weight, dpost_weight, dgate), the last three float32 in their
    parameters' shapes, None where the parameter is None.  h_out and y are the
    forward pass's.  `out` may pass the five tensors to reuse them (dh may be
    dh_out), `workspace` float32 scratch of at least
    fp8g_norm_residual_backward_workspace_bytes(rows, H) bytes (of the largest
    batch, to keep one for all)."""
    dev = _rows(y, "y")
    rows, H = y.shape
    _operand(h_out, y.dtype, (rows, H), dev, "h_out")
    for name, t in (("dz", dz), ("dh_out", dh_out)):
        if t is not None:
            _operand(t, y.dtype, (rows, H), dev, name)
    kind = _norm_params(y, post_weight, gate, pre_weight)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return norm_residual_backward(dz, dh_out, h_out, y, post_weight, gate, scale, pre_weight, eps, out,
                                          workspace)
    raw = _current_raw(dev)
    if out is None:
        dh, dy = torch.empty_like(y), torch.empty_like(y)
        dpre = None if pre_weight is None else torch.empty_like(pre_weight)
        dpost = None if post_weight is None else torch.empty_like(post_weight)
        dgate = None if gate is None else torch.empty_like(gate)
    else:
        dh, dy, dpre, dpost, dgate = out
        _operand(dh, y.dtype, (rows, H), dev, "dh"), _operand(dy, y.dtype, (rows, H), dev, "dy")
        for name, p, d in (("dpre_weight", pre_weight, dpre), ("dpost_weight", post_weight, dpost),
                           ("dgate", gate, dgate)):
            if (p is None) != (d is None):
                raise ValueError(f"{name}: an output exactly if its parameter is given")
            if d is not None:
                _operand(d, torch.float32, p.shape, dev, name)
    if workspace is not None:
        _operand(workspace, torch.float32, workspace.shape, dev, "workspace")
    elif kind == 1 or pre_weight is not None or post_weight is not None:
        need = lib.fp8g_norm_residual_backward_workspace_bytes(rows, H) // 4
        workspace = torch.empty_strided((need,), (1,), dtype=torch.float32, device=y.device)
    _check(lib.fp8g_norm_residual_backward(_addr(dz), _addr(dh_out), h_out.data_ptr(), y.data_ptr(),
                                           _IN_DTYPE[y.dtype], rows, H, _addr(post_weight), _addr(gate), kind,
                                           float(scale), _addr(pre_weight), float(eps), dh.data_ptr(), dy.data_ptr(), _addr(dpre),
                                           _addr(dpost), _addr(dgate), _addr(workspace),
                                           0 if workspace is None else workspace.numel() * 4, raw),
           "fp8g_norm_residual_backward")
    return dh, dy, dpre, dpost, dgate


def bf16_gemm_nt(A, B, D=None, stream=None):
    """BF16 NT GEMM: A [M, K], B [N, K] bfloat16 -> D [M, N] bfloat16 (FP32 accumulation)."""
    _dev(A, torch.bfloat16, "A"), _dev(B, torch.bfloat16, "B")
    M, K = A.shape
    N = B.shape[0]
    if D is None:
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _dev(D, torch.bfloat16, "D")
    dev = _one_device(A=A, B=B, D=D)
    with torch.cuda.device(dev):
        _check(lib.bf16_gemm_nt(_ptr(A), _ptr(B), _ptr(D), M, N, K, _stream(stream, dev)), "bf16_gemm_nt")
    return D


def fp8_gemm_nt_ue8m0(A, sfa, B, sfb, D=None, stream=None):
    """Dense NT GEMM with power-of-two scales: A [M,K] uint8 e4m3, sfa [K/128, ld]
    uint8 (E8M0: 2^(e-127)), B [N,K] uint8, sfb [ceil(N/128), K/128] uint8 ->
    D [M,N] bfloat16 (block-scaled tensor-core MMA, FP32 accumulation over K)."""
    M, K = A.shape
    N = B.shape[0]
    _dev(A, torch.uint8, "A"), _dev(B, torch.uint8, "B"), _dev(sfa, torch.uint8, "sfa"), _dev(sfb, torch.uint8, "sfb")
    if D is None:
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _dev(D, torch.bfloat16, "D")
    dev = _one_device(A=A, sfa=sfa, B=B, sfb=sfb, D=D)
    with torch.cuda.device(dev):
        _check(lib.fp8_gemm_nt_ue8m0(_ptr(A), _ptr(sfa), sfa.shape[1], _ptr(B), _ptr(sfb), _ptr(D), M, N, K,
                                     _stream(stream, dev)), "fp8_gemm_nt_ue8m0")
    return D
