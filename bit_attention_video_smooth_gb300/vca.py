"""Thin ctypes binding of ``libvca.so`` (the C ABI in ``include/vca.h``).

The functions keep the C entry points' names and only marshal arguments:
PyTorch tensors provide device memory and the current CUDA stream; every step
of the computation runs in the library's CUDA kernels.  If the library has not
been built (``__graft_entry__.build()`` or ``python
bit_attention_video_smooth_gb300/build.py``) importing this module raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libvca.so")

VCA_OK, VCA_ERR_INVALID_ARG, VCA_ERR_UNSUPPORTED, VCA_ERR_CUDA, VCA_ERR_TIMEOUT, VCA_ERR_WORKSPACE, VCA_ERR_FULL = range(7)
VCA_V_E4M3, VCA_V_NVFP4 = 0, 1
VCA_OP_GROUP, VCA_OP_PREP, VCA_OP_ATTENTION, VCA_OP_PREP_KSMOOTH = 0, 1, 2, 3
VCA_OP_CACHE_ATTENTION, VCA_OP_CACHE_WEIGH = 4, 5

# Entry points declared in include/vca.h (the ABI test checks they are exported).
EXPORTS = ("vca_status_string", "vca_version", "vca_workspace_bytes", "vca_group", "vca_prep_quant",
           "vca_attention", "vca_expcast_codes", "vca_e4m3_encode_bits", "vca_selftest_timeout",
           "vca_set_wait_limit_ns", "vca_prep_quant_noalloc", "vca_prep_quant_ex",
           "vca_cache_workspace_bytes", "vca_cache_append", "vca_cache_append_ex", "vca_cache_attention",
           "vca_cache_weigh", "vca_cache_evict", "vca_cache_plan", "vca_cache_fresh", "vca_prompt_attention")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libvca.so is not built ({LIB_PATH}); run __graft_entry__.build() -- "
                      "there is no fallback implementation")

_lib = ctypes.CDLL(LIB_PATH)
_P, _I, _I64, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class _CacheStruct(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k8", "v8", "sk", "sv", "table", "len")] + \
        [(n, _I) for n in ("pages", "H", "d", "B", "cols")]


_C = ctypes.POINTER(_CacheStruct)
_SIGS = {
    "vca_status_string": (ctypes.c_char_p, [_I]),
    "vca_version": (_I, []),
    "vca_workspace_bytes": (_SZ, [_I] * 7),
    "vca_group": (_I, [_P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "vca_prep_quant": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "vca_attention": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _I, _P, _P, _P]),
    "vca_expcast_codes": (_I, [_P, _P, _P, _I64, _P, _P]),
    "vca_e4m3_encode_bits": (_I, [ctypes.c_uint32, _I64, _P, _P]),
    "vca_selftest_timeout": (_I, [_P, ctypes.c_uint64, _P]),
    "vca_set_wait_limit_ns": (None, [ctypes.c_uint64]),
    "vca_prep_quant_noalloc": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "vca_prep_quant_ex": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_uint32, _P, _P, _P, _P, _P, _P, _P, _P,
                               _P, _SZ, _P]),
    "vca_cache_workspace_bytes": (_SZ, [_I] * 6),
    "vca_cache_append": (_I, [_C, _P, _I64, _I64, _P, _I64, _I64, _P, _I, _P, _P]),
    "vca_cache_append_ex": (_I, [_C, _P, _I64, _I64, _P, _I64, _I64, _P, _I, _P, _P, _P]),
    "vca_cache_attention": (_I, [_C, _P, _I64, _I64, _P, _I, _I, _I, _F, _F, _P, _P, _P, _SZ, _P, _P]),
    "vca_cache_weigh": (_I, [_C, _P, _I64, _I64, _P, _I, _I, _I, _F, _F, _P, _P, _P, _SZ, _P, _P]),
    "vca_cache_evict": (_I, [_C, _P, _P, _I, _I, _I, _P, _P, _P, _P]),
    "vca_cache_plan": (_I, [_P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _I, _P, _P]),
    "vca_cache_fresh": (_I, [_P, _P, _I, _I, _I, _I, _P, _I, _P, _P]),
    "vca_prompt_attention": (_I, [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I, _I, _I, _I, _I, _I, _F, _F,
                                  _P, _P, _P, _P, _P, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class VCAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {vca_status_string(status)} ({status})")


def vca_status_string(status: int) -> str:
    return _lib.vca_status_string(int(status)).decode()


def vca_version() -> int:
    return int(_lib.vca_version())


def vca_workspace_bytes(op: int, B: int, H: int, N: int, d: int = 128, k: int = 1, vmode: int = 0) -> int:
    return int(_lib.vca_workspace_bytes(op, B, H, N, d, k, vmode))


def vca_set_wait_limit_ns(limit_ns: int) -> None:
    _lib.vca_set_wait_limit_ns(int(limit_ns))


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return ctypes.c_void_p(t.data_ptr())


def _buffers(where: str, need) -> torch.device:
    """The library sees plain pointers and cannot check what they point to, so
    the binding does: every (name, tensor, bytes) entry with a tensor must be
    contiguous and hold at least `bytes` bytes, and all of them must sit on one
    CUDA device, which is returned.  Sizes are checked first, so a call with
    host tensors of the right sizes fails only on the device check."""
    need = [(n, t, b) for n, t, b in need if t is not None]
    for name, t, nbytes in need:
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")
        have = t.numel() * t.element_size()
        if have < nbytes:
            raise ValueError(f"{where}: {name} holds {have} bytes, {nbytes} needed")
    for name, t, _ in need:
        if not t.is_cuda:
            raise ValueError(f"{where}: {name} is not a CUDA tensor")
    devs = {t.device for _, t, _ in need}
    if len(devs) != 1:
        raise ValueError(f"{where}: tensors on several devices {sorted(str(d) for d in devs)}")
    return devs.pop()


def _stream(stream=None, device=None):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, where: str) -> None:
    if status != VCA_OK:
        raise VCAError(status, where)


def _u16(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def vca_group(V: torch.Tensor, k: int, iters: int, labels: torch.Tensor, perm: torch.Tensor,
              counts: Optional[torch.Tensor], centroids: Optional[torch.Tensor], ws: torch.Tensor,
              dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    B, H, N, d = V.shape
    tok = B * H * N
    dev = _buffers("vca_group", [("V", V, 2 * tok * d), ("labels", labels, 4 * tok), ("perm", perm, 4 * tok),
                                 ("counts", counts, 4 * B * H * k), ("centroids", centroids, 4 * B * H * k * d),
                                 ("ws", ws, 0), ("dev_status", dev_status, 4)])
    with torch.cuda.device(dev):
        st = _lib.vca_group(_ptr(_u16(V)), B, H, N, d, k, iters, _ptr(labels), _ptr(perm), _ptr(counts),
                            _ptr(centroids), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status),
                            _stream(stream, dev))
    _check(st, "vca_group")


def vca_prep_quant(Q, K, V, perm, vmode: int, q8, sq, k8, sk, v_res, v_sf, v_scale, v_mean, ws,
                   stream=None) -> None:
    B, H, N, d = Q.shape
    dev = _prep_buffers("vca_prep_quant", B, H, N, d, vmode, Q, K, V, perm, q8, sq, k8, sk, v_res, v_sf, v_scale,
                        v_mean, ws=ws)
    with torch.cuda.device(dev):
        st = _lib.vca_prep_quant(_ptr(_u16(Q)), _ptr(_u16(K)), _ptr(_u16(V)), _ptr(perm), B, H, N, d, vmode,
                                 _ptr(q8), _ptr(sq), _ptr(k8), _ptr(sk), _ptr(v_res), _ptr(v_sf), _ptr(v_scale),
                                 _ptr(_u16(v_mean)), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream, dev))
    _check(st, "vca_prep_quant")


VCA_PREP_QK_HADAMARD = 1
VCA_PREP_K_SMOOTH = 2


def _prep_buffers(where, B, H, N, d, vmode, Q, K, V, perm, q8, sq, k8, sk, v_res, v_sf, v_scale, v_mean,
                  O=None, ws=None, dev_status=None):
    """Byte counts of the prep's inputs and outputs (the attention's operands)
    at this size and V format, checked against the tensors given."""
    BH, tok, nb = B * H, B * H * N, N // 128
    fp4 = vmode == VCA_V_NVFP4
    return _buffers(where, [
        ("Q", Q, 2 * tok * d), ("K", K, 2 * tok * d), ("V", V, 2 * tok * d), ("perm", perm, 4 * tok),
        ("q8", q8, tok * d), ("sq", sq, 4 * BH * nb), ("k8", k8, tok * d), ("sk", sk, 4 * BH * nb),
        ("v_res", v_res, tok * d // 2 if fp4 else tok * d), ("v_sf", v_sf, tok * d // 16 if fp4 else 0),
        ("v_scale", v_scale, 4 * BH if fp4 else 4 * BH * d), ("v_mean", v_mean, 2 * BH * nb * d),
        ("O", O, 2 * tok * d), ("ws", ws, 0), ("dev_status", dev_status, 4)])


def vca_prep_quant_ex(Q, K, V, perm, vmode: int, flags: int, q8, sq, k8, sk, v_res, v_sf, v_scale, v_mean, ws,
                      stream=None) -> None:
    B, H, N, d = Q.shape
    dev = _prep_buffers("vca_prep_quant_ex", B, H, N, d, vmode, Q, K, V, perm, q8, sq, k8, sk, v_res, v_sf,
                        v_scale, v_mean, ws=ws)
    with torch.cuda.device(dev):
        st = _lib.vca_prep_quant_ex(_ptr(_u16(Q)), _ptr(_u16(K)), _ptr(_u16(V)), _ptr(perm), B, H, N, d, vmode,
                                    flags, _ptr(q8), _ptr(sq), _ptr(k8), _ptr(sk), _ptr(v_res), _ptr(v_sf),
                                    _ptr(v_scale), _ptr(_u16(v_mean)), _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream(stream, dev))
    _check(st, "vca_prep_quant_ex")


def vca_prep_quant_noalloc(Q, K, V, perm, vmode: int, q8, sq, k8, sk, v_res, v_sf, v_scale, v_mean,
                           stream=None) -> None:
    """vca_prep_quant without a workspace argument: the scratch is a buffer built
    into the library (for callers that cannot provide device scratch memory).
    Calls that overlap on the GPU share that buffer and must be ordered."""
    B, H, N, d = Q.shape
    dev = _prep_buffers("vca_prep_quant_noalloc", B, H, N, d, vmode, Q, K, V, perm, q8, sq, k8, sk, v_res, v_sf,
                        v_scale, v_mean)
    with torch.cuda.device(dev):
        st = _lib.vca_prep_quant_noalloc(_ptr(_u16(Q)), _ptr(_u16(K)), _ptr(_u16(V)), _ptr(perm), B, H, N, d,
                                         vmode, _ptr(q8), _ptr(sq), _ptr(k8), _ptr(sk), _ptr(v_res), _ptr(v_sf),
                                         _ptr(v_scale), _ptr(_u16(v_mean)), _stream(stream, dev))
    _check(st, "vca_prep_quant_noalloc")


def vca_attention(q8, sq, k8, sk, v_res, v_sf, v_scale, v_mean, B: int, H: int, N: int, d: int,
                  softmax_scale: float, expcast: int, vmode: int, O, dev_status=None, stream=None) -> None:
    dev = _prep_buffers("vca_attention", B, H, N, d, vmode, None, None, None, None, q8, sq, k8, sk, v_res, v_sf,
                        v_scale, v_mean, O=O, dev_status=dev_status)
    with torch.cuda.device(dev):
        st = _lib.vca_attention(_ptr(q8), _ptr(sq), _ptr(k8), _ptr(sk), _ptr(v_res), _ptr(v_sf), _ptr(v_scale),
                                _ptr(_u16(v_mean)), B, H, N, d, float(softmax_scale), int(expcast), int(vmode),
                                _ptr(_u16(O)), _ptr(dev_status), _stream(stream, dev))
    _check(st, "vca_attention")


def vca_expcast_codes(s_raw, c, m, out, stream=None) -> None:
    n = s_raw.numel()
    dev = _buffers("vca_expcast_codes", [("s_raw", s_raw, 4 * n), ("c", c, 4 * n), ("m", m, 4 * n), ("out", out, n)])
    with torch.cuda.device(dev):
        _check(_lib.vca_expcast_codes(_ptr(s_raw), _ptr(c), _ptr(m), n, _ptr(out), _stream(stream, dev)),
               "vca_expcast_codes")


def vca_e4m3_encode_bits(start: int, n: int, out, stream=None) -> None:
    dev = _buffers("vca_e4m3_encode_bits", [("out", out, n)])
    with torch.cuda.device(dev):
        _check(_lib.vca_e4m3_encode_bits(ctypes.c_uint32(start), n, _ptr(out), _stream(stream, dev)),
               "vca_e4m3_encode_bits")


def vca_selftest_timeout(dev_status, limit_ns: int, stream=None) -> None:
    dev = _buffers("vca_selftest_timeout", [("dev_status", dev_status, 4)])
    with torch.cuda.device(dev):
        _check(_lib.vca_selftest_timeout(_ptr(dev_status), ctypes.c_uint64(limit_ns), _stream(stream, dev)),
               "vca_selftest_timeout")


# ---------------------------------------------------------------------------
# Buffer sets and the whole path (allocation through PyTorch)
# ---------------------------------------------------------------------------
@dataclass
class Grouped:
    labels: torch.Tensor
    perm: torch.Tensor
    counts: torch.Tensor
    centroids: torch.Tensor
    ws: torch.Tensor


@dataclass
class Prepared:
    q8: torch.Tensor
    sq: torch.Tensor
    k8: torch.Tensor
    sk: torch.Tensor
    v_res: torch.Tensor
    v_sf: Optional[torch.Tensor]
    v_scale: torch.Tensor
    v_mean: torch.Tensor
    ws: torch.Tensor
    vmode: int


def alloc_group(B, H, N, k, device="cuda") -> Grouped:
    BH = B * H
    ws = torch.empty(max(16, vca_workspace_bytes(VCA_OP_GROUP, B, H, N, 128, k, 0)), dtype=torch.uint8, device=device)
    return Grouped(torch.empty((BH, N), dtype=torch.int32, device=device),
                   torch.empty((BH, N), dtype=torch.int32, device=device),
                   torch.empty((BH, k), dtype=torch.int32, device=device),
                   torch.empty((BH, k, 128), dtype=torch.float32, device=device), ws)


def alloc_prep(B, H, N, vmode=VCA_V_E4M3, device="cuda", k_smooth: bool = False) -> Prepared:
    BH, nb, d = B * H, N // 128, 128
    op = VCA_OP_PREP_KSMOOTH if k_smooth else VCA_OP_PREP
    ws = torch.empty(max(16, vca_workspace_bytes(op, B, H, N, d, 1, vmode)), dtype=torch.uint8, device=device)
    if vmode == VCA_V_E4M3:
        v_res = torch.empty((BH, nb, d, 128), dtype=torch.uint8, device=device)
        v_sf = None
        v_scale = torch.empty((BH, d), dtype=torch.float32, device=device)
    else:
        v_res = torch.empty((BH, nb, d, 64), dtype=torch.uint8, device=device)
        v_sf = torch.empty((BH, nb, d, 8), dtype=torch.uint8, device=device)
        v_scale = torch.empty((BH,), dtype=torch.float32, device=device)
    return Prepared(torch.empty((BH, N, d), dtype=torch.uint8, device=device),
                    torch.empty((BH, nb), dtype=torch.float32, device=device),
                    torch.empty((BH, N, d), dtype=torch.uint8, device=device),
                    torch.empty((BH, nb), dtype=torch.float32, device=device),
                    v_res, v_sf, v_scale,
                    torch.empty((BH, nb, d), dtype=torch.bfloat16, device=device), ws, vmode)


def group(V: torch.Tensor, k: int, iters: int, out: Optional[Grouped] = None,
          dev_status: Optional[torch.Tensor] = None) -> Grouped:
    B, H, N, _ = V.shape
    g = out or alloc_group(B, H, N, k, V.device)
    vca_group(V, k, iters, g.labels, g.perm, g.counts, g.centroids, g.ws, dev_status)
    return g


def prep_quant(Q, K, V, perm, vmode=VCA_V_E4M3, out: Optional[Prepared] = None,
               qk_hadamard: bool = False, k_smooth: bool = False) -> Prepared:
    B, H, N, _ = Q.shape
    p = out or alloc_prep(B, H, N, vmode, Q.device, k_smooth=k_smooth)
    flags = (VCA_PREP_QK_HADAMARD if qk_hadamard else 0) | (VCA_PREP_K_SMOOTH if k_smooth else 0)
    vca_prep_quant_ex(Q, K, V, perm, vmode, flags, p.q8, p.sq, p.k8, p.sk, p.v_res, p.v_sf, p.v_scale, p.v_mean,
                      p.ws)
    return p


def attention(p: Prepared, B: int, H: int, N: int, expcast: bool = True, softmax_scale: float = 0.0,
              out: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    O = out if out is not None else torch.empty((B, H, N, 128), dtype=torch.bfloat16, device=p.q8.device)
    vca_attention(p.q8, p.sq, p.k8, p.sk, p.v_res, p.v_sf, p.v_scale, p.v_mean, B, H, N, 128,
                  softmax_scale, int(expcast), p.vmode, O, dev_status)
    return O


def vc_attention(Q, K, V, k: int = 64, iters: int = 8, expcast: bool = True, vmode: int = VCA_V_E4M3,
                 softmax_scale: float = 0.0):
    """The whole hot path: group -> prep -> attention.  Returns (O, grouped, prepared)."""
    B, H, N, _ = Q.shape
    g = group(V, k, iters)
    p = prep_quant(Q, K, V, g.perm, vmode)
    O = attention(p, B, H, N, expcast=expcast, softmax_scale=softmax_scale)
    return O, g, p


# ---------------------------------------------------------------------------
# The 8-bit cache (layouts and formulas: include/vca.h)
# ---------------------------------------------------------------------------
@dataclass
class Cache:
    """Pages of E4M3 keys and values with one power-of-two scale per page and
    head, and the sequences that own them.  `length` counts each sequence's
    tokens with the new ones of the next call included."""
    k8: torch.Tensor        # uint8 [pages, H, 128, 128]
    v8: torch.Tensor
    sk: torch.Tensor        # float32 [pages, H]
    sv: torch.Tensor
    table: torch.Tensor     # int32 [B, cols]
    length: torch.Tensor    # int32 [B]


def alloc_cache(pages: int, H: int, B: int, cols: int, device="cuda") -> Cache:
    """An empty cache: every length 0, every table entry -1."""
    return Cache(torch.zeros((pages, H, 128, 128), dtype=torch.uint8, device=device),
                 torch.zeros((pages, H, 128, 128), dtype=torch.uint8, device=device),
                 torch.full((pages, H), 2.0 ** -120, dtype=torch.float32, device=device),
                 torch.full((pages, H), 2.0 ** -120, dtype=torch.float32, device=device),
                 torch.full((B, cols), -1, dtype=torch.int32, device=device),
                 torch.zeros((B,), dtype=torch.int32, device=device))


_MOST = 2 ** 31 - 1      # the C interface's int; ctypes cuts larger numbers


def vca_cache_workspace_bytes(op: int, T: int, Hq: int, H: int, B: int, cols: int) -> int:
    if max(T, Hq, H, B, cols) > _MOST:
        return 0
    return int(_lib.vca_cache_workspace_bytes(op, T, Hq, H, B, cols))


def _ranks(where, cache: Cache):
    if cache.k8.dim() != 4 or cache.table.dim() != 2:
        raise ValueError(f"{where}: k8 must be [pages, H, 128, 128] and table [B, cols]")


def _typed(where, name, t, dtype, shape):
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{where}: {name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")


def _few_enough(where, name, t):
    if max(t.shape[:2], default=0) > _MOST:
        raise ValueError(f"{where}: {name} has more than {_MOST} rows or heads")


def _cache_call(where, cache: Cache, rows, others, start=None, ws=None):
    """Checks a call's tensors and returns the C struct and the device: every
    tensor of the types and shapes of include/vca.h, all on one CUDA device.
    `rows` are (name, tensor, heads) of [T, heads, 128] bf16 with contiguous
    channels, `others` (name, tensor, dtype, shape), the tensor None where it is
    not given; `ws` is a workspace or None."""
    k8, v8, sk, sv, table, length = cache.k8, cache.v8, cache.sk, cache.sv, cache.table, cache.length
    if k8.dim() != 4 or table.dim() != 2:
        _ranks(where, cache)
    pages, H = k8.shape[:2]
    B, cols = table.shape
    codes, scales = (pages, H, 128, 128), (pages, H)
    seen = [("k8", k8, torch.uint8, codes), ("v8", v8, torch.uint8, codes), ("sk", sk, torch.float32, scales),
            ("sv", sv, torch.float32, scales), ("table", table, torch.int32, (B, cols)),
            ("length", length, torch.int32, (B,))]
    if start is not None:
        seen.append(("start", start, torch.int32, (B + 1,)))
    seen += [x for x in others if x[1] is not None]
    # a launch of a few microseconds waits for these checks: all at once, and by name only where one fails
    dev = k8.get_device()
    ok = dev >= 0 and (ws is None or (ws.get_device() == dev and ws.is_contiguous()))
    for _, t, dtype, shape in seen:
        ok = ok and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()
    T = rows[0][1].shape[0] if rows and rows[0][1].dim() else 0
    for _, t, heads in rows:
        ok = ok and T <= _MOST and heads <= _MOST
        ok = ok and t.dtype is torch.bfloat16 and t.shape == (T, heads, 128) and t.stride(2) == 1 and t.get_device() == dev
    if not ok:
        _refuse(where, k8, seen, rows, ws)
    s = _CacheStruct(k8.data_ptr(), v8.data_ptr(), sk.data_ptr(), sv.data_ptr(), table.data_ptr(), length.data_ptr(),
                     pages, H, 128, B, cols)
    return s, dev


def _refuse(where, k8, seen, rows, ws, first="k8"):
    """Names the first tensor of a call that is not as it must be; `k8`, named `first`, is on the call's device."""
    T = None
    for name, t, heads in rows:
        _few_enough(where, name, t)
        shape = t.shape
        if t.dtype != torch.bfloat16 or len(shape) != 3 or shape[1] != heads or shape[2] != 128:
            raise ValueError(f"{where}: {name} must be bfloat16 [T, {heads}, 128], got {t.dtype} {tuple(shape)}")
        if t.stride(2) != 1:
            raise ValueError(f"{where}: the channels of {name} must be contiguous")
        if T is not None and shape[0] != T:
            raise ValueError(f"{where}: {name} has {shape[0]} rows, not {T}")
        T = shape[0]
    for name, t, dtype, shape in seen:
        _typed(where, name, t, dtype, shape)
    if ws is not None and not ws.is_contiguous():
        raise ValueError(f"{where}: ws must be contiguous")
    named = [x[:2] for x in (*seen, *rows)] + ([("ws", ws)] if ws is not None else [])
    for name, t in named:
        if not t.is_cuda:
            raise ValueError(f"{where}: {name} is not a CUDA tensor")
        if t.device != k8.device:
            raise ValueError(f"{where}: tensors on several devices: {name} on {t.device}, {first} on {k8.device}")
    raise ValueError(f"{where}: tensors that do not fit together")


def _launch(where, dev, fn, *args, stream=None):
    """fn(*args, stream) with device `dev` current, on its current stream unless one is given."""
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, raw)
    if st != VCA_OK:
        _check(st, where)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def vca_cache_append(cache: Cache, K, V, start, dev_status=None, stream=None, weight=None) -> None:
    H = cache.k8.shape[1] if cache.k8.dim() == 4 else 0
    s, dev = _cache_call("vca_cache_append", cache, (("K", K, H), ("V", V, H)),
                         (("weight", weight, torch.float32, (*cache.sk.shape, 128)),
                          ("dev_status", dev_status, torch.int32, (1,))), start)
    _launch("vca_cache_append", dev, _lib.vca_cache_append_ex, s, K.data_ptr(), K.stride(0), K.stride(1), V.data_ptr(),
            V.stride(0), V.stride(1), start.data_ptr(), K.shape[0], _at(weight), _at(dev_status), stream=stream)


def vca_cache_attention(cache: Cache, Q, start, causal: int, softmax_scale: float, softcap: float, O, lse, ws,
                        dev_status=None, stream=None) -> None:
    T, Hq = (Q.shape[0], Q.shape[1]) if Q.dim() == 3 else (0, 0)
    s, dev = _cache_call("vca_cache_attention", cache, (("Q", Q, Hq),),
                         (("O", O, torch.bfloat16, (T, Hq, 128)), ("lse", lse, torch.float32, (T, Hq)),
                          ("dev_status", dev_status, torch.int32, (1,))), start, ws)
    _launch("vca_cache_attention", dev, _lib.vca_cache_attention, s, Q.data_ptr(), Q.stride(0), Q.stride(1),
            start.data_ptr(), T, Hq, int(causal), softmax_scale, softcap, O.data_ptr(), _at(lse), _at(ws),
            0 if ws is None else ws.numel() * ws.element_size(), _at(dev_status), stream=stream)


def vca_cache_weigh(cache: Cache, Q, start, causal: int, softmax_scale: float, softcap: float, lse, weight, ws,
                    dev_status=None, stream=None) -> None:
    T, Hq = (Q.shape[0], Q.shape[1]) if Q.dim() == 3 else (0, 0)
    s, dev = _cache_call("vca_cache_weigh", cache, (("Q", Q, Hq),),
                         (("lse", lse, torch.float32, (T, Hq)),
                          ("weight", weight, torch.float32, (*cache.sk.shape, 128)),
                          ("dev_status", dev_status, torch.int32, (1,))), start, ws)
    _launch("vca_cache_weigh", dev, _lib.vca_cache_weigh, s, Q.data_ptr(), Q.stride(0), Q.stride(1), start.data_ptr(),
            T, Hq, int(causal), softmax_scale, softcap, lse.data_ptr(), weight.data_ptr(), _at(ws),
            0 if ws is None else ws.numel() * ws.element_size(), _at(dev_status), stream=stream)


def _cut(budget, recent, dst_cols):
    if not (-_MOST <= budget <= _MOST and -_MOST <= recent <= _MOST and dst_cols <= _MOST):
        raise ValueError(f"vca_cache_evict: budget {budget}, recent {recent} and dst_cols {dst_cols} must fit 32 bits")


def vca_cache_evict(cache: Cache, weight, dst_table, budget: int, recent: int, new_len, kept, dev_status=None,
                    stream=None) -> None:
    if dst_table.dim() != 2:
        raise ValueError("vca_cache_evict: dst_table must be [B, dst_cols]")
    _cut(budget, recent, dst_table.shape[1])
    B, H = cache.table.shape[:1], cache.sk.shape[1:]
    s, dev = _cache_call("vca_cache_evict", cache, (),
                         (("weight", weight, torch.float32, (*cache.sk.shape, 128)),
                          ("dst_table", dst_table, torch.int32, (*B, dst_table.shape[1])),
                          ("new_len", new_len, torch.int32, B), ("kept", kept, torch.int32, (*B, *H, budget)),
                          ("dev_status", dev_status, torch.int32, (1,))))
    _launch("vca_cache_evict", dev, _lib.vca_cache_evict, s, weight.data_ptr(), dst_table.data_ptr(),
            dst_table.shape[1], budget, recent, new_len.data_ptr(), kept.data_ptr(), _at(dev_status), stream=stream)


def _cache_ws(where, op, cache: Cache, Q):
    _ranks(where, cache)
    if Q.dim() != 3:
        raise ValueError(f"{where}: Q must be bfloat16 [T, Hq, 128], got {Q.dtype} {tuple(Q.shape)}")
    _few_enough(where, "Q", Q)
    need = vca_cache_workspace_bytes(op, Q.shape[0], Q.shape[1], cache.k8.shape[1], *cache.table.shape)
    return torch.empty(need, dtype=torch.uint8, device=cache.k8.device) if need else None


def cache_append(cache: Cache, K, V, start, dev_status=None, weight: Optional[torch.Tensor] = None) -> None:
    """Quantises the new rows K, V [T, H, 128] into the cache's pages; sequence b
    owns the rows start[b] .. start[b+1] - 1, its newest tokens.  `weight`
    [pages, H, 128], where the tokens are weighed: theirs becomes 0."""
    vca_cache_append(cache, K, V, start, dev_status, weight=weight)


def cache_attention(cache: Cache, Q, start, causal: bool = True, softmax_scale: float = 0.0, softcap: float = 0.0,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None):
    """Attention of Q [T, Hq, 128] over the cache.  Returns (O [T, Hq, 128], lse [T, Hq])."""
    if ws is None:
        ws = _cache_ws("vca_cache_attention", VCA_OP_CACHE_ATTENTION, cache, Q)
    O = out if out is not None else torch.empty(Q.shape, dtype=torch.bfloat16, device=Q.device)
    lse = lse if lse is not None else torch.empty(Q.shape[:2], dtype=torch.float32, device=Q.device)
    vca_cache_attention(cache, Q, start, causal, softmax_scale, softcap, O, lse, ws, dev_status)
    return O, lse


def cache_weigh(cache: Cache, Q, start, lse, weight, causal: bool = True, softmax_scale: float = 0.0,
                softcap: float = 0.0, ws: Optional[torch.Tensor] = None,
                dev_status: Optional[torch.Tensor] = None) -> None:
    """Adds to weight [pages, H, 128] the attention that each cached token gets
    from Q; lse is cache_attention's.  cache_append(weight=...) makes a new
    token's weight 0."""
    if ws is None:
        ws = _cache_ws("vca_cache_weigh", VCA_OP_CACHE_WEIGH, cache, Q)
    vca_cache_weigh(cache, Q, start, causal, softmax_scale, softcap, lse, weight, ws, dev_status)


def cache_evict(cache: Cache, weight, dst_table, budget: int, recent: int, kept: Optional[torch.Tensor] = None,
                dev_status: Optional[torch.Tensor] = None):
    """Cuts every sequence to `budget` tokens per head into the pages of
    dst_table.  Returns (new_len [B], kept [B, H, budget]); the cut sequences are
    Cache(k8, v8, sk, sv, dst_table, new_len)."""
    _ranks("vca_cache_evict", cache)
    B, H = cache.table.shape[0], cache.k8.shape[1]
    new_len = torch.empty((B,), dtype=torch.int32, device=cache.k8.device)
    if kept is None:
        _cut(budget, recent, 0)
        kept = torch.full((B, H, budget), -1, dtype=torch.int32, device=cache.k8.device)
    vca_cache_evict(cache, weight, dst_table, budget, recent, new_len, kept, dev_status)
    return new_len, kept


# ---------------------------------------------------------------------------
# The cache's pages, and prompts on their way into it (include/vca.h)
# ---------------------------------------------------------------------------
def _refuse_ints(where, cache: Cache, ints):
    """Names the first tensor (name, tensor or None, shape) of a planning call that is not int32, contiguous, of its shape
    and on the table's CUDA device."""
    if cache.table.dim() != 2 or cache.k8.dim() != 4 or max(cache.k8.shape[0], *cache.table.shape) > _MOST:
        raise ValueError(f"{where}: k8 must be [pages, H, 128, 128] and table [B, cols]")
    given = [x for x in ints if x[1] is not None]
    for name, t, shape in given:
        _typed(where, name, t, torch.int32, shape)
    for name, t, _ in given:
        if not t.is_cuda:
            raise ValueError(f"{where}: {name} is not a CUDA tensor")
        if t.device != cache.table.device:
            raise ValueError(f"{where}: tensors on several devices: {name} on {t.device}, table on {cache.table.device}")
    raise ValueError(f"{where}: tensors that do not fit together")


def _is_ints(t, n, dev):
    return t.dtype is torch.int32 and t.shape == n and t.get_device() == dev and t.is_contiguous()


def vca_cache_plan(cache: Cache, held, news, T: int, start, slot, position, dev_status=None, stream=None) -> None:
    if not 0 <= T <= _MOST:
        raise ValueError(f"vca_cache_plan: T = {T} must be 0 .. {_MOST}")
    table, length = cache.table, cache.length
    shape, pages, dev = table.shape, cache.k8.shape[0] if cache.k8.dim() == 4 else 0, table.get_device()
    B = shape[0] if shape else 0
    one, rows = (B,), (T,)
    # all at once, and by name only where one fails, as in _cache_call
    ok = (dev >= 0 and len(shape) == 2 and 0 < pages <= _MOST and max(shape) <= _MOST and _is_ints(table, shape, dev)
          and _is_ints(length, one, dev) and (held is length or _is_ints(held, one, dev)) and _is_ints(news, one, dev)
          and _is_ints(start, (B + 1,), dev) and (slot is None or _is_ints(slot, rows, dev))
          and (position is None or _is_ints(position, rows, dev)) and (dev_status is None or _is_ints(dev_status, (1,), dev)))
    if not ok:
        _refuse_ints("vca_cache_plan", cache, (
            ("table", table, shape), ("length", length, one), ("held", held, one), ("news", news, one), ("start", start, (B + 1,)),
            ("slot", slot, rows), ("position", position, rows), ("dev_status", dev_status, (1,))))
    _launch("vca_cache_plan", dev, _lib.vca_cache_plan, table.data_ptr(), length.data_ptr(), pages, B, shape[1], held.data_ptr(),
            news.data_ptr(), start.data_ptr(), _at(slot), _at(position), T, _at(dev_status), stream=stream)


def vca_cache_fresh(cache: Cache, budget: int, dst_table, dev_status=None, stream=None) -> None:
    if dst_table.dim() != 2:
        raise ValueError("vca_cache_fresh: dst_table must be [B, dst_cols]")
    if not (-_MOST <= budget <= _MOST and dst_table.shape[1] <= _MOST):
        raise ValueError(f"vca_cache_fresh: budget {budget} and dst_cols {dst_table.shape[1]} must fit 32 bits")
    table, length = cache.table, cache.length
    shape, pages, dev = table.shape, cache.k8.shape[0] if cache.k8.dim() == 4 else 0, table.get_device()
    B = shape[0] if shape else 0
    dst = (B, dst_table.shape[1])
    ok = (dev >= 0 and len(shape) == 2 and 0 < pages <= _MOST and max(shape) <= _MOST and _is_ints(table, shape, dev)
          and _is_ints(length, (B,), dev) and _is_ints(dst_table, dst, dev) and (dev_status is None or _is_ints(dev_status, (1,), dev)))
    if not ok:
        _refuse_ints("vca_cache_fresh", cache, (("table", table, shape), ("length", length, (B,)), ("dst_table", dst_table, dst),
                                                ("dev_status", dev_status, (1,))))
    _launch("vca_cache_fresh", dev, _lib.vca_cache_fresh, table.data_ptr(), length.data_ptr(), pages, B, shape[1], budget,
            dst_table.data_ptr(), dst_table.shape[1], _at(dev_status), stream=stream)


def cache_plan(cache: Cache, news, T: int, held: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
               slot: Optional[torch.Tensor] = None, position: Optional[torch.Tensor] = None,
               dev_status: Optional[torch.Tensor] = None):
    """Pages, lengths and places for news [B] new tokens of each sequence behind
    the held [B] ones (cache.length, which becomes their sum); T is how many rows the
    call will have room for.  Returns (start [B + 1], slot [T], position [T]); slot
    and position are -1 behind the last row where they are made here.  With too few
    free pages (dev_status: VCA_ERR_FULL) start is 0 throughout and nothing changes."""
    table = cache.table
    if T < 0 or T > _MOST or table.dim() != 2:
        raise ValueError(f"vca_cache_plan: T = {T} must be 0 .. {_MOST} and table [B, cols]")
    if start is None:
        start = torch.empty((table.shape[0] + 1,), dtype=torch.int32, device=table.device)
    if slot is None:
        slot = torch.full((T,), -1, dtype=torch.int32, device=table.device)
    if position is None:
        position = torch.full((T,), -1, dtype=torch.int32, device=table.device)
    vca_cache_plan(cache, cache.length if held is None else held, news, T, start, slot, position, dev_status)
    return start, slot, position


def cache_fresh(cache: Cache, budget: int, out: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None):
    """Free pages for cache_evict to `budget` tokens: its dst_table [B, ceil(budget / 128)],
    -1 where a sequence needs none."""
    if out is None:
        if cache.table.dim() != 2 or not 1 <= budget <= _MOST:
            raise ValueError(f"vca_cache_fresh: budget {budget} must be 1 .. {_MOST} and table [B, cols]")
        out = torch.full((cache.table.shape[0], -(-budget // 128)), -1, dtype=torch.int32, device=cache.table.device)
    vca_cache_fresh(cache, budget, out, dev_status)
    return out


def vca_prompt_attention(Q, K, V, start, causal: int, softmax_scale: float, softcap: float, prior, prior_lse, O, lse,
                         dev_status=None, stream=None) -> None:
    if Q.dim() != 3 or K.dim() != 3 or start.dim() != 1:
        raise ValueError(f"vca_prompt_attention: Q must be bfloat16 [T, Hq, 128], K and V [T, H, 128] and start int32 [B + 1], "
                         f"got {tuple(Q.shape)}, {tuple(K.shape)} and {tuple(start.shape)}")
    (T, Hq, _), H, B = Q.shape, K.shape[1], start.shape[0] - 1
    dev, kv, wide, per_row, bf16, f32 = Q.get_device(), (T, H, 128), (T, Hq, 128), (T, Hq), torch.bfloat16, torch.float32
    sq, sk, sv = Q.stride(), K.stride(), V.stride()
    # a launch of a few microseconds waits for these checks: all at once, and by name only where one fails
    ok = (dev >= 0 and Q.dtype is bf16 and Q.shape == wide and sq[2] == 1 and K.dtype is bf16 and K.shape == kv and sk[2] == 1
          and V.dtype is bf16 and V.shape == kv and sv[2] == 1 and start.dtype is torch.int32 and start.is_contiguous()
          and O.dtype is bf16 and O.shape == wide and O.is_contiguous() and (prior is None) == (prior_lse is None)
          and K.get_device() == dev and V.get_device() == dev and start.get_device() == dev and O.get_device() == dev
          and max(T, Hq, H, B) <= _MOST)
    for t, dtype, shape in ((lse, f32, per_row), (prior, bf16, wide), (prior_lse, f32, per_row), (dev_status, torch.int32, (1,))):
        if t is not None:
            ok = ok and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()
    if not ok:
        if (prior is None) != (prior_lse is None):
            raise ValueError("vca_prompt_attention: prior and prior_lse are given together")
        _few_enough("vca_prompt_attention", "start", start)
        seen = (("start", start, torch.int32, (B + 1,)), ("O", O, bf16, wide), ("lse", lse, f32, per_row), ("prior", prior, bf16, wide),
                ("prior_lse", prior_lse, f32, per_row), ("dev_status", dev_status, torch.int32, (1,)))
        _refuse("vca_prompt_attention", Q, [x for x in seen if x[1] is not None], (("Q", Q, Hq), ("K", K, H), ("V", V, H)), None, "Q")
    _launch("vca_prompt_attention", dev, _lib.vca_prompt_attention, Q.data_ptr(), sq[0], sq[1], K.data_ptr(), sk[0], sk[1],
            V.data_ptr(), sv[0], sv[1], start.data_ptr(), B, T, Hq, H, 128, int(causal), softmax_scale, softcap, _at(prior),
            _at(prior_lse), O.data_ptr(), _at(lse), _at(dev_status), stream=stream)


def prompt_attention(Q, K, V, start, causal: bool = True, softmax_scale: float = 0.0, softcap: float = 0.0, prior=None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None):
    """Attention of packed prompts Q [T, Hq, 128] over their own K, V [T, H, 128]; sequence
    b owns the rows start[b] .. start[b+1] - 1.  `prior`, the (O, lse) of an attention
    over what came before (cache_attention's), is joined in.  Returns (O [T, Hq, 128],
    lse [T, Hq])."""
    O = out if out is not None else torch.empty(Q.shape, dtype=torch.bfloat16, device=Q.device)
    lse = lse if lse is not None else torch.empty(Q.shape[:2], dtype=torch.float32, device=Q.device)
    before, before_lse = prior if prior is not None else (None, None)
    vca_prompt_attention(Q, K, V, start, causal, softmax_scale, softcap, before, before_lse, O, lse, dev_status)
    return O, lse
