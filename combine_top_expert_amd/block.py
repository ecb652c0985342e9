"""Python binding of libmoe_block.so -- what stands around and inside the MoE
share in a transformer block: residual add + RMS norm, group-limited routing,
dispatch of rows that are in block FP8 already, and the experts' products with
4-bit weights.

The same manner as the package's other entry points (argument marshalling
only; every name here is also a name of the package), plus: all tensors of a
call must be on one device, which need not be the current one.
"""
from __future__ import annotations

import ctypes
import os
from pathlib import Path

import torch

from . import MOE_BF16, MOE_EPI_SILU_MUL, MOE_EPI_STORE_G, MOE_F32, MOE_FP8_E4M3, MoEError, _need, _offsets, _stream

__all__ = [
    "BLOCK_LIB_PATH", "block_lib", "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID", "MOE_W4_INT4", "MOE_W4_E2M1",
    "moe_block_abi_version", "moe_add_rms_norm", "moe_add_rms_norm_backward",
    "moe_add_rms_norm_backward_workspace_bytes", "moe_router_group_topk", "moe_router_group_topk_backward",
    "moe_permute_fp8", "moe_pack_w4", "moe_grouped_gemv_w4",
]

BLOCK_LIB_PATH = Path(os.environ.get("MOE_BLOCK_LIB", Path(__file__).resolve().parent / "libmoe_block.so"))

MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_W4_INT4, MOE_W4_E2M1 = 0, 1


class _NotBuilt:
    """In the library's place where it is missing: a program that uses the share
    only (libmoe_ep.so) needs none of it, and one that calls into it is told."""

    def __getattr__(self, name):
        raise ImportError(f"{name}: {BLOCK_LIB_PATH} is not built; run `python combine_top_expert_amd/build.py` "
                          "(these operators have no fallback without their HIP library)")


if BLOCK_LIB_PATH.exists():
    block_lib = ctypes.CDLL(str(BLOCK_LIB_PATH))
elif "MOE_BLOCK_LIB" in os.environ:                  # asked for by name
    raise ImportError(f"MOE_BLOCK_LIB={BLOCK_LIB_PATH} is not built")
else:
    block_lib = _NotBuilt()

_p, _i, _i64, _sz, _fl = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_SIG = {
    "moe_block_abi_version": (_i, []),
    "moe_add_rms_norm": (_i, [_p, _p, _i, _p, _i, _fl, _i, _i, _p, _p, _p, _p, _p]),
    "moe_add_rms_norm_backward_workspace_bytes": (_sz, [_i, _i]),
    "moe_add_rms_norm_backward": (_i, [_p, _p, _p, _i, _p, _i, _fl, _i, _i, _p, _p, _p, _sz, _p]),
    "moe_router_group_topk": (_i, [_p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _fl, _p, _p, _p]),
    "moe_router_group_topk_backward": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _fl, _p, _p]),
    "moe_permute_fp8": (_i, [_p, _p, _i, _i, _i, _p, _i64, _p, _p, _p]),
    "moe_pack_w4": (_i, [_p, _p, _i, _i, _i, _i, _i, _i, _p, _p, _p]),
    "moe_grouped_gemv_w4": (_i, [_p, _i, _p, _p, _p, _i, _i, _i, _p, _p, _i, _i64, _i, _i, _i, _p, _i, _p]),
}
for _name, (_res, _args) in _SIG.items() if BLOCK_LIB_PATH.exists() else ():
    if not hasattr(block_lib, _name):
        raise ImportError(f"{BLOCK_LIB_PATH} lacks {_name}: it predates these sources; rebuild with "
                          "`python combine_top_expert_amd/build.py`")
    _f = getattr(block_lib, _name)
    _f.restype, _f.argtypes = _res, _args


def moe_block_abi_version() -> int:
    return int(block_lib.moe_block_abi_version())


# ---------------------------------------------------------------- marshalling helpers
#
# A decode step calls these operators for a few microseconds of GPU time each,
# so a call's checks are one pass over its tensors that only compares, and what
# is wrong is found out where something is.

_CODE = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float8_e4m3fn: MOE_FP8_E4M3,
         torch.uint8: MOE_FP8_E4M3}
_F32, _I32, _U8 = (torch.float32,), (torch.int32,), (torch.uint8,)
_REAL, _FP8 = (torch.float32, torch.bfloat16), (torch.float8_e4m3fn, torch.uint8)
_ANY = tuple(_CODE)


def _refuse(specs) -> None:
    """Raise for the first fault among (name, tensor, dtypes, shape): shapes
    and dtypes first (the C ABI receives sizes, not extents), then placement."""
    given = [s for s in specs if s[1] is not None]
    for name, t, _, shape in given:
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    for name, t, dtypes, _ in given:
        if t.dtype not in dtypes:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    for name, t, _, _ in given:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if t.device != given[0][1].device:
            raise ValueError(f"{name} is on {t.device}, expected {given[0][1].device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    raise ValueError("unsupported tensor arguments")


def _pointers(*specs):
    """Device index of the first tensor and the data pointers of all (None for
    None), each checked for device, dtype, shape and contiguity."""
    dev = specs[0][1].get_device()
    out = []
    for _, t, dtypes, shape in specs:
        if t is None:
            out.append(None)
            continue
        if dev < 0 or t.get_device() != dev or t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
            _refuse(specs)
        out.append(t.data_ptr())
    return dev, out


# the current stream's handle without building a torch.cuda.Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: _stream(torch.empty(0, device=torch.device("cuda", dev))))


_INT_MAX, _UNSUPPORTED = 0x7fffffff, -2


def _too_large(fn: str):
    """A size that the C ABI's int does not hold (ctypes would cut it off and
    the call work on what is left)."""
    raise MoEError(fn, _UNSUPPORTED)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _Calls(dict):
    """The entry points, looked up in the library once."""

    def __missing__(self, name):
        self[name] = getattr(block_lib, name)
        return self[name]


_CALL = _Calls()


def _run(fn: str, bind: bool, dev: int, args: tuple):
    """Call C entry point ``fn`` with device ``dev`` current (launches go to the
    current device), or return that call as a zero-argument callable."""
    if bind:
        return lambda: _run(fn, False, dev, args)
    if _current_device() == dev:
        st = _CALL[fn](*args)
    else:
        with torch.cuda.device(dev):
            st = _CALL[fn](*args)
    if st != 0:
        raise MoEError(fn, st)


# ---------------------------------------------------------------- norm

def moe_add_rms_norm(x, residual, weight, eps, h_out=None, y=None, y8=None, y8_scales=None, bind=False):
    """x [T,H] (+ residual [T,H], or None) -> h_out = x + residual, y = its RMS
    norm times weight [H], y8/y8_scales = y in block FP8 (any of the three may
    be None).  h_out or y may be x or residual itself."""
    T, H = rows = x.shape
    if T > _INT_MAX or H > _INT_MAX:
        _too_large("moe_add_rms_norm")
    dt = (x.dtype,) if x.dtype in _REAL else _REAL
    if y8 is not None or y8_scales is not None:
        _need(y8_scales, "y8_scales", True)
        _need(y8, "y8", True)
    dev, (px, pr, pw, ph, py, p8, ps) = _pointers(
        ("x", x, dt, rows), ("residual", residual, dt, rows), ("weight", weight, _REAL, (H,)),
        ("h_out", h_out, dt, rows), ("y", y, dt, rows), ("y8", y8, _FP8, rows),
        ("y8_scales", y8_scales, _F32, (T, H // 128)))
    return _run("moe_add_rms_norm", bind, dev, (
        px, pr, _CODE[x.dtype], pw, _CODE[weight.dtype], eps, T, H, ph, py, p8, ps, _raw_stream(dev)))


def moe_add_rms_norm_backward_workspace_bytes(T: int, H: int) -> int:
    if max(T, H) > _INT_MAX or min(T, H) < 0:
        return 0
    return int(block_lib.moe_add_rms_norm_backward_workspace_bytes(T, H))


def moe_add_rms_norm_backward(dy, h, weight, eps, dx, d_weight, workspace, dh=None, bind=False):
    """dy [T,H], the forward's h [T,H] (and dh [T,H], the gradient of h_out) ->
    dx [T,H], the gradient of x and of residual, and d_weight [H] fp32.
    workspace: moe_add_rms_norm_backward_workspace_bytes(T, H) bytes or more."""
    T, H = rows = dy.shape
    if T > _INT_MAX or H > _INT_MAX:
        _too_large("moe_add_rms_norm_backward")
    dt = (dy.dtype,) if dy.dtype in _REAL else _REAL
    dev, (pdy, ph, pdh, pw, pdx, pdw, pws) = _pointers(
        ("dy", dy, dt, rows), ("h", h, dt, rows), ("dh", dh, dt, rows), ("weight", weight, _REAL, (H,)),
        ("dx", dx, dt, rows), ("d_weight", d_weight, _F32, (H,)),
        ("workspace", workspace, (workspace.dtype,), workspace.shape))
    return _run("moe_add_rms_norm_backward", bind, dev, (
        pdy, ph, pdh, _CODE[dy.dtype], pw, _CODE[weight.dtype], eps, T, H, pdx, pdw, pws,
        workspace.numel() * workspace.element_size(), _raw_stream(dev)))


# ---------------------------------------------------------------- routing

def moe_router_group_topk(logits, K, topk_ids, topk_weights, bias=None, score=MOE_SCORE_SIGMOID, n_group=1,
                          topk_group=1, group_top=2, renorm=True, route_scale=1.0, bind=False):
    """logits [T,E] fp32 (+ bias [E] fp32, for the choice only) -> topk_ids
    [T,K] int32 (-1 where no expert remains), topk_weights [T,K] fp32."""
    T, E = rows = logits.shape
    if max(T, E, K, n_group, topk_group) > _INT_MAX:
        _too_large("moe_router_group_topk")
    dev, (pl, pb, pi, pw) = _pointers(
        ("logits", logits, _F32, rows), ("bias", bias, _F32, (E,)), ("topk_ids", topk_ids, _I32, (T, K)),
        ("topk_weights", topk_weights, _F32, (T, K)))
    return _run("moe_router_group_topk", bind, dev, (
        pl, pb, T, E, K, score, n_group, topk_group, group_top, 1 if renorm else 0, route_scale, pi, pw,
        _raw_stream(dev)))


def moe_router_group_topk_backward(logits, topk_ids, d_weights, d_logits, score=MOE_SCORE_SIGMOID, renorm=True,
                                   route_scale=1.0, bind=False):
    """d_weights [T,K] (gradient of topk_weights), the forward's logits [T,E]
    and topk_ids [T,K] -> d_logits [T,E] fp32, every element written."""
    T, E = rows = logits.shape
    K = topk_ids.shape[1]
    if max(T, E, K) > _INT_MAX:
        _too_large("moe_router_group_topk_backward")
    dev, (pl, pi, pdw, pdl) = _pointers(
        ("logits", logits, _F32, rows), ("topk_ids", topk_ids, _I32, (T, K)),
        ("d_weights", d_weights, _F32, (T, K)), ("d_logits", d_logits, _F32, rows))
    return _run("moe_router_group_topk_backward", bind, dev, (
        pl, pi, pdw, T, E, K, score, 1 if renorm else 0, route_scale, pdl, _raw_stream(dev)))


# ---------------------------------------------------------------- dispatch of FP8 rows

def moe_permute_fp8(x8, x8_scales, slot_of, buf, buf_scales, bind=False):
    """x8 [T,H] e4m3fn with x8_scales [T,H/128], slot_of [T,K] -> buf
    [rows_cap,H], buf_scales [rows_cap,H/128], copied bit for bit."""
    T, H = x8.shape
    K, cap = slot_of.shape[1], buf.shape[0]
    if max(T, H, K) > _INT_MAX:
        _too_large("moe_permute_fp8")
    dev, (px, pxs, psl, pb, pbs) = _pointers(
        ("x8", x8, _FP8, (T, H)), ("x8_scales", x8_scales, _F32, (T, H // 128)), ("slot_of", slot_of, _I32, (T, K)),
        ("buf", buf, _FP8, (cap, H)), ("buf_scales", buf_scales, _F32, (cap, H // 128)))
    return _run("moe_permute_fp8", bind, dev, (px, pxs, T, K, H, psl, cap, pb, pbs, _raw_stream(dev)))


# ---------------------------------------------------------------- 4-bit weights

def _group(K: int, scales: torch.Tensor, name: str) -> int:
    if scales.dim() != 3 or scales.shape[2] < 1 or K % scales.shape[2] != 0:
        raise ValueError(f"{name} has shape {tuple(scales.shape)}, expected [L, N, K / group]")
    return K // scales.shape[2]


def moe_pack_w4(codes, scales, fmt, codes_packed, scales_packed, bind=False):
    """codes [L,N,K/2] uint8 (two 4-bit codes a byte, the even column low) and
    scales [L,N,K/group] (fp32|bf16) -> the same in the order that
    moe_grouped_gemv_w4 reads (same shapes and dtypes)."""
    L, N, half = codes.shape
    if max(L, N, 2 * half) > _INT_MAX:
        _too_large("moe_pack_w4")
    group = _group(2 * half, scales, "scales")
    dt = (scales.dtype,) if scales.dtype in _REAL else _REAL
    per = (L, N, 2 * half // group)
    dev, (pc, ps, qc, qs) = _pointers(
        ("codes", codes, _U8, (L, N, half)), ("scales", scales, dt, per),
        ("codes_packed", codes_packed, _U8, (L, N, half)), ("scales_packed", scales_packed, dt, per))
    return _run("moe_pack_w4", bind, dev, (
        pc, ps, _CODE[scales.dtype], fmt, L, N, 2 * half, group, qc, qs, _raw_stream(dev)))


def moe_grouped_gemv_w4(a, a_scales, codes_packed, scales_packed, fmt, counts, offsets, epi, out, bind=False):
    """a [rows_cap,K] (bf16, or e4m3fn with a_scales [rows_cap,K/128]) and the
    weights of moe_pack_w4 -> out [rows_cap,N] = G, or with MOE_EPI_SILU_MUL
    [rows_cap,N/2] = SiLU(gate) * up (fp32|bf16), on valid rows only."""
    L, N, half = codes_packed.shape
    rows_cap, K = a.shape[0], 2 * half
    if max(L, N, K) > _INT_MAX:
        _too_large("moe_grouped_gemv_w4")
    group = _group(K, scales_packed, "scales_packed")
    fp8 = a.dtype in _FP8
    _need(a_scales, "a_scales", fp8)
    if not fp8 and a_scales is not None:
        raise ValueError("a_scales goes with FP8 rows only")
    if epi not in (MOE_EPI_STORE_G, MOE_EPI_SILU_MUL):
        raise ValueError(f"epi is {epi}, expected MOE_EPI_STORE_G or MOE_EPI_SILU_MUL")
    _offsets(offsets, L)
    dev, (pa, pas, pc, ps, pn, po, pout) = _pointers(
        ("a", a, _ANY, (rows_cap, K)), ("a_scales", a_scales, _F32, (rows_cap, K // 128)),
        ("codes_packed", codes_packed, _U8, (L, N, half)),
        ("scales_packed", scales_packed, _REAL, (L, N, K // group)), ("counts", counts, _I32, (L,)),
        ("offsets", offsets, _I32, offsets.shape),
        ("out", out, _REAL, (rows_cap, N if epi == MOE_EPI_STORE_G else N // 2)))
    return _run("moe_grouped_gemv_w4", bind, dev, (
        pa, _CODE[a.dtype], pas, pc, ps, _CODE[scales_packed.dtype], fmt, group, pn, po, L, rows_cap, N, K, epi, pout,
        _CODE[out.dtype], _raw_stream(dev)))
