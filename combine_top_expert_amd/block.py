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

from . import MOE_EPI_SILU_MUL, MOE_EPI_STORE_G, MOE_FP8_E4M3, MoEError, _f32, _i32, _need, _offsets, _ptr, _shape, _stream, dtype_code

__all__ = [
    "BLOCK_LIB_PATH", "block_lib", "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID", "MOE_W4_INT4", "MOE_W4_E2M1",
    "moe_block_abi_version", "moe_add_rms_norm", "moe_add_rms_norm_backward",
    "moe_add_rms_norm_backward_workspace_bytes", "moe_router_group_topk", "moe_router_group_topk_backward",
    "moe_permute_fp8", "moe_pack_w4", "moe_grouped_gemv_w4",
]

BLOCK_LIB_PATH = Path(os.environ.get("MOE_BLOCK_LIB", Path(__file__).resolve().parent / "libmoe_block.so"))

MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_W4_INT4, MOE_W4_E2M1 = 0, 1

if not BLOCK_LIB_PATH.exists():
    raise ImportError(f"{BLOCK_LIB_PATH} is not built; run `python combine_top_expert_amd/build.py` "
                      "(these operators have no fallback without their HIP library)")
block_lib = ctypes.CDLL(str(BLOCK_LIB_PATH))

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
for _name, (_res, _args) in _SIG.items():
    if not hasattr(block_lib, _name):
        raise ImportError(f"{BLOCK_LIB_PATH} lacks {_name}: it predates these sources; rebuild with "
                          "`python combine_top_expert_amd/build.py`")
    _f = getattr(block_lib, _name)
    _f.restype, _f.argtypes = _res, _args


def moe_block_abi_version() -> int:
    return int(block_lib.moe_block_abi_version())


# ---------------------------------------------------------------- marshalling helpers

def _one_device(ref: torch.Tensor, **others: torch.Tensor | None) -> None:
    for name, t in others.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{name} is on {t.device}, expected {ref.device}")


def _like(ref: torch.Tensor, **others: torch.Tensor | None) -> None:
    """Raise unless every given tensor has ref's dtype."""
    for name, t in others.items():
        if t is not None and t.dtype != ref.dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {ref.dtype}")


def _fp8(t: torch.Tensor | None, name: str) -> int | None:
    if t is not None and dtype_code(t) != MOE_FP8_E4M3:
        raise TypeError(f"{name} must hold e4m3fn codes (float8_e4m3fn or uint8)")
    return _ptr(t, name)


def _u8(t: torch.Tensor, name: str) -> int | None:
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must be uint8")
    return _ptr(t, name)


def _run(fn: str, bind: bool, ref: torch.Tensor, args: tuple):
    """Call C entry point ``fn`` with ref's device current (launches go to the
    current device), or return that call as a zero-argument callable."""
    f, dev = getattr(block_lib, fn), ref.device.index

    def call():
        if torch.cuda.current_device() == dev:
            st = f(*args)
        else:
            with torch.cuda.device(dev):
                st = f(*args)
        if st != 0:
            raise MoEError(fn, st)
    return call if bind else call()


# ---------------------------------------------------------------- norm

def moe_add_rms_norm(x, residual, weight, eps, h_out=None, y=None, y8=None, y8_scales=None, bind=False):
    """x [T,H] (+ residual [T,H], or None) -> h_out = x + residual, y = its RMS
    norm times weight [H], y8/y8_scales = y in block FP8 (any of the three may
    be None).  h_out or y may be x or residual itself."""
    T, H = x.shape
    _shape(residual, "residual", T, H)
    _shape(weight, "weight", H)
    _shape(h_out, "h_out", T, H)
    _shape(y, "y", T, H)
    _shape(y8, "y8", T, H)
    _need(y8_scales, "y8_scales", y8 is not None)
    _need(y8, "y8", y8_scales is not None)
    _shape(y8_scales, "y8_scales", T, H // 128)
    _like(x, residual=residual, h_out=h_out, y=y)
    _one_device(x, residual=residual, weight=weight, h_out=h_out, y=y, y8=y8, y8_scales=y8_scales)
    return _run("moe_add_rms_norm", bind, x, (
        _ptr(x, "x"), _ptr(residual, "residual"), dtype_code(x), _ptr(weight, "weight"), dtype_code(weight), eps, T, H,
        _ptr(h_out, "h_out"), _ptr(y, "y"), _fp8(y8, "y8"), _f32(y8_scales, "y8_scales"), _stream(x)))


def moe_add_rms_norm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(block_lib.moe_add_rms_norm_backward_workspace_bytes(T, H))


def moe_add_rms_norm_backward(dy, h, weight, eps, dx, d_weight, workspace, dh=None, bind=False):
    """dy [T,H], the forward's h [T,H] (and dh [T,H], the gradient of h_out) ->
    dx [T,H], the gradient of x and of residual, and d_weight [H] fp32."""
    T, H = dy.shape
    _shape(h, "h", T, H)
    _shape(dh, "dh", T, H)
    _shape(dx, "dx", T, H)
    _shape(weight, "weight", H)
    _shape(d_weight, "d_weight", H)
    _like(dy, h=h, dh=dh, dx=dx)
    _one_device(dy, h=h, dh=dh, dx=dx, weight=weight, d_weight=d_weight, workspace=workspace)
    return _run("moe_add_rms_norm_backward", bind, dy, (
        _ptr(dy, "dy"), _ptr(h, "h"), _ptr(dh, "dh"), dtype_code(dy), _ptr(weight, "weight"), dtype_code(weight), eps,
        T, H, _ptr(dx, "dx"), _f32(d_weight, "d_weight"), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(dy)))


# ---------------------------------------------------------------- routing

def moe_router_group_topk(logits, K, topk_ids, topk_weights, bias=None, score=MOE_SCORE_SIGMOID, n_group=1,
                          topk_group=1, group_top=2, renorm=True, route_scale=1.0, bind=False):
    """logits [T,E] fp32 (+ bias [E] fp32, for the choice only) -> topk_ids
    [T,K] int32 (-1 where no expert remains), topk_weights [T,K] fp32."""
    T, E = logits.shape
    _shape(bias, "bias", E)
    _shape(topk_ids, "topk_ids", T, K)
    _shape(topk_weights, "topk_weights", T, K)
    _one_device(logits, bias=bias, topk_ids=topk_ids, topk_weights=topk_weights)
    return _run("moe_router_group_topk", bind, logits, (
        _f32(logits, "logits"), _f32(bias, "bias"), T, E, K, int(score), n_group, topk_group, group_top,
        1 if renorm else 0, route_scale, _i32(topk_ids, "topk_ids"), _f32(topk_weights, "topk_weights"),
        _stream(logits)))


def moe_router_group_topk_backward(logits, topk_ids, d_weights, d_logits, score=MOE_SCORE_SIGMOID, renorm=True,
                                   route_scale=1.0, bind=False):
    """d_weights [T,K] (gradient of topk_weights), the forward's logits [T,E]
    and topk_ids [T,K] -> d_logits [T,E] fp32, every element written."""
    T, E = logits.shape
    K = topk_ids.shape[1]
    _shape(topk_ids, "topk_ids", T, K)
    _shape(d_weights, "d_weights", T, K)
    _shape(d_logits, "d_logits", T, E)
    _one_device(logits, topk_ids=topk_ids, d_weights=d_weights, d_logits=d_logits)
    return _run("moe_router_group_topk_backward", bind, logits, (
        _f32(logits, "logits"), _i32(topk_ids, "topk_ids"), _f32(d_weights, "d_weights"), T, E, K, int(score),
        1 if renorm else 0, route_scale, _f32(d_logits, "d_logits"), _stream(logits)))


# ---------------------------------------------------------------- dispatch of FP8 rows

def moe_permute_fp8(x8, x8_scales, slot_of, buf, buf_scales, bind=False):
    """x8 [T,H] e4m3fn with x8_scales [T,H/128], slot_of [T,K] -> buf
    [rows_cap,H], buf_scales [rows_cap,H/128], copied bit for bit."""
    T, H = x8.shape
    K = slot_of.shape[1]
    _shape(x8_scales, "x8_scales", T, H // 128)
    _shape(slot_of, "slot_of", T, K)
    _shape(buf, "buf", buf.shape[0], H)
    _shape(buf_scales, "buf_scales", buf.shape[0], H // 128)
    _one_device(x8, x8_scales=x8_scales, slot_of=slot_of, buf=buf, buf_scales=buf_scales)
    return _run("moe_permute_fp8", bind, x8, (
        _fp8(x8, "x8"), _f32(x8_scales, "x8_scales"), T, K, H, _i32(slot_of, "slot_of"), buf.shape[0],
        _fp8(buf, "buf"), _f32(buf_scales, "buf_scales"), _stream(x8)))


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
    group = _group(2 * half, scales, "scales")
    _shape(scales, "scales", L, N, 2 * half // group)
    _shape(codes_packed, "codes_packed", L, N, half)
    _shape(scales_packed, "scales_packed", *scales.shape)
    _like(scales, scales_packed=scales_packed)
    _one_device(codes, scales=scales, codes_packed=codes_packed, scales_packed=scales_packed)
    return _run("moe_pack_w4", bind, codes, (
        _u8(codes, "codes"), _ptr(scales, "scales"), dtype_code(scales), int(fmt), L, N, 2 * half, group,
        _u8(codes_packed, "codes_packed"), _ptr(scales_packed, "scales_packed"), _stream(codes)))


def moe_grouped_gemv_w4(a, a_scales, codes_packed, scales_packed, fmt, counts, offsets, epi, out, bind=False):
    """a [rows_cap,K] (bf16, or e4m3fn with a_scales [rows_cap,K/128]) and the
    weights of moe_pack_w4 -> out [rows_cap,N] = G, or with MOE_EPI_SILU_MUL
    [rows_cap,N/2] = SiLU(gate) * up (fp32|bf16), on valid rows only."""
    L, N, half = codes_packed.shape
    rows_cap, K = a.shape[0], 2 * half
    _shape(a, "a", rows_cap, K)
    group = _group(K, scales_packed, "scales_packed")
    _shape(scales_packed, "scales_packed", L, N, K // group)
    fp8 = dtype_code(a) == MOE_FP8_E4M3
    _need(a_scales, "a_scales", fp8)
    if fp8:
        _shape(a_scales, "a_scales", rows_cap, K // 128)
    elif a_scales is not None:
        raise ValueError("a_scales goes with FP8 rows only")
    _shape(counts, "counts", L)
    _offsets(offsets, L)
    if int(epi) not in (MOE_EPI_STORE_G, MOE_EPI_SILU_MUL):
        raise ValueError(f"epi is {epi}, expected MOE_EPI_STORE_G or MOE_EPI_SILU_MUL")
    _shape(out, "out", rows_cap, N if int(epi) == MOE_EPI_STORE_G else N // 2)
    _one_device(a, a_scales=a_scales, codes_packed=codes_packed, scales_packed=scales_packed, counts=counts,
                offsets=offsets, out=out)
    return _run("moe_grouped_gemv_w4", bind, a, (
        _ptr(a, "a"), dtype_code(a), _f32(a_scales, "a_scales"), _u8(codes_packed, "codes_packed"),
        _ptr(scales_packed, "scales_packed"), dtype_code(scales_packed), int(fmt), group, _i32(counts, "counts"),
        _i32(offsets, "offsets"), L, rows_cap, N, K, int(epi), _ptr(out, "out"), dtype_code(out), _stream(a)))
