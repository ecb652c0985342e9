"""Python binding of libmoe_experts.so -- what trains and serves the experts'
weights: rows and weights in microscaled 4 bits (MX4), the experts' products of
both, and the AdamW step.

The same manner as the package's other entry points (argument marshalling
only; every name here is also a name of the package), with all tensors of a
call on one device, which need not be the current one.
"""
from __future__ import annotations

import ctypes
import os
from pathlib import Path

import torch

from . import MOE_EPI_SILU_MUL, MOE_EPI_STORE_G, MOE_F32, MOE_FP8_E4M3, MoEError, _need, _offsets
from .block import (_CODE, _F32, _FP8, _I32, _INT_MAX, _REAL, _U8, _current_device, _pointers, _raw_stream,
                    _too_large)

__all__ = [
    "EXPERTS_LIB_PATH", "experts_lib", "moe_experts_abi_version", "moe_quantize_mx4", "moe_permute_mx4", "moe_pack_mx4",
    "moe_grouped_gemm_mx4", "moe_adamw_step",
]

EXPERTS_LIB_PATH = Path(os.environ.get("MOE_EXPERTS_LIB", Path(__file__).resolve().parent / "libmoe_experts.so"))


class _NotBuilt:
    """In the library's place where it is missing: a program that uses the other
    libraries needs none of it, and one that calls into it is told."""

    def __getattr__(self, name):
        raise ImportError(f"{name}: {EXPERTS_LIB_PATH} is not built; run `python combine_top_expert_amd/build.py` "
                          "(these operators have no fallback without their HIP library)")


if EXPERTS_LIB_PATH.exists():
    experts_lib = ctypes.CDLL(str(EXPERTS_LIB_PATH))
elif "MOE_EXPERTS_LIB" in os.environ:                # asked for by name
    raise ImportError(f"MOE_EXPERTS_LIB={EXPERTS_LIB_PATH} is not built")
else:
    experts_lib = _NotBuilt()

_p, _i, _i64, _dbl = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double


class AdamwTensor(ctypes.Structure):
    """moe_adamw_tensor"""
    _fields_ = [("param", _p), ("master", _p), ("grad", _p), ("exp_avg", _p), ("exp_avg_sq", _p), ("exp_avg_scale", _p),
                ("exp_avg_sq_scale", _p), ("n", _i64)]


class AdamwConfig(ctypes.Structure):
    """moe_adamw_config"""
    _fields_ = [("lr", _dbl), ("beta1", _dbl), ("beta2", _dbl), ("eps", _dbl), ("weight_decay", _dbl), ("step", _i64),
                ("lr_device", _p), ("step_device", _p), ("grad_scale", _p), ("seed", ctypes.c_uint32)]


_SIG = {
    "moe_experts_abi_version": (_i, []),
    "moe_quantize_mx4": (_i, [_p, _i, _i64, _i, _p, _p, _p, _p]),
    "moe_permute_mx4": (_i, [_p, _i, _i, _i, _i, _p, _i64, _p, _p, _p]),
    "moe_pack_mx4": (_i, [_p, _p, _i, _i, _i, _p, _p, _p]),
    "moe_grouped_gemm_mx4": (_i, [_p, _p, _p, _p, _p, _p, _i, _i64, _i, _i, _i, _p, _i, _p, _p]),
    "moe_adamw_step": (_i, [_p, _i, _i, _i, _i, _p, _p]),
}
for _name, (_res, _args) in _SIG.items() if EXPERTS_LIB_PATH.exists() else ():
    if not hasattr(experts_lib, _name):
        raise ImportError(f"{EXPERTS_LIB_PATH} lacks {_name}: it predates these sources; rebuild with "
                          "`python combine_top_expert_amd/build.py`")
    _f = getattr(experts_lib, _name)
    _f.restype, _f.argtypes = _res, _args


def moe_experts_abi_version() -> int:
    return int(experts_lib.moe_experts_abi_version())


class _Calls(dict):
    """The entry points, looked up in the library once."""

    def __missing__(self, name):
        self[name] = getattr(experts_lib, name)
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


# ---------------------------------------------------------------- rows and weights in MX4

def moe_quantize_mx4(x, codes, scales, values=None, bind=False):
    """x [..,K] (fp32|bf16) -> codes [..,K/2] uint8 (two a byte, the even column
    low) and scales [..,K/32] uint8 (a power of two per 32 columns), and values
    [..,K] of x's dtype: what the codes stand for (may be x itself)."""
    K = x.shape[-1]
    rows = x.numel() // K if K else 0
    if K > _INT_MAX:
        _too_large("moe_quantize_mx4")
    lead, dt = x.shape[:-1], (x.dtype,) if x.dtype in _REAL else _REAL
    dev, (px, pc, ps, pv) = _pointers(
        ("x", x, dt, x.shape), ("codes", codes, _U8, (*lead, K // 2)), ("scales", scales, _U8, (*lead, K // 32)),
        ("values", values, dt, x.shape))
    return _run("moe_quantize_mx4", bind, dev, (px, _CODE[x.dtype], rows, K, pc, ps, pv, _raw_stream(dev)))


def moe_permute_mx4(x, slot_of, buf, buf_scales, bind=False):
    """x [T,H] (fp32|bf16), slot_of [T,K] -> buf [rows_cap,H/2] and buf_scales
    [rows_cap,H/32] uint8: each token's row in MX4 at its slots."""
    T, H = x.shape
    K, cap = slot_of.shape[1], buf.shape[0]
    if max(T, H, K) > _INT_MAX:
        _too_large("moe_permute_mx4")
    dev, (px, psl, pb, pbs) = _pointers(
        ("x", x, _REAL, (T, H)), ("slot_of", slot_of, _I32, (T, K)), ("buf", buf, _U8, (cap, H // 2)),
        ("buf_scales", buf_scales, _U8, (cap, H // 32)))
    return _run("moe_permute_mx4", bind, dev, (px, _CODE[x.dtype], T, K, H, psl, cap, pb, pbs, _raw_stream(dev)))


def moe_pack_mx4(codes, scales, codes_packed, scales_packed, bind=False):
    """codes [L,N,K/2] and scales [L,N,K/32] (uint8, as moe_quantize_mx4 writes
    them) -> the same in the order that moe_grouped_gemm_mx4 reads (same shapes)."""
    L, N, half = codes.shape
    if max(L, N, 2 * half) > _INT_MAX:
        _too_large("moe_pack_mx4")
    per = (L, N, half // 16)
    dev, (pc, ps, qc, qs) = _pointers(
        ("codes", codes, _U8, (L, N, half)), ("scales", scales, _U8, per), ("codes_packed", codes_packed, _U8, (L, N, half)),
        ("scales_packed", scales_packed, _U8, per))
    return _run("moe_pack_mx4", bind, dev, (pc, ps, L, N, 2 * half, qc, qs, _raw_stream(dev)))


def moe_grouped_gemm_mx4(a, a_scales, codes_packed, scales_packed, counts, offsets, epi, out, out_scales=None, bind=False):
    """a [rows_cap,K/2] and a_scales [rows_cap,K/32] (MX4 rows) and the weights of
    moe_pack_mx4 -> out [rows_cap,N] = G, or with MOE_EPI_SILU_MUL [rows_cap,N/2] =
    SiLU(gate) * up (fp32|bf16), on valid rows only.  With out_scales
    [rows_cap,N/64] uint8, out [rows_cap,N/4] uint8 is that product in MX4."""
    L, N, half = codes_packed.shape
    rows_cap, K = a.shape[0], 2 * half
    if max(L, N, K) > _INT_MAX:
        _too_large("moe_grouped_gemm_mx4")
    if epi not in (MOE_EPI_STORE_G, MOE_EPI_SILU_MUL):
        raise ValueError(f"epi is {epi}, expected MOE_EPI_STORE_G or MOE_EPI_SILU_MUL")
    _offsets(offsets, L)
    mx4 = out_scales is not None
    if mx4 and epi != MOE_EPI_SILU_MUL:
        raise ValueError("out_scales goes with MOE_EPI_SILU_MUL only")
    cols = N if epi == MOE_EPI_STORE_G else N // 4 if mx4 else N // 2
    dev, (pa, pas, pc, ps, pn, po, pout, pos) = _pointers(
        ("a", a, _U8, (rows_cap, half)), ("a_scales", a_scales, _U8, (rows_cap, half // 16)),
        ("codes_packed", codes_packed, _U8, (L, N, half)), ("scales_packed", scales_packed, _U8, (L, N, half // 16)),
        ("counts", counts, _I32, (L,)), ("offsets", offsets, _I32, offsets.shape),
        ("out", out, _U8 if mx4 else _REAL, (rows_cap, cols)), ("out_scales", out_scales, _U8, (rows_cap, N // 64)))
    return _run("moe_grouped_gemm_mx4", bind, dev, (
        pa, pas, pc, ps, pn, po, L, rows_cap, N, K, epi, pout, _CODE[out.dtype], pos, _raw_stream(dev)))


# ---------------------------------------------------------------- AdamW

def _list(name, tensors, sizes, device, dtypes, written=True):
    """Data pointers of a list of tensors of one dtype, with these numbers of elements."""
    if len(tensors) != len(sizes):
        raise ValueError(f"{name} has {len(tensors)} tensors, expected {len(sizes)}")
    dtype = tensors[0].dtype
    if (dtype not in dtypes or [t.numel() for t in tensors] != sizes or {t.dtype for t in tensors} != {dtype}
            or {t.get_device() for t in tensors} != {device} or not all(t.is_contiguous() for t in tensors)):
        for i, (t, n) in enumerate(zip(tensors, sizes)):
            if t.dtype != dtype or dtype not in dtypes:
                raise TypeError(f"{name}[{i}] has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}, one for all")
            if t.get_device() != device:
                raise ValueError(f"{name}[{i}] is on {t.device}, expected cuda:{device}")
            if t.numel() != n:
                raise ValueError(f"{name}[{i}] has {t.numel()} elements, expected {n}")
            if not t.is_contiguous():
                raise ValueError(f"{name}[{i}] must be contiguous")
    pointers = [t.data_ptr() for t in tensors]
    if written and len(set(pointers)) < len(pointers):                 # one update would race with the other
        some = [v for v, n in zip(pointers, sizes) if n]
        if len(set(some)) < len(some):
            raise ValueError(f"{name} holds the same tensor twice")
    return pointers


def _distinct(lists, sizes):
    """Refuse a tensor that two of these lists of pointers name (each names it once at most)."""
    if 0 in sizes:
        lists = [[v for v, n in zip(pointers, sizes) if n] for pointers in lists]
    used = [pointers for pointers in lists if any(pointers)]
    if len(set().union(*used)) < sum(map(len, used)):
        raise ValueError("params, masters, exp_avgs, exp_avg_sqs and their scales name the same tensor twice")


def _scalar(name, t, dtype, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.numel() != 1 or t.get_device() != device:
        raise ValueError(f"{name} must be one value on cuda:{device}")
    return t.data_ptr()


class _AdamwCall:
    """A marshalled moe_adamw_step: called with other lr or step numbers, or none."""

    def __init__(self, device, table, dtypes, config, stream):
        self._args, self._config, self._device, self._stream = (table, len(table), *dtypes), config, device, stream

    def __call__(self, step=None, lr=None):
        if step is not None:
            _number(self._config, "step", step)
        if lr is not None:
            _number(self._config, "lr", lr)
        _run("moe_adamw_step", False, self._device, (*self._args, ctypes.byref(self._config), self._stream))


def _number(config, name, v):
    if name == "step" and not -1 << 63 <= v < 1 << 63:
        _too_large("moe_adamw_step")
    if getattr(config, name + "_device"):
        raise ValueError(f"{name} of this call is a device tensor")
    setattr(config, name, v)


def moe_adamw_step(params, grads, exp_avgs, exp_avg_sqs, lr, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                   masters=None, exp_avg_scales=None, exp_avg_sq_scales=None, grad_scale=None, seed=0, bind=False):
    """One AdamW update, in place, of the lists params (fp32|bf16), exp_avgs and
    exp_avg_sqs (fp32; or e4m3fn codes of m and sqrt(v), with the fp32 lists
    exp_avg_scales and exp_avg_sq_scales of ceil(n/128) each) from the list
    grads (fp32|bf16).  masters: fp32 copies that are updated in place of bf16
    params, which become their rounded copies.  lr and step (1 for the first
    update): numbers, or device tensors (fp32, int64) that are read when the
    step runs, as a captured step needs.  grad_scale: fp32 device tensor, a
    factor of every gradient; not finite, the step is skipped.  seed (32 bits):
    of the 8-bit rounding.  With bind the callable takes later step and lr
    numbers (call(step=2)); the tensors must stay alive."""
    if not len(params):
        return (lambda step=None, lr=None: None) if bind else None
    device = params[0].get_device()
    if device < 0:
        raise ValueError("params must be device tensors")
    sizes = [t.numel() for t in params]
    s8 = len(exp_avgs) > 0 and exp_avgs[0].dtype in _FP8
    state, blocks = (_FP8, [(n + 127) // 128 for n in sizes]) if s8 else (_F32, None)
    _need(exp_avg_scales, "exp_avg_scales", s8)
    _need(exp_avg_sq_scales, "exp_avg_sq_scales", s8)
    if not s8 and (exp_avg_scales is not None or exp_avg_sq_scales is not None):
        raise ValueError("exp_avg_scales and exp_avg_sq_scales go with 8-bit states only")
    zeros = [0] * len(sizes)
    lists = (
        _list("params", params, sizes, device, _REAL),
        zeros if masters is None else _list("masters", masters, sizes, device, _F32),
        _list("grads", grads, sizes, device, _REAL, written=False),
        _list("exp_avgs", exp_avgs, sizes, device, state), _list("exp_avg_sqs", exp_avg_sqs, sizes, device, state),
        _list("exp_avg_scales", exp_avg_scales, blocks, device, _F32) if s8 else zeros,
        _list("exp_avg_sq_scales", exp_avg_sq_scales, blocks, device, _F32) if s8 else zeros, sizes)
    _distinct(lists[:2] + lists[3:7], sizes)
    table = (AdamwTensor * len(sizes))(*zip(*lists))
    if not 0 <= seed < 1 << 32:
        raise ValueError(f"seed is {seed}, expected 32 bits")
    config = AdamwConfig(beta1=betas[0], beta2=betas[1], eps=eps, weight_decay=weight_decay, seed=seed)
    if isinstance(lr, torch.Tensor):
        config.lr_device = _scalar("lr", lr, torch.float32, device)
    else:
        _number(config, "lr", lr)
    if isinstance(step, torch.Tensor):
        config.step_device = _scalar("step", step, torch.int64, device)
    else:
        _number(config, "step", step)
    if grad_scale is not None:
        config.grad_scale = _scalar("grad_scale", grad_scale, torch.float32, device)
    call = _AdamwCall(device, table, (_CODE[params[0].dtype], _CODE[grads[0].dtype], MOE_FP8_E4M3 if s8 else MOE_F32),
                      config, _raw_stream(device))
    return call if bind else call()
