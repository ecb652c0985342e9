"""C-ABI and binding checks of libmoe_block.so that need no GPU: exports,
header, and refusals (all before any HIP runtime call)."""
import ctypes
import os
import re
import subprocess
import sys
from pathlib import Path

import pytest
import torch

ROOT = Path(__file__).resolve().parents[1]
HEADER = ROOT / "include" / "moe_block.h"
LIB = ROOT / "combine_top_expert_amd" / "libmoe_block.so"
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
F32, BF16, FP8 = 0, 1, 2
INF, NAN = float("inf"), float("nan")


def declared_functions():
    return sorted(set(re.findall(r"^\s*(?:moe_status|size_t|int)\s+(moe_\w+)\s*\(", HEADER.read_text(), flags=re.M)))


@pytest.fixture(scope="module")
def ep():
    if not LIB.exists():
        import __graft_entry__
        __graft_entry__._build_module().build(verbose=False)
    import combine_top_expert_amd as ep
    return ep


def P(v=256):
    return ctypes.c_void_p(v) if v else None


def test_exports_are_the_header(ep):
    out = subprocess.run(["nm", "-D", "--defined-only", str(LIB)], capture_output=True, text=True).stdout
    assert set(re.findall(r" T (\w+)$", out, flags=re.M)) - {"_init", "_fini"} == set(declared_functions())
    assert len(declared_functions()) == 9
    for name in declared_functions():
        assert callable(getattr(ep, name)) and name in ep.__all__
    assert ep.moe_block_abi_version() == 1


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "moe_block.h"\nint main(void) { return moe_block_abi_version == 0; }\n')
    r = subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{ROOT / 'include'}", "-c", str(src),
                        "-o", str(tmp_path / "t.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_import_fails_loudly_without_library(tmp_path):
    env = dict(os.environ, MOE_BLOCK_LIB=str(tmp_path / "missing.so"))
    r = subprocess.run([sys.executable, "-c", "import combine_top_expert_amd"], cwd=ROOT, env=env,
                       capture_output=True, text=True)
    assert r.returncode != 0 and "not built" in r.stderr


def test_norm_refusals(ep):
    def call(x=256, res=256, xdt=BF16, w=256, wdt=BF16, eps=1e-6, T=4, H=256, h=512, y=768, y8=None, sc=None):
        return ep.block_lib.moe_add_rms_norm(P(x), P(res), xdt, P(w), wdt, eps, T, H, P(h), P(y), P(y8), P(sc), None)
    assert call(T=0, x=None, w=None) == OK
    assert call(T=-1) == INVALID and call(H=0) == INVALID
    assert call(H=252) == UNSUPPORTED and call(H=16392) == UNSUPPORTED and call(T=(1 << 30) + 1) == UNSUPPORTED
    assert call(H=136, y8=512, sc=512) == UNSUPPORTED              # FP8 groups of 128
    assert call(y8=512) == INVALID and call(sc=512) == INVALID     # codes and scales go together
    assert call(h=None, y=None) == INVALID                         # nothing to write
    assert call(h=512, y=512) == INVALID
    assert call(x=None) == INVALID and call(w=None) == INVALID
    assert call(xdt=FP8) == UNSUPPORTED and call(wdt=FP8) == UNSUPPORTED and call(xdt=9) == INVALID
    for eps in (-1e-6, INF, NAN):
        assert call(eps=eps) == INVALID
    for name in ("x", "res", "w", "h", "y"):
        assert call(**{name: 520}) == INVALID, name                # 16-byte alignment
    assert call(y8=520, sc=512) == INVALID


def test_norm_backward_refusals(ep):
    need = ep.moe_add_rms_norm_backward_workspace_bytes
    assert need(4, 256) > 0 and need(0, 256) == 0 and need(-1, 256) == 0 and need(4, 252) == 0 and need((1 << 30) + 1, 8) == 0
    assert need(100000, 4096) < 64 << 20                           # bounded for long batches

    def call(dy=256, h=256, dh=256, dt=BF16, w=256, wdt=F32, eps=1e-6, T=4, H=256, dx=512, dw=512, ws=256, wsb=1 << 20):
        return ep.block_lib.moe_add_rms_norm_backward(P(dy), P(h), P(dh), dt, P(w), wdt, eps, T, H, P(dx), P(dw), P(ws),
                                                      wsb, None)
    assert call(H=100) == UNSUPPORTED and call(H=20000) == UNSUPPORTED and call(T=(1 << 30) + 1) == UNSUPPORTED
    assert call(dt=FP8) == UNSUPPORTED and call(wdt=FP8) == UNSUPPORTED and call(dt=-1) == INVALID
    assert call(wsb=need(4, 256) - 1) == WORKSPACE
    assert call(eps=-1.0) == INVALID and call(T=-1) == INVALID
    for name in ("dy", "h", "w", "dx", "dw", "ws"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: 264}) == INVALID, name


def test_route_refusals(ep):
    def call(lg=256, T=4, E=64, K=8, score=1, n=8, keep=4, top=2, scale=1.0, ids=256, w=256):
        return ep.block_lib.moe_router_group_topk(P(lg), None, T, E, K, score, n, keep, top, 1, scale, P(ids), P(w), None)
    assert call(T=0, lg=None, ids=None, w=None) == OK
    assert call(K=0) == INVALID and call(K=65) == INVALID
    assert call(K=33, n=1, keep=1) == UNSUPPORTED
    assert call(E=2048, n=1, keep=1) == UNSUPPORTED and call(T=(1 << 30) + 1) == UNSUPPORTED
    assert call(n=7) == UNSUPPORTED                                # E % n_group
    assert call(n=0) == INVALID and call(n=128) == INVALID and call(keep=9) == INVALID and call(keep=0) == INVALID
    assert call(E=1024, n=128, keep=4) == UNSUPPORTED              # more groups than lanes
    assert call(K=9, keep=1) == INVALID                            # more experts than the kept groups hold
    assert call(top=0) == INVALID and call(top=3) == INVALID and call(score=2) == INVALID
    assert call(scale=NAN) == INVALID and call(scale=INF) == INVALID
    for name in ("lg", "ids", "w"):
        assert call(**{name: None}) == INVALID

    def bw(lg=256, ids=256, dw=256, T=4, E=64, K=8, score=1, scale=1.0, dl=512):
        return ep.block_lib.moe_router_group_topk_backward(P(lg), P(ids), P(dw), T, E, K, score, 1, scale, P(dl), None)
    assert bw(T=0, lg=None, ids=None, dw=None, dl=None) == OK
    assert bw(T=(1 << 30) + 1) == UNSUPPORTED
    assert bw(K=33) == UNSUPPORTED and bw(E=1025) == UNSUPPORTED and bw(K=0) == INVALID and bw(score=-1) == INVALID
    assert bw(dl=256) == INVALID and bw(scale=NAN) == INVALID
    for name in ("lg", "ids", "dw", "dl"):
        assert bw(**{name: None}) == INVALID


def test_permute_fp8_refusals(ep):
    def call(x=256, xs=256, T=4, K=2, H=256, slot=256, cap=8, buf=512, bs=512):
        return ep.block_lib.moe_permute_fp8(P(x), P(xs), T, K, H, P(slot), cap, P(buf), P(bs), None)
    assert call(T=0, x=None) == OK and call(cap=0, x=None) == OK
    assert call(H=192) == UNSUPPORTED and call(K=65) == UNSUPPORTED
    assert call(K=0) == INVALID and call(H=0) == INVALID and call(T=-1) == INVALID and call(cap=-1) == INVALID
    for name in ("x", "xs", "slot", "buf", "bs"):
        assert call(**{name: None}) == INVALID
    assert call(x=264) == INVALID and call(buf=264) == INVALID
    assert call(T=1 << 30, H=1 << 14) == UNSUPPORTED               # grid


def test_w4_refusals(ep):
    def pack(c=256, s=256, sdt=F32, fmt=0, L=2, N=128, K=256, group=128, cp=512, sp=512):
        return ep.block_lib.moe_pack_w4(P(c), P(s), sdt, fmt, L, N, K, group, P(cp), P(sp), None)

    def gemv(a=256, adt=BF16, asc=None, c=256, s=256, sdt=F32, fmt=0, group=128, cnt=256, off=256, L=2, cap=16, N=128,
             K=256, epi=0, out=512, odt=BF16):
        return ep.block_lib.moe_grouped_gemv_w4(P(a), adt, P(asc), P(c), P(s), sdt, fmt, group, P(cnt), P(off), L, cap, N,
                                                K, epi, P(out), odt, None)
    for f in (pack, gemv):
        assert f(N=64) == UNSUPPORTED and f(K=192) == UNSUPPORTED and f(L=1025) == UNSUPPORTED
        assert f(N=1 << 16, K=(1 << 15) + 128) == UNSUPPORTED and f(N=128, K=(1 << 24) + 128) == UNSUPPORTED
        assert f(group=16) == UNSUPPORTED and f(group=256) == UNSUPPORTED and f(group=0) == UNSUPPORTED
        assert f(sdt=FP8) == UNSUPPORTED and f(sdt=7) == INVALID and f(fmt=2) == INVALID
        assert f(L=0) == INVALID and f(N=0) == INVALID and f(K=-128) == INVALID
    assert pack(cp=256) == INVALID and pack(sp=256) == INVALID     # in place
    for name in ("c", "s", "cp", "sp"):
        assert pack(**{name: None}) == INVALID
    assert pack(c=264) == INVALID and pack(cp=264) == INVALID and pack(sp=264) == INVALID
    assert gemv(cap=0, a=None, out=None) == OK
    assert gemv(cap=-1) == INVALID and gemv(epi=2) == INVALID
    assert gemv(adt=F32) == UNSUPPORTED and gemv(odt=FP8) == UNSUPPORTED and gemv(adt=5) == INVALID
    assert gemv(adt=FP8) == INVALID                                # FP8 rows without scales
    for name in ("a", "c", "s", "cnt", "off", "out"):
        assert gemv(**{name: None}) == INVALID
    for name in ("a", "c", "s", "out"):
        assert gemv(**{name: 264}) == INVALID


# ---------------------------------------------------------------- the binding

def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


def refused(match, fn, *args, exc=ValueError, **kw):
    with pytest.raises(exc, match=match):
        fn(*args, **kw)


def test_binding_checks(ep):
    x, w = z(4, 256, dtype=BF), z(256, dtype=BF)
    ok = "device tensor"
    refused(ok, ep.moe_add_rms_norm, x, x, w, 1e-6, x, z(4, 256, dtype=BF), z(4, 256, dtype=U8), z(4, 2))
    refused("shape", ep.moe_add_rms_norm, x, z(5, 256, dtype=BF), w, 1e-6, x)
    refused("shape", ep.moe_add_rms_norm, x, None, z(128), 1e-6, None, x)
    refused("shape", ep.moe_add_rms_norm, x, None, w, 1e-6, None, None, z(4, 256, dtype=U8), z(4, 1))
    refused("required", ep.moe_add_rms_norm, x, None, w, 1e-6, None, None, z(4, 256, dtype=U8))
    refused("dtype", ep.moe_add_rms_norm, x, z(4, 256), w, 1e-6, x, exc=TypeError)
    ws = z(1 << 20, dtype=U8)
    refused(ok, ep.moe_add_rms_norm_backward, x, x, w, 1e-6, x, z(256), ws)
    refused("shape", ep.moe_add_rms_norm_backward, x, x, w, 1e-6, x, z(255), ws)
    refused("dtype", ep.moe_add_rms_norm_backward, x, z(4, 256), w, 1e-6, x, z(256), ws, exc=TypeError)
    lg, ids, wt = z(4, 16), z(4, 2, dtype=I32), z(4, 2)
    refused(ok, ep.moe_router_group_topk, lg, 2, ids, wt)
    refused("shape", ep.moe_router_group_topk, lg, 3, ids, wt)
    refused("shape", ep.moe_router_group_topk, lg, 2, ids, wt, bias=z(15))
    refused("float32", ep.moe_router_group_topk, z(4, 16, dtype=BF), 2, ids, wt, exc=TypeError)
    refused(ok, ep.moe_router_group_topk_backward, lg, ids, wt, z(4, 16))
    refused("shape", ep.moe_router_group_topk_backward, lg, ids, wt, z(4, 15))
    x8, xs, slot = z(4, 256, dtype=U8), z(4, 2), z(4, 3, dtype=I32)
    refused(ok, ep.moe_permute_fp8, x8, xs, slot, z(9, 256, dtype=U8), z(9, 2))
    refused("shape", ep.moe_permute_fp8, x8, z(4, 1), slot, z(9, 256, dtype=U8), z(9, 2))
    refused("shape", ep.moe_permute_fp8, x8, xs, slot, z(9, 256, dtype=U8), z(8, 2))
    refused("e4m3fn", ep.moe_permute_fp8, x, xs, slot, z(9, 256, dtype=U8), z(9, 2), exc=TypeError)
    c, s = z(2, 128, 128, dtype=U8), z(2, 128, 2)
    refused(ok, ep.moe_pack_w4, c, s, ep.MOE_W4_INT4, c.clone(), s.clone())
    refused("shape", ep.moe_pack_w4, c, s, ep.MOE_W4_INT4, z(2, 128, 64, dtype=U8), s.clone())
    refused("shape", ep.moe_pack_w4, c, z(2, 128, 3), ep.MOE_W4_INT4, c.clone(), s.clone())
    a, cnt, off = z(9, 256, dtype=BF), z(2, dtype=I32), z(3, dtype=I32)
    refused(ok, ep.moe_grouped_gemv_w4, a, None, c, s, 0, cnt, off, ep.MOE_EPI_STORE_G, z(9, 128))
    refused("shape", ep.moe_grouped_gemv_w4, a, None, c, s, 0, cnt, off, ep.MOE_EPI_SILU_MUL, z(9, 128))
    refused("shape", ep.moe_grouped_gemv_w4, z(9, 128, dtype=BF), None, c, s, 0, cnt, off, 0, z(9, 128))
    refused("required", ep.moe_grouped_gemv_w4, z(9, 256, dtype=U8), None, c, s, 0, cnt, off, 0, z(9, 128))
    refused("FP8", ep.moe_grouped_gemv_w4, a, z(9, 2), c, s, 0, cnt, off, 0, z(9, 128))
    refused("epi", ep.moe_grouped_gemv_w4, a, None, c, s, 0, cnt, off, 5, z(9, 128))
