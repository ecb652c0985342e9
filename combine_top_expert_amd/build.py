"""Build libmoe_ep.so and libmoe_block.so (gfx950) in-tree with hipcc.

    python combine_top_expert_amd/build.py [--jobs N]

(Run it as a script, not as ``-m combine_top_expert_amd.build``: importing the
package loads the library, which may be missing or stale before a build.)

Compiles every source under csrc/ and csrc/block/ to an object in _build/ (in
parallel) and links the two folders' objects into
combine_top_expert_amd/libmoe_ep.so and libmoe_block.so.  Always rebuilds.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
BUILD = PKG / "_build"
LIB = PKG / "libmoe_ep.so"
LIB_BLOCK = PKG / "libmoe_block.so"
ARCH = os.environ.get("MOE_OFFLOAD_ARCH", "gfx950")

# Packed fp32 (v_pk_*_f32) is turned off for all device code.
HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17", "-Wall",
    "-Wno-unused-function", "-Wno-unused-variable",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{ROOT / 'include'}", f"-I{CSRC}",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def _compile(src: Path) -> Path:
    obj = BUILD / ("_".join(src.relative_to(CSRC).parts).replace(".", "_") + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, "-c", str(src), "-o", str(obj)]
    if src.suffix == ".cpp":
        cmd.insert(1, "-x")
        cmd.insert(2, "hip")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    noisy = [ln for ln in r.stderr.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
    if noisy:
        print("\n".join(noisy), file=sys.stderr)
    return obj


def _link(objs, lib: Path) -> None:
    tmp = lib.with_suffix(".so.tmp")
    # --no-undefined: an unresolved symbol (e.g. a kernel stub the host pass
    # did not emit) fails the build instead of the first dlopen
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,--no-undefined", "-o", str(tmp),
           *map(str, objs)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


def build(jobs: int = 8, verbose: bool = True) -> Path:
    BUILD.mkdir(exist_ok=True)
    groups = {lib: sorted(list(d.glob("*.hip")) + list(d.glob("*.cpp")))
              for lib, d in ((LIB, CSRC), (LIB_BLOCK, CSRC / "block"))}
    srcs = [src for g in groups.values() for src in g]
    with ThreadPoolExecutor(max_workers=max(1, min(jobs, len(srcs)))) as ex:
        objs = dict(zip(srcs, ex.map(_compile, srcs)))
    for lib, g in groups.items():
        _link([objs[src] for src in g], lib)
        if verbose:
            print(f"built {lib} from {len(g)} sources")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=8)
    build(ap.parse_args().jobs)
