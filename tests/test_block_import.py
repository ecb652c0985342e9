"""The package without libmoe_block.so: the share's entry points work, and the
block's say what is missing where they are called."""
import os
import shutil
import subprocess
import sys
from pathlib import Path

ROOT = Path(__file__).resolve().parents[1]

PROGRAM = """
import combine_top_expert_amd as ep
from combine_top_expert_amd.pipeline import LayerShape, MoELayer
assert ep.moe_abi_version() >= 9 and ep.moe_dispatch_layout_workspace_bytes(128, 8, 32) >= 0
for call in (ep.moe_block_abi_version, lambda: ep.moe_add_rms_norm_backward_workspace_bytes(4, 256),
             lambda: ep.block_lib.moe_pack_w4):
    try:
        call()
    except ImportError as e:
        assert "libmoe_block.so" in str(e) and "not built" in str(e), e
    else:
        raise SystemExit("no error")
print("fine")
"""


def test_share_without_the_block_library(tmp_path):
    pkg = tmp_path / "combine_top_expert_amd"
    pkg.mkdir()
    src = ROOT / "combine_top_expert_amd"
    if not (src / "libmoe_ep.so").exists():
        import __graft_entry__
        __graft_entry__._build_module().build(verbose=False)
    for f in [*src.glob("*.py"), src / "libmoe_ep.so"]:
        shutil.copy(f, pkg / f.name)
    env = {k: v for k, v in os.environ.items() if k not in ("MOE_BLOCK_LIB", "MOE_EP_LIB")}
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, env=env, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr
