"""Calls of more waves than one grid holds are cut into several launches: each
slice of each token must be worked on once (queries turned in place twice would be
turned by twice the angle).  The host code of the launches runs here with the
runtime's launch replaced (append_parts_driver.cpp); no GPU is needed."""
import os
import subprocess

import pytest

from test_host_sanitizers import CSRC, ROOT, _hipcc


def test_every_slice_of_every_token_is_taken_once(tmp_path):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    flags = ["-xhip", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]
    objs = []
    for src in (os.path.join(CSRC, "kv_rope.hip"), os.path.join(CSRC, "rope.hip"),
                os.path.join(ROOT, "tests", "append_parts_driver.cpp")):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        res = subprocess.run([hipcc, *flags, "-c", src, "-o", objs[-1]], capture_output=True, text=True)
        assert res.returncode == 0, f"hipcc failed on {src}:\n{res.stderr[-4000:]}"
    exe = str(tmp_path / "append_parts")
    # (The kernels' code is not there, and not needed: its symbols stay unresolved.)
    res = subprocess.run([hipcc, *objs, "-Wl,--unresolved-symbols=ignore-all", "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, f"link failed:\n{res.stderr[-4000:]}"
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, f"driver failed (rc={run.returncode}):\n{run.stderr[-4000:]}"
    assert "every task once" in run.stdout
