"""After the first call on a device no stand-alone operator loads code,
allocates, copies or synchronises (tests/operators_steady_child.py under
rocprofv3, as test_gpu_steady_state.py does for the layer)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from lora_expert_gemm_amd import profiling  # noqa: E402

pytestmark = pytest.mark.gpu

LAUNCH_ONLY = {"hipLaunchKernel", "__hipPushCallConfiguration", "__hipPopCallConfiguration",
               "hipGetLastError", "hipFuncSetAttribute", "hipGetDevice"}


@pytest.mark.skipif(shutil.which("rocprofv3") is None, reason="rocprofv3 not installed")
def test_operators_load_and_allocate_nothing_after_the_first_call(tmp_path):
    out = tmp_path / "trace"
    cmd = ["rocprofv3", "--hip-trace", "--hsa-trace", "--memory-allocation-trace",
           "--kernel-trace", "-f", "csv", "-d", str(out), "-o", "steady", "--",
           sys.executable, os.path.join(ROOT, "tests", "operators_steady_child.py")]
    print("[steady] " + " ".join(cmd), flush=True)
    p = subprocess.run(cmd, cwd="/tmp", env=dict(os.environ, TMPDIR="/tmp"),
                       capture_output=True, text=True, timeout=110)
    # (the profiler may exit non-zero after a complete run; the child's own
    # last line and the trace files decide)
    assert "[child] done" in p.stdout, (p.stdout[-3000:], p.stderr[-3000:])
    n = int(p.stdout.split("[child] done: ")[1].split()[0])
    w = profiling.steady_window(str(out))
    assert w["forbidden_inside"] == {}, w["forbidden_inside"]
    assert w["alloc_inside"] == {}, w["alloc_inside"]
    extra = set(w["hip_inside"]) - LAUNCH_ONLY
    assert not extra, {k: w["hip_inside"][k] for k in extra}
    assert w["hip_inside"].get("hipLaunchKernel", 0) >= n
