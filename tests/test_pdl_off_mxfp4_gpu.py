"""The MXFP4 calls and the few-token layer on a build whose launches never overlap their
predecessor (MOE_USE_PDL=0).

With the overlap on, the layer copies weights and ranks its entries before it waits for
the launch before; that is right only while the order of the call's launches makes it so.
With it off the order cannot matter.  The same tests have to pass on either build; the second one goes to a
temporary directory and is loaded by a child process through MOE_GB300_LIB."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CASES = ["tests/test_expert_layer_gpu.py", "tests/test_expert_layer_bounds_gpu.py",
         "tests/test_expert_gemm_mxfp4_gpu.py", "tests/test_mxfp4_gpu.py::test_dispatch",
         "tests/test_mxfp4_gpu.py::test_graph_and_streams", "tests/test_mxfp4_long_sums_gpu.py",
         "tests/test_pdl_off_gpu.py::test_loaded_library_is_the_requested_build"]


@pytest.mark.timeout(1800)
def test_with_pdl_off(tmp_path):
    from combine_moe_plan_02_gb300 import build
    lib = build.build(force=True, out=str(tmp_path / "libmoe_gb300_nopdl.so"),
                      build_dir=str(tmp_path / "obj"), defines=("MOE_USE_PDL=0",))
    env = dict(os.environ, MOE_GB300_LIB=lib)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu",
                        "-p", "no:cacheprovider", *CASES],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1700)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "skipped" not in r.stdout.splitlines()[-1]
