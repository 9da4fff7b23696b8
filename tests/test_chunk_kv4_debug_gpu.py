"""The suites of rotary positions and of chunks over the 4-bit cache once more under the bounds-checking debug
build (see test_debug_build_gpu.py), in child processes that load libdiffattn_debug.so."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("suite", ["test_rope_gpu.py", "test_chunk_kv4_gpu.py"])
def test_suite_under_the_debug_build(suite):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, DIFFATTN_DEBUG_BUILD="1")
    build = subprocess.run([sys.executable, "-c", "import differential_attention_gb300 as da; print(da.build())"],
                           cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert build.returncode == 0, build.stdout[-2000:] + build.stderr[-4000:]
    run = subprocess.run([sys.executable, "-m", "pytest", f"tests/{suite}", "-m", "gpu", "-x", "-q", "-p",
                          "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert run.returncode == 0, run.stdout[-4000:] + run.stderr[-2000:]
    assert " passed" in run.stdout
