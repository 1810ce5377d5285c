"""The tests of drafts, page lists and table widths once more under the checked
build: none of them records a failed check (each asks for the device error)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FILES = ["test_gpu_cache_drafts.py", "test_gpu_cache_lists.py", "test_gpu_cache_widths.py", "test_gpu_cache_values.py"]


@pytest.mark.gpu
def test_the_checked_build_runs_them(tmp_path):
    env = dict(os.environ, STA_CHECKED="1")
    asks = [sys.executable, "-c", "import block_sparse_attention_28_b200 as s; assert s.sta_debug_build() == 1"]
    subprocess.run(asks, env=env, cwd=ROOT, check=True, timeout=300)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-k", "not costs_little"] +
                       [os.path.join(ROOT, "tests", f) for f in FILES], env=env, cwd=ROOT, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
