"""The checked build (device-side checks of indices and addresses) runs the
cache calls without recording a failed check, bit-identical to the product
build."""
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(path, checked):
    env = dict(os.environ, STA_CHECKED="1" if checked else "0")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "_checked_cache_cases.py"), str(path)], env=env,
                       cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return dict(np.load(path))


@pytest.mark.gpu
def test_checked_build_agrees_on_the_cache(tmp_path):
    chk, prod = _run(tmp_path / "checked.npz", True), _run(tmp_path / "product.npz", False)
    assert int(chk.pop("debug_build")) == 1 and int(prod.pop("debug_build")) == 0
    statuses = {k: (int(chk[k]), int(prod[k])) for k in chk if k.startswith("status_")}
    assert statuses and all(v == (0, 0) for v in statuses.values()), statuses
    assert sorted(chk) == sorted(prod)
    for k in chk:
        equal = np.array_equal(chk[k], prod[k], equal_nan=chk[k].dtype.kind == "f")
        assert chk[k].shape == prod[k].shape and equal, k
