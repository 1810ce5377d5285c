"""What the build looks at to tell whether a library is up to date."""
import os
import re
import runpy
import shutil

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILD = os.path.join(ROOT, "block_sparse_attention_28_b200", "build.py")


def included(path, seen):
    """path and every file of the repository that it includes, directly or not."""
    path = os.path.realpath(path)
    if path in seen:
        return seen
    seen.add(path)
    for name in re.findall(r'^\s*#\s*include\s+"([^"]+)"', open(path).read(), re.M):
        of = os.path.join(os.path.dirname(path), name)
        assert os.path.exists(of), (path, name)
        included(of, seen)
    return seen


def test_every_included_file_is_a_source():
    """A change to any file that a library is compiled from makes it out of
    date, headers next to the kernels included."""
    b = runpy.run_path(BUILD, run_name="sta_build")
    known = {os.path.realpath(p) for p in b["sources"]()}
    for src, _, _ in b["TARGETS"]:
        missing = included(src, set()) - known
        assert not missing, missing


def test_a_change_to_any_file_makes_a_library_out_of_date(tmp_path):
    """In a copy whose files are all older than the library, each one in turn
    is changed after it."""
    package = tmp_path / "block_sparse_attention_28_b200"
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    shutil.copytree(os.path.join(os.path.dirname(BUILD), "csrc"), package / "csrc")
    shutil.copy(BUILD, package)
    b = runpy.run_path(str(package / "build.py"), run_name="sta_build")
    out = package / "libsta.so"
    out.write_bytes(b"")
    files = included(b["SRC"], set()) | included(b["PROBE_SRC"], set())
    assert any(os.path.basename(f) == "sta_cache_index.h" for f in files)
    for f in files:
        os.utime(f, (1000, 1000))
    for p in b["sources"]():
        os.utime(p, (1000, 1000))
    os.utime(out, (2000, 2000))
    assert b["up_to_date"](str(out))
    for f in files:
        os.utime(f, (3000, 3000))
        assert not b["up_to_date"](str(out)), f
        os.utime(f, (1000, 1000))
