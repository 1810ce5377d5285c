"""The checked build's device checks decide something: no kernel calls one and
goes on with the access whatever it says."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_result_of_every_check_is_used():
    checks, found = r"(?:dbg_ok|(?:a|work)\.has_\w+)", 0
    for path in glob.glob(os.path.join(ROOT, "block_sparse_attention_28_b200", "csrc", "*.cuh")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        found += len(re.findall(checks + r"\(", text))
        alone = re.findall(r"(?:[;{}]|\bif \(\w+\)|\belse)\s*" + checks + r"\([^\n]*", text)
        assert not alone, (os.path.basename(path), alone)
    assert found > 20
