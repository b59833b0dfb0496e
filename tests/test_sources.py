"""Rules that the device code keeps (read from its sources; no GPU needed)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_tree_verification_amd", "csrc")


def test_no_instruction_is_written_in_assembly():
    """The compiler counts the cycles that a matrix product's result needs before an instruction may read it, on
    every path to that instruction, but only for instructions of its own. (An empty template hides a value from
    it and is no instruction.)"""
    files = sorted(glob.glob(os.path.join(CSRC, "*.h*")))
    assert len(files) > 10
    for f in files:
        text = re.sub(r"//[^\n]*", "", open(f).read())
        for m in re.finditer(r"\basm\b\s*(?:volatile\s*)?\(\s*\"([^\"]*)\"", text):
            assert m.group(1) == "", f"{os.path.basename(f)}: {m.group(0)}"
        assert len(re.findall(r"\basm\b", text)) == len(re.findall(r"\basm\b\s*(?:volatile\s*)?\(\s*\"\"", text)), f
