"""The packed-MXFP4 tile kernels as their source has them: what no run on a
GPU can show."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_autoround_amd", "csrc")


def _code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_stages_are_read_before_the_epilogue_writes_over_them():
    # finish_tile writes where other wavefronts' fragments were.  A barrier alone does not tell that those reads are done:
    # each wavefront has to wait for its own first.
    code = _code("mxfp4_tiles.h")
    assert re.search(r"void lds_written_barrier\(\) \{ asm volatile\(\"s_waitcnt lgkmcnt\(0\)\\n\\ts_barrier\"", code)
    calls = [m.start() for m in re.finditer(r"(?<!void )finish_tile<", code)]
    assert len(calls) == 2
    for at in calls:
        barriers = re.findall(r"\b(\w*barrier)\(\);", code[:at])
        assert barriers[-1] == "lds_written_barrier"
