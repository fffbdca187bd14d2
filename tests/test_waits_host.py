"""No bounded wait of the kernels may run out unseen: a wait without a status word to report to
has its result looked at.  (A source check: a GPU wait that runs out is not provoked.)"""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "grouped_expert_gemm_gb300", "csrc")


def unseen(text):
    """Statements that are a wait with a null status word and nothing more."""
    return re.findall(r"[;{}]\s*((?:\w+\.)?wait(?:_bounded(?:<\w+>)?)?\([^;]*\bnullptr\b[^;]*\);)",
                      re.sub(r"//[^\n]*", "", text))


def test_no_wait_runs_out_unseen():
    assert unseen("f();\n  ring.wait(flag, nullptr);") == ["ring.wait(flag, nullptr);"]
    assert unseen("{ wait_bounded<true>(b, p, f, nullptr); }") and not unseen("x = wait(f, nullptr);")
    files = glob.glob(os.path.join(CSRC, "*.cu*"))
    assert len(files) > 10
    for name in files:
        with open(name) as f:
            assert unseen(f.read()) == [], os.path.basename(name)
