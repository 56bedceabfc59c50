"""How a warp gives a stage of a ring back, read from the source: a run would not show reliably that it does so too
early.  One lane arrives for the whole warp; the other lanes' reads of the stage, and of what the copying warp wrote
about it, have to be behind them, which only a warp barrier in front of the arrival says.  It also orders that lane's
own stores, so the arrival itself has to be one that the compiler moves no access across."""
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "weight_transfer_gb300", "csrc")


def test_a_warp_meets_before_one_lane_gives_its_stage_back():
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for m in re.finditer(r'asm volatile\("mbarrier\.arrive\.shared::cta\.b64 _, \[%0\];"[^;]*&empty\[[^;]*;', text):
            seen += 1
            assert '"memory"' in m.group(), name
            before = text[:m.start()]
            turn = before[before.rindex("mbar_wait(&full["):]         # since this stage was waited for
            lane0 = turn.rindex("if (lane == 0)")
            assert re.search(r"__syncwarp\(\);\s*(//[^\n]*\s*)?$", turn[:lane0]), name
    assert seen == 2
