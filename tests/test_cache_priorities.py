"""Priorities in the second-level cache, read from the source: evict_last stays on a line until something else takes it
off, so that what it was given to would stand in the way of whatever runs after the call.  No call leaves any behind."""
import os

from conftest import ROOT

CSRC = os.path.join(ROOT, "weight_transfer_gb300", "csrc")


def test_no_priority_outlives_a_call():
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            for line in f:
                code = line.split("//")[0]
                assert "evict_last" not in code and "AccessPolicyWindow" not in code, (name, line)
