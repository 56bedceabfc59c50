"""Barriers that two CTAs of a cluster share, read from the source: a missing scope is no failure that a run would
show reliably.  An arrival on another CTA's barrier is released to the cluster, and the waits of kernels that run as
pairs acquire from it: without both, what the other CTA wrote before its arrival is not ordered before what the waiting
thread does next."""
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "weight_transfer_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_remote_arrivals_are_released_to_the_cluster():
    seen = 0
    for name in os.listdir(CSRC):
        text = source(name)
        for m in re.finditer(r"mbarrier\.arrive[\w.:]*", text):
            if "shared::cluster" in m.group():
                seen += 1
                before = text[:m.start()].rsplit("asm volatile(", 1)[1]
                assert ".release.cluster" in m.group() or (
                    ".relaxed.cluster" in m.group() and "fence.release.sync_restrict::shared::cta.cluster;" in before), name
    assert seen == 1


def test_waits_for_the_other_cta_acquire_from_the_cluster():
    """The first CTA's issuing thread waits for arrivals of the other one's threads: stages full, accumulators read."""
    device, product = source("fp8q_device.cuh"), source("moe_product.cu")
    assert "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64" in device
    issue = product[product.index("const uint32_t st0 = operand_desc"):product.index("} else if (warp == 2) {")]
    waits = re.findall(r"mp_wait(<PAIR>)?\(&(\w+)", issue)
    assert waits == [("<PAIR>", "acc_empty"), ("<PAIR>", "full")]
