"""The kernels that run as pairs of CTAs, read as text: a barrier that the other
CTA's threads or commits arrive on is waited for with acquire at cluster scope,
and remote arrivals name their scope (the unqualified forms are of CTA scope, and
order nothing between two CTAs)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bitlinear_bl_forward_b200", "csrc")

# barriers that the other CTA's threads or commits arrive on
PAIR = {
    "bl_gemm_2sm.cuh": {"done", "afull", "accfull", "accempty"},
    "bl_grad_tc.cuh": {"done", "ready", "accfull", "accempty"},
}


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", sorted(PAIR))
def test_waits_on_the_pairs_barriers_acquire_at_cluster_scope(name):
    waits = re.findall(r"\b(mbar_\w*wait\w*)\(&(\w+)\[", source(name))
    assert PAIR[name] <= {bar for _, bar in waits}
    for call, bar in waits:
        if bar in PAIR[name]:
            assert call.endswith("_cluster"), f"{name}: {call} on {bar}"


@pytest.mark.parametrize("name", ["bl_common.cuh", "bl_gemm_2sm.cuh", "bl_grad_tc.cuh", "bl_tc_common.cuh"])
def test_cluster_forms_name_their_scope(name):
    text = source(name)
    # "mbarrier.arrive....shared::cluster" is an arrival on another CTA's barrier
    for op in re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", text):
        assert re.search(r"\.(release|relaxed)\.cluster\.", op), op
    # a wrapper called ..._cluster waits with acquire at cluster scope
    for body in re.findall(r"bool mbar_(?:try|test)_wait_cluster\(.*?\n}", text, flags=re.S):
        assert re.search(r"mbarrier\.(?:try|test)_wait\.parity\.acquire\.cluster\.", body), body


def test_expanded_tiles_are_fenced_before_their_arrival():
    # a relaxed arrival on ready orders nothing by itself: every lane's proxy fence
    # and the warp's meeting come directly before it
    text = source("bl_grad_tc.cuh")
    at = [m.start() for m in re.finditer(r"mbar_arrive_cluster_relaxed\(&ready\[", text)]
    assert len(at) == 1
    before = re.sub(r"\s+", " ", text[:at[0]])
    assert before.endswith("fence_proxy_async_smem(); __syncwarp(); if (lane == 0) ")
