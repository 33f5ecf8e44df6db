"""What the shapes of the GPU tests reach: every kernel of the gradients, with tiles
written whole and with sums in parts.  The cost model chooses; a constant that is
retuned so that a kernel or a cut is no longer tested fails here."""

import collections

import pytest

from bitlinear_bl_forward_b200 import bl
from bitlinear_bl_forward_b200 import build as blbuild
from tests.test_gpu_grad import REACH_INPUT, REACH_REST, REACH_WEIGHT, SHAPES

SHAPE, UNSUP = 2, 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    blbuild.build()


def cut(plan):
    bn, tiles, whole, stages, per, parts = plan
    assert bn in (32, 64, 128, 192, 256) and 0 <= whole <= tiles and per >= 1 and parts >= 1
    if whole == tiles:
        assert parts == 1
        return "whole"
    if whole:
        return "behind waves"   # whole waves of whole tiles, the other tiles' stages dealt out
    # every tile in the same number of parts, or all stages dealt out
    return "equal" if parts == -(-stages // per) else "dealt out"


def reached(weight, flags, shapes):
    got = collections.defaultdict(set)
    for s in shapes:
        plan = bl.bl_gradient_plan(weight, *s, flags)
        got[plan[0]].add(cut(plan))
    return got


ALL = {"whole", "equal", "dealt out", "behind waves"}


def test_input_gradient_shapes_reach_every_kernel():
    got = reached(False, 0, SHAPES + REACH_INPUT + REACH_REST)
    assert set(got) == {32, 64, 128, 192, 256}
    assert all({"whole", "equal"} <= cuts for cuts in got.values())
    assert {"dealt out"} <= got[32] & got[128] and {"behind waves"} <= got[192] & got[256]
    assert set.union(*got.values()) == ALL


@pytest.mark.parametrize("flags", [0, 2])
def test_weight_gradient_shapes_reach_every_kernel(flags):
    got = reached(True, flags, SHAPES + REACH_WEIGHT + REACH_REST)
    assert set(got) == {128, 192, 256}
    assert all({"whole", "equal", "dealt out"} <= cuts for cuts in got.values())
    assert {"behind waves"} <= got[192] & got[256]


def test_the_weight_gradients_plan_does_not_depend_on_accumulating():
    for s in REACH_WEIGHT:
        assert bl.bl_gradient_plan(True, *s, 0) == bl.bl_gradient_plan(True, *s, 1)
        assert bl.bl_gradient_plan(True, *s, 2) == bl.bl_gradient_plan(True, *s, 3)


@pytest.mark.parametrize("args,status", [((False, 0, 64, 8), SHAPE), ((False, 4, 60, 8), SHAPE),
                                         ((True, 4, 64, 0), SHAPE), ((False, 4, 64, 8, 2), UNSUP),
                                         ((True, 4, 64, 8, 4), UNSUP)])
def test_refusals(args, status):
    with pytest.raises(bl.BLError) as e:
        bl.bl_gradient_plan(*args)
    assert e.value.status == status
    assert bl.lib().bl_gradient_plan(2, 4, 64, 8, 0, None) == UNSUP
    assert bl.lib().bl_gradient_plan(0, 4, 64, 8, 0, None) == 1
