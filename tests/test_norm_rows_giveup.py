"""The norm backward's ring, read as text: a wait for rows that gives up ends the
group's loop.  (Going on would fetch rows with a second arrival on a barrier whose
phase is still open.)  The group's results are not numbers then, and the copies in
flight are waited for before the CTA ends."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bitlinear_bl_forward_b200", "csrc")


def kernel():
    with open(os.path.join(CSRC, "bl_norm_grad.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    text = text[text.index("bl_norm_bwd_kernel("):]
    return re.sub(r"\s+", " ", text[:text.index("bl_norm_dx_wide_kernel(")])


def test_no_rows_are_fetched_after_a_wait_that_gave_up():
    text = kernel()
    loop = text[text.index("m0 < a.M; m0 += step, ++it"):]
    assert "ok = mbar_wait(&full[grp][st], ph, nullptr, limit_ns, kSiteNormRows);" in loop
    # the group decides as one, at its barrier, before any stage is filled again
    leave = loop.index("ok = named_bar_and(1 + grp, T, ok); if (!ok) break;")
    assert re.search(r"if \(a\.dX\) ok = group_sum<NS>\([^;]*, ok\); else $", loop[:leave])
    assert loop.index("mbar_wait(") < leave < loop.index("fetch(")


def test_copies_in_flight_are_waited_for_after_giving_up():
    text = kernel()
    after = text[text.index("if (!ok) {"):]
    assert "dw[e] = db[e] = f2_both(__int_as_float(0x7FFFFFFF))" in after
    assert re.search(r"if \(tid == 0\) for \(int i = it, m = m0; i < \(it \? it \+ ST - 1 : ST\) && m < a\.M; "
                     r"\+\+i, m \+= step\) "
                     r"mbar_wait\(&full\[grp\]\[i % ST\], \(i / ST\) & 1, nullptr, limit_ns, kSiteDrain\)", after)
    assert after.index("mbar_wait(") < after.index("pdl_launch_dependents()")


def test_the_steps_in_flight():
    # a model of the ring: which steps have been fetched, and not waited for with
    # success, when the wait of step `it` gives up
    for st in (4, 6):
        for steps in range(1, 20):
            fetched = list(range(min(st, steps)))
            for it in range(steps):
                # the range that is drained, in the kernel's words
                drained = [i for i in range(it, it + st - 1 if it else st) if i < steps]
                assert drained == [i for i in fetched if i >= it]
                if it > 0 and it + st - 1 < steps:
                    fetched.append(it + st - 1)
