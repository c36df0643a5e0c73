"""How a pair of CTAs ends (diff_fwd_wide.cu).  What one CTA's tensor core or scheduler request sends to the
other's barriers (commits to both, the answer to a request for a unit) arrives by itself, ordered by no cluster
barrier, so the receiver waits for it before it leaves.  Read from the source: the window is too short for a run
to show."""
import os
import re

from exact_attention_55_gb300 import build


def code_of(name):
    with open(os.path.join(build.CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernel():
    body = code_of("diff_fwd_wide.cu")
    return body[body.index("diff_out_kernel(const __grid_constant__"):body.index("static cudaError_t launch_one")]


def block(code, start):
    """The braces that open behind `start`, with what they hold."""
    i = code.index("{", start)
    depth = 0
    for j in range(i, len(code)):
        depth += {"{": 1, "}": -1}.get(code[j], 0)
        if depth == 0:
            return code[i:j + 1]
    raise AssertionError("unbalanced braces")


def test_both_ctas_wait_for_the_last_commit():
    code = kernel()
    assert "pair_commit_warp(&bars->drain)" in code
    waits = [m.start() for m in re.finditer(r"mbar_wait\(smem_u32\(&bars->drain\)", code)]
    assert waits
    for m in re.finditer(r"if \(rank == 0\)", code):     # no such wait is one CTA's alone
        rest = code[m.end():].lstrip()
        own = block(code, m.end()) if rest.startswith("{") else rest[:rest.index(";") + 1]
        assert "mbar_wait(smem_u32(&bars->drain)" not in own


def test_what_is_committed_to_both_is_waited_for():
    """Each barrier that commits reach in both CTAs has a wait for its last phase behind the walk over the units
    (s_full and o_full have it within)."""
    code = kernel()
    both = set(re.findall(r"pair_commit_warp\(&bars->(\w+)", code))
    assert both == {"kv_empty", "s_full", "q_empty", "w_free", "o_full", "drain"}
    ends = code[code.index("units.give(w, ok)"):code.index("units.finish(ok);")]
    for bar, last in (("kv_empty[k % C::NSLOT]", "(k / C::NSLOT) & 1"), ("q_empty", "(uc - 1) & 1")):
        assert f"mbar_wait(smem_u32(&bars->{bar}), {last}, " in ends, bar
    compute = code[code.index("uint8_t* w_row"):]
    tail = compute[compute.index("pair_arrive(&bars->o_empty)"):]
    assert "&bars->w_free" in tail


def test_the_second_cta_waits_for_an_answer_after_an_abort():
    """CTA 0 may send a request, whose answer lands in both, after CTA 1 gave up: CTA 1 looks again once CTA 0
    sends nothing more, behind a barrier of both."""
    code = kernel()
    end = code[code.rindex("__syncthreads();"):]
    assert "hand.last_answer()" in end[end.index("pair_sync()"):]
    units = code_of("diff_units.cuh")
    assert "hand->owed = " in block(units, units.index("void finish(bool ok)"))
    assert "mbar_wait(smem_u32(&steal)" in block(units, units.index("void last_answer()"))
