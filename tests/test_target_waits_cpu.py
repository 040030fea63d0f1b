"""The bounded waits of the target-side kernels, by reading their source: no test makes one run out on a GPU, so what a kernel
does then is held to rules that can be read."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "draft_head_gb300", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def part(text, start, end):
    assert text.count(start) == 1, start
    text = text[text.index(start) + len(start):]
    return text[:text.index(end)]


# A wait whose answer decides where the lane goes on.
DECIDES = re.compile(r"(!|=|&&|\breturn)\s*mbar_wait\(")


def test_whole_warps_leave_a_wait_with_one_answer():
    """Where whole warps wait and go on to a warp's or a block's barrier, a lane's own answer may differ from its
    neighbours' (one sees the phase, another its limit), and the warp would be split at the barrier: they go by the vote."""
    text = source("attention_tc.cu")
    assert DECIDES.search("if (!mbar_wait(") and DECIDES.search("ok = mbar_wait(")
    roles = {"mma": part(text, "} else if (warp == 1) {", "} else if (warp >= 2) {"),
             "queries and values": part(text, "} else if (warp >= 2) {", "setmaxnreg.inc"),
             "softmax": part(text, "setmaxnreg.inc", "tmem_dealloc(tmem, 512)")}
    for name, role in roles.items():
        assert "warp_wait(" in role and not DECIDES.search(role), name


def test_copies_land_before_attention_gives_up_its_memory():
    """Key, value and query boxes and products in flight are waited for on every way out, also by a role that is through while
    another has given up, and with a limit that is not the caller's."""
    text = source("attention_tc.cu")
    keys = part(text, "if (warp == 0 && lane == 0) {", "} else if (warp == 1) {")
    after = keys[keys.index("walk.next("):]
    assert "mbar_land(&full[" in after and "if (!ok)" not in after
    assert "mbar_land(drain" in part(text, "} else if (warp == 1) {", "} else if (warp >= 2) {")
    queries = part(text, "} else if (warp >= 2) {", "setmaxnreg.inc")
    assert "mbar_land(q_ready" in queries[queries.index("++item;"):]
    land = part(source("waits.cuh"), "void mbar_land(", "\n}")
    assert "timeout" not in land


def test_rows_on_their_way_land_before_the_ring_is_given_up():
    """The block leaves the loop when any of its threads gives up; the thread that waits for the copies then goes by the block's
    answer, not by its own, waits for the rows that were asked for and no others, and not with the caller's limit."""
    run = part(source("norm_rope.cu"), "norm_rope_run_kernel(const NormRopeArgs a", "template <typename T, int MODE>\ncudaError_t")
    assert re.search(r"\bok = __syncthreads_and\(mbar_wait\(", run)
    assert len(re.findall(r"\bok = ", run)) == 2  # its first value, and the block's answer
    land = run[run.index("if (!ok && threadIdx.x == 0)"):]
    assert "t + k < t_end" in land and "mbar_land(&full[st]" in land and "mbar_wait(" not in land
