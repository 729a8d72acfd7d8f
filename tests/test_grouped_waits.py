"""Give-up paths of the grouped and int8 product (its source; no GPU is made to wait).

Two epilogue warps meet at barriers that count both, so they have to leave the tile loop together.  A thread that reads
the abort flag on its own may see it set where its neighbour a moment earlier did not, and the neighbour would wait at
the next such barrier for good.  The flag is therefore read inside the bounded waits alone, whose outcome the two warps
vote on."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_delayed_scaling_03_b200", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def test_no_thread_reads_the_abort_flag_outside_a_bounded_wait():
    uses = re.findall(r"\*abort_flag\b[^;]*;", source("grouped.cu"))
    assert uses == ["*abort_flag = 0;"], uses


def test_the_two_warps_vote_on_every_wait_between_their_barriers():
    text = source("grouped.cu")
    loop = text[text.index("auto hand_back"):]
    waits = re.findall(r"[^\n]*\bmbar_await\(|[^\n]*\bduo_await\(", loop)
    assert waits and all("duo_await(" in w for w in waits), waits
    assert "break" not in loop[loop.index("for (int st = half"):loop.index("if (++acc == 2)")]


def test_a_block_that_gave_up_outlives_its_copies():
    """Bulk loads (and partial sums of a cluster) that are under way when a wait gives up land in shared memory that the
    block still owns: after its last barrier it waits a bounded time for them.  Nothing else follows that barrier but
    the release of tensor memory."""
    text = source("grouped.cu")
    end = text[text.rindex("else cta_sync();"):text.index("cudaError_t launch_build")]
    assert "settle_copies(abort_flag)" in end
    helper = source("device.cuh")
    body = helper[helper.index("void settle_copies("):]
    body = body[:body.index("\n}")]
    assert "globaltimer_ns()" in body and "kSettleNs" in body, body
