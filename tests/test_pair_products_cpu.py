"""What the e4m3 product's kernel waits for before it leaves or uses warp-wide instructions, read from its
source: a wait that is missing shows on a GPU by chance at most."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "folded_tensor_sequence_tsp_gb300", "csrc", "matmul_e4m3.cu")


@pytest.fixture(scope="module")
def text():
    with open(SOURCE) as fh:
        return re.sub(r"//[^\n]*", "", fh.read())


def part(text, first, last):
    a = text.index(first)
    return text[a:text.index(last, a)]


def test_the_second_cta_stays_for_the_first_ones_commits(text):
    """Every barrier that a commit of the pair's MMA warp arrives at is waited for in the second CTA too."""
    issuer = part(text, "if (warp == 1 && (!PAIR || rank == 0))", "if (warp >= 2)")
    barriers = set(re.findall(r"mma_commit_pair\((?:&)?(\w+)", issuer))
    assert barriers == {"acc_full", "empty", "drain"}
    producer = part(text, "if (warp == 0 && lane == 0)", "if (warp == 1 && (!PAIR || rank == 0))")
    leaving = producer[producer.index("WaitBound wd"):]
    # by the producer, whether a wait gave up before or not; the sums, in both CTAs, wait for every product
    assert re.search(r"if \(rank != 0\) mbar_wait\(drain, 0, wd", leaving)
    assert re.search(r"last_parity\[s\] >= 0\) ok = mbar_wait\(&empty\[s\], \(uint32_t\)last_parity\[s\], wb", leaving)
    sums = text[text.index("setmaxnreg.inc"):]
    assert re.search(r"mbar_wait_poll\(&acc_full\[acc\], acc_phase", sums)


def test_lanes_of_the_sums_stay_together_when_a_wait_gives_up(text):
    """A lane whose wait gave up must not leave the others in a tensor memory load of the whole warp: what it goes
    through does not depend on its own waits, and the warp meets between a wait and the loads."""
    sums = text[text.index("setmaxnreg.inc"):]
    loop = re.search(r"for \(int kb = kb0; ([^;]*); \+\+kb\) \{(.*?)tc_fence_after\(\);", sums, flags=re.S)
    assert loop.group(1) == "kb < kb1" and "break" not in loop.group(2)
    assert re.search(r"if \(!ready\) waited\(mbar_wait_poll\(&acc_full[^;]*;\s*__syncwarp\(\);\s*$", loop.group(2), flags=re.S)
    # a lane that gave up waits for nothing and arrives nowhere, and nothing else goes by it
    sums = sums[:sums.index("if constexpr (TURNED)")]
    assert re.search(r"if \(!done\) ok = arrives = false;", sums)
    assert len(re.findall(r"mbar_wait_\w+\(", sums)) == len(re.findall(r"waited\(mbar_wait_\w+\(", sums)) == 3
    conditions = set(re.findall(r"if \(([^()]*\b(?:ok|ready|arrives)\b[^()]*)\)", sums))
    assert conditions == {"!ready", "arrives", "ok && kb + 1 < kb1", "ok && kb0 < kb1"}
    assert re.findall(r"\bready = ([^;]*);", sums) == ["mbar_try_wait(&acc_full[acc], acc_phase) || !ok", "!ok"]
    assert not re.search(r"if \(lane == 0\)", sums)
