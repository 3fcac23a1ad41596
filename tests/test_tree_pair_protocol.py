"""The pair kernel's synchronisation across its two CTAs (mla_decode_tree_sm103a.cu), on the CPU.

Two CTAs share barriers, operands in shared memory and accumulators.  An mbarrier operation
without a scope orders the threads of one CTA alone, so every arrival on the other CTA's barrier
has to release, and every wait on a barrier that the pair arrives on to acquire, at cluster scope.
And a wait names a phase by its parity, so a barrier may not run two phases ahead of a waiter.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_attention_paged_gb300", "csrc")


@pytest.fixture(scope="module")
def source():
    with open(os.path.join(CSRC, "mla_decode_tree_sm103a.cu")) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", text)


def _function(text, name):
    """The body of a device function of that name."""
    at = re.search(r"\b" + name + r"\([^;{]*\)\s*\{", text)
    assert at, name
    depth, i = 1, at.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at.end():i]


def test_arrivals_at_the_other_cta_release_at_cluster_scope(source):
    arrivals = re.findall(r"(?:fence[.\w:]*;\\n\\t\"\s*\")?mbarrier\.arrive[.\w:]*", source)
    assert arrivals
    for a in arrivals:
        if "shared::cluster" not in a:
            continue
        released = "mbarrier.arrive.release.cluster." in a
        fenced = "mbarrier.arrive.relaxed.cluster." in a and re.match(r"fence\.(release|acq_rel)[.\w:]*\.cluster;", a)
        assert released or fenced, a


def test_waits_of_the_pair_acquire_at_cluster_scope(source):
    waits = re.findall(r"mbarrier\.(?:try|test)_wait[.\w:]*", source)
    assert waits and all(".acquire.cluster." in w for w in waits), waits
    # and the kernel's roles use no other wait (drain_wait only ends a CTA that gave up)
    kernel = _function(source, "decode_tree_pair_kernel")
    assert "mbar_wait(" not in kernel and "mbar_try_wait(" not in kernel and "mbar_arrive(" not in kernel


class Barrier:
    """An mbarrier of one arrival, waited for by parity."""

    def __init__(self):
        self.phase = 0

    def arrive(self):
        self.phase += 1

    def passed(self, parity):
        return (self.phase & 1) != parity


def _runs_dry(barrier_of, parity_of, tiles=2):
    """Whether some order of BMM1's arrivals and the softmax's waits leaves the softmax waiting.

    BMM1 reaches tile j (s_full j, v_here j) once the softmax has read the scores of tile j - 2; the
    softmax waits for v_here j after it has read the scores of tile j."""
    seen, todo = set(), [(0, 0, 0)]  # tiles that BMM1 has issued, scores read, V waits passed
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        issued, read, waited = state
        bars = [Barrier(), Barrier()]
        for j in range(issued):
            bars[barrier_of(j)].arrive()
        moves = []
        if issued < tiles and read >= issued - 1:
            moves.append((issued + 1, read, waited))
        if read < issued and read == waited:
            moves.append((issued, read + 1, waited))
        if waited < read and bars[barrier_of(waited)].passed(parity_of(waited)):
            moves.append((issued, read, waited + 1))
        if not moves and waited < tiles:
            return True
        todo += moves
    return False


def test_the_value_tiles_barriers_are_never_two_phases_ahead():
    assert not _runs_dry(lambda j: j, lambda j: 0)         # one barrier a tile, as in the kernel
    assert _runs_dry(lambda j: 0, lambda j: j & 1)         # one for both would miss the first tile's phase


def test_drafts_lie_in_at_most_two_tiles_of_a_cta():
    for T in range(1, 65):
        for p0 in range(0, 200, 3):
            L = p0 + T
            for chunk in (64, 128, 320):
                for start in range(0, L, chunk):
                    end = min(L, start + chunk)
                    ntiles = -(-(end - start) // 64)
                    tail = max(0, p0 - start) // 64
                    assert ntiles - tail <= 2


def test_the_kernel_has_a_barrier_for_each_tile_that_holds_drafts(source):
    assert re.search(r"uint64_t v_here\[2\];", source)
    assert len(re.findall(r"v_here\[j - tail_tile\]", source)) == 2
