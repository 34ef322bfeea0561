"""CPU: the ring of linear_int8, whose stages two groups of warps take in turn. A wait on an
mbarrier names a phase by its parity, which tells it from the phase before only: a group that
waits for use k of a place has to find k or k + 1 uses of it landed. Copies land in any order,
so what orders them is what each group has waited for before."""
import pytest

from test_launch_rules import code


def landed_before(stage, stages):
    """The stages that have surely landed when the group of `stage` waits for it: its own earlier
    ones, and all that the MMAs before its last free copy have read (two copies, MMAs in order)."""
    own = set(range(stage % 2, stage, 2))
    # to convert stage - 2 it waited for the MMA of stage - 4, which came after all MMAs before
    return own | set(range(max(0, stage - 3)))


def released_before(stage, stages):
    """With an odd ring the group also waits until the place's use before has been released, which
    names one phase: the release before that was its own."""
    return {stage - stages} if stages % 2 else set()


@pytest.mark.parametrize("stages", [2, 3, 4, 5, 6])
def test_a_wait_names_one_phase_only(stages):
    for stage in range(stages, 200):
        assert stage - stages in landed_before(stage, stages) | released_before(stage, stages)
        if stages % 2 and stage >= 2 * stages:  # the release of use k - 2 was this group's own
            assert stage - 2 * stages in range(stage % 2, stage, 2)


def test_three_stages_need_the_second_wait():
    assert any(s - 3 not in landed_before(s, 3) for s in range(3, 200))


def test_the_kernel_has_it():
    text = code("ops_eight.cuh")
    first = text.index("(NST & 1) != 0 && st >= st0 + NST")
    wait = text[first:text.index("{", first)]
    assert "mbar_wait(empty_bar(stage), phase ^ 1u" in wait
    assert first < text.index("mbar_wait(full_bar(stage), phase, p.wait)", first)
