"""How the four warps of a row tile of the prefix kernel leave a run in which
waits give up: a model of the control flow of that role (attn_tc.cu, warps 4..7
and 8..11), walked over every combination of waits that succeed and give up.

Each warp decides by its own waits: one gives up, and the next finds the phase
complete a moment later.  The row tile's barriers count all four warps, so no
combination may leave some of them at one while the others are at the kernel's
end."""
import itertools

import pytest

WARPS, TILES = 4, 1


def warp_role(runs, waits, vote, has_rows):
    """Yields ("tile", ok) at a barrier of the row tile, with what the vote gets,
    and receives the vote's result; ("end", None) at the end of the kernel.
    waits(): the outcome of this warp's next wait."""
    ok = True
    for _ in range(runs):
        if not ok:
            break
        if not has_rows:                       # an empty row tile waits for the run's end
            ok = waits()
            if vote:
                ok = yield ("tile", ok)
            continue
        yield ("tile", True)                   # the rows' numbers are written
        for _ in range(TILES):
            ok = waits()                       # scores
            if not ok:
                break
        ok = ok and waits()                    # the run's sums
        if vote:
            ok = yield ("tile", ok)
        if not ok:
            break
        for _ in range(4):                     # two halves of the sums through shared memory
            yield ("tile", True)
    yield ("end", None)


def stuck(outcomes, runs, vote, has_rows):
    """Whether four such warps, with these outcomes of their waits, stay at a barrier for ever."""
    warps = [warp_role(runs, iter(o).__next__, vote, has_rows) for o in outcomes]
    at = [next(w) for w in warps]
    while True:
        names = {name for name, _ in at}
        if names == {"end"}:
            return False
        if "end" in names:
            return True                        # the others' barrier never has its 128 threads
        ok = all(v for _, v in at)
        at = [w.send(ok) for w in warps]


@pytest.mark.parametrize("has_rows,without", [(True, True), (False, False)])
def test_no_combination_of_waits_that_give_up_leaves_a_warp_behind(has_rows, without):
    runs = 2
    n = runs * (TILES + 1) if has_rows else runs
    one = list(itertools.product([True, False], repeat=n))
    found = 0
    for outcomes in itertools.product(one, repeat=WARPS):
        assert not stuck(outcomes, runs, True, has_rows)
        if without and found == 0:
            found += stuck(outcomes, runs, False, has_rows)
    if without:
        assert found                           # without the vote the model does get stuck
