"""The place of the second query tile, which the e4m3 prefill lends to its ring while units have one
tile: a model of the barriers that guard it, through every order of events (no GPU needed).

The walk gives out items through two slots and loads each unit's queries, the second tile's over the
lent place.  The copy warps, a team for the keys and one for the values, read a single tile's unit's
rows there.  The products let a unit's queries go when its keys' products are done, and hold its item
until the values' are.  A barrier is what the hardware's is: a phase ends with the count of its
arrivals, whoever they come from, and a wait tells phases by their parity.
"""
import os

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(os.path.dirname(HERE), "attention_backward_flashattention_gb300", "csrc",
                      "attn_prefill.cuh")
WARPS = (0, 0, 1, 1)  # the copy warps' teams (two of each are enough for one to be ahead)


def passes(arrivals, count, phase):
    """Whether a wait for the end of `phase` passes, by its parity."""
    return ((arrivals // count) ^ phase) & 1 == 1


def explore(twins, release_last):
    """(place overwritten while a warp may still read it, some order of events gets stuck).

    twins: for each unit whether it has a single tile.  release_last: the copy warps let go of an
    item behind the lent place, not at the start of its unit."""
    N = len(twins)
    before = [sum(twins[:n]) for n in range(N + 1)]
    # what each actor does, in order
    walk = [(what, n) for n in range(N) for what in ("give", "load")]
    copy = [(what, n) for n in range(N) for what in
            (("take", "read", "free") if release_last else ("take+let go", "read", "free"))]
    products = [(what, n) for n in range(N) for what in ("keys", "values")]
    programs = (walk,) + (copy,) * len(WARPS) + (products,)

    def counts(state):
        """Items given, queries loaded, arrivals, and units read, from the actors' places."""
        at = [p[:i] for p, i in zip(programs, state)]
        given = sum(w == "give" for w, _ in at[0])
        loaded = sum(w == "load" for w, _ in at[0])
        let_go = [0, 0]
        free = [0, 0]
        read = []
        for team, done in zip(WARPS, at[1:-1]):
            read.append(sum(w == "read" for w, _ in done))
            for w, n in done:
                if w == ("free" if release_last else "take+let go"):
                    let_go[n & 1] += 1
                if w == "free" and twins[n]:
                    free[team] += 1
        keys = sum(w == "keys" for w, _ in at[-1])
        for w, n in at[-1]:
            if w == "values":
                let_go[n & 1] += 1
        return given, loaded, let_go, free, read, keys

    each = len(WARPS) // 2
    bad = stuck = False
    start = (0,) * len(programs)
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        given, loaded, let_go, free, read, keys = counts(state)
        moves = []
        for a, i in enumerate(state):
            if i == len(programs[a]):
                continue
            what, n = programs[a][i]
            if what == "give":
                go = n < 2 or passes(let_go[n & 1], len(WARPS) + 1, n // 2 - 1)
            elif what == "load":
                go = keys >= n  # (q_empty of the unit in front)
                if go and not twins[n] and before[n] > 0:
                    go = all(passes(f, each, before[n] - 1) for f in free)
                    if go and any(r <= m for r in read for m in range(n) if twins[m]):
                        bad = True
            elif what in ("take", "take+let go"):
                go = given > n
            elif what == "keys":
                go = loaded > n and all(r > n for r, t in zip(read, WARPS) if t == 0)
            elif what == "values":
                go = all(r > n for r, t in zip(read, WARPS) if t == 1)
            else:  # (a unit's rows may be read before its queries are there)
                go = True
            if go:
                moves.append(a)
        if not moves and any(i < len(p) for i, p in zip(state, programs)):
            stuck = True
        for a in moves:
            nxt = state[:a] + (state[a] + 1,) + state[a + 1:]
            if nxt not in seen:
                seen.add(nxt)
                todo.append(nxt)
    return bad, stuck


UNITS = [(1, 0), (1, 1, 0), (1, 1, 1, 0), (1, 0, 1, 0), (0, 1, 1, 0), (1, 1, 0, 0, 1), (1, 0, 0, 1, 0)]


@pytest.mark.parametrize("twins", UNITS)
def test_place_is_read_before_it_is_overwritten(twins):
    assert explore(twins, release_last=True) == (False, False)


def test_the_model_sees_an_item_let_go_of_early():
    assert explore((1, 0), release_last=False) == (False, False)
    assert explore((1, 1, 0), release_last=False)[0]


def test_the_copy_warps_let_go_in_the_model_s_order():
    """The model's order is the source's: with the lent place, a copy warp's only arrival on an item's
    slot comes right behind its arrival for the place."""
    text = open(SOURCE).read()
    copy = text[text.index("---- keys and values"):text.index("---- softmax")]
    let_go = "mbar_arrive(smem_u32(&bars->item_empty[n & 1]));"
    assert copy.count(let_go) == 2
    early, late = copy.index(let_go), copy.rindex(let_go)
    assert "if constexpr (!C::kSpareQ) {" in copy[early - 120:early]
    assert "mbar_arrive(smem_u32(&bars->spare_free[team]));" in copy[late - 90:late]
