"""The order in which eviction's moves read, announce and write, played on the
host under random interleavings: destination tables that mix a sequence's own
pages with others (units on other pages announce their read late, with their
stores), and units whose read never completes."""
import random

import pytest

PAGE = 16  # blocks


def play(rng, unit, keep, nb, tail, own, fails, announces_failed_reads=False):
    """Units of `unit` destination blocks over a sequence of nb complete blocks (and an open one); own[P]: page P of
    the destination is the sequence's own.  A unit in `fails` never gets its blocks.  Returns (the own pages' slots,
    what each unit read, the units that wrote)."""
    moved = keep + ([nb] if tail else [])
    slots = list(range(nb + 1))
    slots += [-1] * (-len(slots) % PAGE)
    units = -(-len(moved) // unit)
    rank = [sum(1 for b in keep if b < unit * u) for u in range(nb // unit + 3)]
    span = [range(unit * u, min(unit * u + unit, len(moved))) for u in range(units)]
    moves = [any(not own[k // PAGE] or moved[k] != k for k in sp) for sp in span]
    reads, announced, ended, state, claimed, resident = {}, set(), set(), {}, 0, rng.randint(1, 6)
    while True:
        steps = []
        if claimed < units and sum(1 for u in range(claimed) if u not in ended) < resident:
            steps.append(("claim", claimed))
        for u in (u for u in range(claimed) if u not in ended):
            if state[u] == "claimed":
                steps.append(("read", u))
            elif state[u] == "read":
                here = own[u * unit // PAGE]
                k0, k1 = rank[u], rank[u + 1]
                waits = range(k0 // unit, min(u - 1, (k1 - 1) // unit) + 1) if here and k1 > k0 and moves[u] else []
                assert all(w < u for w in waits)
                if all(w in announced for w in waits):
                    steps.append(("write", u))
        if not steps:      # what is left waits for a read that failed: its bounded wait runs out
            return slots, reads, {u for u in ended if u not in fails}
        what, u = rng.choice(steps)
        if what == "claim":
            state[u], claimed = "claimed", claimed + 1
        elif what == "read":
            if u in fails and moves[u]:
                ended.add(u)
                if announces_failed_reads:
                    announced.add(u)
                continue
            reads[u] = [slots[moved[k]] for k in span[u]]
            state[u] = "read"
            if own[u * unit // PAGE] or not moves[u]:
                announced.add(u)
        else:
            if own[u * unit // PAGE]:
                for k, x in zip(span[u], reads[u]):
                    slots[k] = x
            announced.add(u)
            ended.add(u)


def scene(rng):
    nb = rng.randint(1, 300)
    part = rng.random()
    keep = [b for b in range(nb) if rng.random() < part] if rng.random() < 0.8 else list(range(nb))
    pages = nb // PAGE + 1
    own = rng.choice([[True] * pages, [False] * pages, [P % 2 == 0 for P in range(pages)],
                      [P >= pages // 2 for P in range(pages)], [P < pages // 2 for P in range(pages)],
                      [rng.random() < 0.5 for _ in range(pages)]])
    return nb, keep, rng.random() < 0.5, own


@pytest.mark.parametrize("unit", [4, 8])
@pytest.mark.parametrize("seed", range(60))
def test_mixed_tables_move_every_block(seed, unit):
    rng = random.Random(seed)
    nb, keep, tail, own = scene(rng)
    moved = keep + ([nb] if tail else [])
    slots, reads, wrote = play(rng, unit, keep, nb, tail, own, set())
    assert len(wrote) == -(-len(moved) // unit)
    for u in wrote:
        assert reads[u] == moved[unit * u:unit * u + unit]
    for k, b in enumerate(moved):
        if own[k // PAGE]:
            assert slots[k] == b


def lost_blocks(rng, unit, announces):
    """Kept blocks that a unit whose read failed should have moved, and that are gone from their old place."""
    nb, keep, tail, own = scene(rng)
    moved = keep + ([nb] if tail else [])
    units = -(-len(moved) // unit)
    fails = {rng.randrange(units)} if units else set()
    slots, reads, wrote = play(rng, unit, keep, nb, tail, own, fails, announces)
    for u in wrote:
        assert reads[u] == moved[unit * u:unit * u + unit]
    return [b for u in fails if u not in wrote for b in moved[unit * u:unit * u + unit]
            if slots[b] != b and not any(b in reads[w] for w in wrote)]


@pytest.mark.parametrize("unit", [4, 8])
def test_a_read_that_never_completes_costs_no_block_its_old_place(unit):
    for seed in range(400):
        assert lost_blocks(random.Random(seed), unit, False) == []
    # the model sees the mistake it is there for: announcing such a read lets others overwrite its blocks
    assert any(lost_blocks(random.Random(seed), unit, True) for seed in range(400))
