"""CPU model of the hand-over between streaming and finishing warps in the persistent kernel of the
vocabulary rows (row_wise_arg_gb300/csrc/logits_stream.cuh): every order in which the warps can run.

Row i uses buffer i mod (F + 1) and finisher i mod F. A named barrier releases everyone when its
number of warps has arrived, whoever they are: two finishers that meet on one are as good to it as a
finisher and a streamer. Successive rows of a buffer belong to different finishers, so a finisher may wait for
its row only once the finisher of the row before has met the streamers there: a turn that goes round
the finishers, a barrier for each pair of neighbours. (A turn per buffer is not enough: its barrier
has changing pairs too.)"""
import pytest


def explore(finishers, rows, streamers, turn):
    """Faults that some order leads to: 'wrong row', 'early buffer' or 'stuck'."""
    buffers = finishers + 1
    full, free, turns = 0, buffers, 2 * buffers  # barriers: full and free + buffer, turns + who waits
    size = [streamers + 1] * (2 * buffers) + [2] * buffers

    def streamer(w):
        for i in range(rows):
            yield ("sync", free + i % buffers)
            yield ("write", i % buffers, w, i)
            yield ("arrive", full + i % buffers)

    def finisher(f):
        for at in range(f, buffers, finishers):
            if at < rows:
                yield ("arrive", free + at)
        for i in range(f, rows, finishers):
            at = i % buffers
            if turn == "per buffer" and finishers > 1 and i >= buffers:
                yield ("sync", turns + at)
            if turn == "round" and finishers > 1 and i > 0:
                yield ("sync", turns + f)
            yield ("sync", full + at)
            if turn == "per buffer" and finishers > 1 and i + buffers < rows:
                yield ("arrive", turns + at)
            if turn == "round" and finishers > 1 and i + 1 < rows:
                yield ("arrive", turns + (f + 1) % finishers)
            yield ("take", at, i)
            if i + buffers < rows:
                yield ("arrive", free + at)

    programs = [list(streamer(w)) for w in range(streamers)] + [list(finisher(f)) for f in range(finishers)]
    # a state: each warp's place, whether it waits, arrivals per barrier, the rows in the buffers, rows taken
    start = (tuple(0 for _ in programs), tuple(False for _ in programs), (0,) * len(size),
             (-1,) * (buffers * streamers), (True,) * buffers)
    seen, todo, faults = {start}, [start], set()
    while todo:
        place, waits, count, held, taken = todo.pop()
        moved = False
        for w, program in enumerate(programs):
            if waits[w] or place[w] == len(program):
                continue
            moved = True
            what, *arg = program[place[w]]
            p, q, c, h, t = list(place), list(waits), list(count), list(held), list(taken)
            p[w] += 1
            if what in ("sync", "arrive"):
                b = arg[0]
                c[b] += 1
                q[w] = what == "sync"
                if c[b] == size[b]:  # release everyone who waits here
                    c[b] = 0
                    for v in range(len(programs)):
                        if q[v] and programs[v][p[v] - 1] == ("sync", b):
                            q[v] = False
            elif what == "write":
                at, s, i = arg
                if s == 0 and not t[at]:
                    faults.add("early buffer")
                h[at * streamers + s] = i
                if s == 0:
                    t[at] = False
            else:
                at, i = arg
                if any(h[at * streamers + s] != i for s in range(streamers)):
                    faults.add("wrong row")
                    continue
                t[at] = True
            state = (tuple(p), tuple(q), tuple(c), tuple(h), tuple(t))
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if not moved and any(waits[w] or place[w] < len(programs[w]) for w in range(len(programs))):
            faults.add("stuck")
    return faults


@pytest.mark.parametrize("finishers,rows,streamers", [(1, 8, 1), (1, 5, 3), (2, 13, 1), (2, 9, 2),
                                                      (3, 17, 1), (3, 12, 2)])
def test_every_order_hands_over_the_right_rows(finishers, rows, streamers):
    for n in range(rows + 1):
        assert explore(finishers, n, streamers, "round") == set(), n


@pytest.mark.parametrize("finishers", [2, 3])
def test_why_the_turns(finishers):
    """Without them, or with one per buffer, a late finisher's row is taken by another."""
    assert "wrong row" in explore(finishers, 3 * finishers, 1, "none")
    assert "wrong row" in explore(finishers, 5 * finishers, 1, "per buffer")
