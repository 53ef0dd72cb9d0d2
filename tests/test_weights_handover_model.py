"""The barriers of the tensor-core weights kernel, walked through every order of steps on the host.

Four groups of warps add the weights of a block's two token tiles (u) from the two score buffers (buf); an item's
query tiles alternate between the buffers, and at its end the group that had the first tile writes its sum and the
other one adds to it, told by one of four barriers used in turn (x_full).  Nothing tells the writer that the reader
has passed its wait, so the writer must never be four exchanges ahead: a barrier that completes a second time would
show the reader the parity of a phase that has not come.

A tile without tokens has no scores to wait for.  The model takes the rule for such tiles as a parameter: as the
kernel has it (no exchange), no order of steps overtakes a reader; with an exchange in them as well (the mistake that
this test guards against) one does, which shows that the model can see it.
"""
import pytest


class Model:
    """items: (query tiles, whether the block's second tile holds tokens).  Each actor is a list of steps, a step a
    wait (barrier, phase that must be complete) or None, and the barriers it arrives on.  The barriers' states follow
    from how far every actor has come."""

    def __init__(self, items, exchange_in_empty_tiles):
        self.count = {}
        actors = []
        self.reads = []           # (actor, step, barrier, phase): a reader's wait for an exchange
        mma, qc, used = [], 0, {}
        for nq, second in items:
            for k in range(nq):
                buf = qc & 1
                for u in range(1 + second):
                    n = used.get((u, buf), 0)
                    used[u, buf] = n + 1
                    mma.append((("s_empty", u, buf), n - 1, [("s_full", u, buf)]))
                qc += 1
        actors.append(mma)
        for h in range(2):        # the log-sum-exps of the even and the odd tiles
            n = (sum(nq for nq, _ in items) + 1 - h) // 2
            actors.append([(("i_empty", h), i - 1, [("i_full", h)]) for i in range(n)])
        for u in range(2):
            for buf in range(2):
                steps, qc, sn, xn = [], 0, 0, 0
                for nq, second in items:
                    active = u == 0 or second
                    skip = (buf - qc) & 1
                    for k in range(skip, nq, 2):
                        steps.append((("i_full", buf), (qc + k) >> 1, []))
                        if active:
                            steps.append((("s_full", u, buf), sn, [("s_empty", u, buf)]))
                            sn += 1
                        steps.append((None, 0, [("i_empty", buf)]))
                    qc += nq
                    if skip < nq and nq > 1 and (active or exchange_in_empty_tiles):
                        bar = ("x_full", u, xn & 3)
                        if skip == 0:
                            steps.append((None, 0, [bar]))
                        else:
                            self.reads.append((len(actors), len(steps), bar, xn >> 2))
                            steps.append((bar, xn >> 2, []))
                        xn += 1
                actors.append(steps)
        self.actors = actors
        for h in range(2):
            self.count["i_empty", h] = 2
        # completed phases of every barrier by how far each actor has come
        self.arrivals = [{} for _ in actors]
        for a, steps in enumerate(actors):
            for i, (_, _, bars) in enumerate(steps):
                for b in bars:
                    self.arrivals[a].setdefault(b, []).append(i)

    def phases(self, bar, at):
        """Phases of a barrier that the steps taken so far complete: every actor arrives once a phase."""
        per = [sum(1 for i in self.arrivals[a].get(bar, ()) if i < at[a])
               for a in range(len(self.actors)) if bar in self.arrivals[a]]
        if not per:
            return 0
        return min(per) if bar in self.count else sum(per)

    def passes(self, wait, phase, at):
        if wait is None or phase < 0:
            return True
        # a wait by parity: the phase under way is of the other parity
        return self.phases(wait, at) % 2 != phase % 2

    def walk(self, limit=3_000_000):
        """Every reachable state: (an exchange that overtakes its reader or None, whether all orders end)."""
        start = tuple(0 for _ in self.actors)
        end = tuple(len(s) for s in self.actors)
        seen, todo, ends = {start}, [start], True
        while todo:
            at = todo.pop()
            for actor, step, bar, phase in self.reads:
                if at[actor] <= step and self.phases(bar, at) > phase + 1:
                    return (actor, step, bar, phase), ends
            moved = False
            for a, steps in enumerate(self.actors):
                if at[a] < len(steps) and self.passes(steps[at[a]][0], steps[at[a]][1], at):
                    moved = True
                    nxt = at[:a] + (at[a] + 1,) + at[a + 1:]
                    if nxt not in seen:
                        seen.add(nxt)
                        todo.append(nxt)
            if not moved and at != end:
                ends = False
            assert len(seen) < limit, "too many states for a test"
        return None, ends


BATCHES = [
    [(2, 0)] * 7,                                       # blocks of up to 128 tokens, two query tiles
    [(2, 1)] + [(2, 0)] * 6,
    [(2, 0), (2, 0), (2, 1), (2, 0), (2, 0), (2, 0), (2, 1)],
    [(3, 0), (2, 0), (1, 0), (2, 0), (3, 0), (2, 0), (2, 0)],
    [(2, 1)] * 6,
    [(3, 1), (1, 1), (2, 1), (3, 1), (2, 1)],
    [(1, 0), (1, 1), (2, 0), (2, 1), (1, 1), (2, 1), (2, 0), (2, 0)],
]


@pytest.mark.parametrize("items", BATCHES)
def test_no_exchange_overtakes_its_reader(items):
    overtaken, ends = Model(items, exchange_in_empty_tiles=False).walk()
    assert overtaken is None and ends


@pytest.mark.parametrize("items", BATCHES[:3])
def test_the_model_sees_an_exchange_in_tiles_without_tokens(items):
    overtaken, _ = Model(items, exchange_in_empty_tiles=True).walk()
    assert overtaken is not None
