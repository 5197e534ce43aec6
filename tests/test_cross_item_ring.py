"""CPU model of the cross attention's forward by warps (csrc/sa_cross_fwd.cu), with what the model by warpgroups
(test_cross_barrier_protocol.py) leaves out: the warp that reads the schedule and the ring of two items that it
hands to eleven others, of which the eight softmax warps read their item in place until they have what its
rows need; P's two halves, each with a barrier of its own; the order of the waits at an item's end. Engine,
barriers and checks are that model's. The backward's ring is the same with copies in every reader."""
import random

import pytest

from test_cross_barrier_protocol import _tma
from test_fwd_barrier_protocol import Bar, Violation, check
from test_stca_barrier_protocol import _engine


def run(items, NS, NB, seed, ring_wait=True, in_place=True, second_half=True, state_wait=True, one_step_wait=True,
        every_reader=True):
    rnd = random.Random(seed)
    later, issue, go = _engine(rnd)
    bars = dict(full=[Bar(1) for _ in range(NS)], empty=[Bar(2) for _ in range(NS)], v_ready=[Bar(1) for _ in range(8)],
                s_full=[Bar(1) for _ in range(NB)], p_full=[[Bar(4), Bar(4)] for _ in range(NB)],
                o_done=[Bar(1), Bar(1)], o_last=[Bar(1), Bar(1)], q_full=Bar(1), q_empty=Bar(1), o_free=Bar(8),
                merge=Bar(4), item_full=[Bar(1), Bar(1)], item_empty=[Bar(11 if every_reader else 10) for _ in range(2)])
    use, seq, ring = [0] * NS, [None] * NS, [None, None]
    st = dict(Q=None, quse=0, S=[None] * NB, sread=[0] * NB, P=[[None] * 8 for _ in range(NB)], O=[[], []], pend=[0, 0],
              ml=[None] * 4)

    def schedule():
        for s in range(len(items) + 1):
            if ring_wait:
                yield lambda: bars["item_empty"][s & 1].passes(((s >> 1) & 1) ^ 1)
            else:
                yield None
            ring[s & 1] = s
            bars["item_full"][s & 1].arrive()

    def get(s):
        """The s-th item, copied; None behind the last one."""
        yield lambda: bars["item_full"][s & 1].passes((s >> 1) & 1)
        check(ring[s & 1] == s, f"item {s} read as {ring[s & 1]}")
        bars["item_empty"][s & 1].arrive()

    def tma():
        i = nq = 0
        for s in range(len(items) + 1):
            yield from get(s)
            n = items[s][0] if s < len(items) else 0
            if n == 0:
                continue
            yield lambda: bars["q_empty"].passes((nq & 1) ^ 1)
            nq += 1
            bars["q_full"].arrive_expect_tx(1)

            def land(s=s):
                check(st["quse"] == 0, "Q overwritten in use")
                st["Q"] = s
                bars["q_full"].complete_tx(1)
            later(land)
            for x in range(2 * n):
                slot = i % NS
                yield lambda: bars["empty"][slot].passes(((i // NS) & 1) ^ 1)
                _tma(later, bars, use, slot, ("KV"[x & 1], s, x >> 1), seq)
                i += 1

    def hand():
        i = v = 0
        for s in range(len(items) + 1):
            yield from get(s)
            for j in range(items[s][0] if s < len(items) else 0):
                for kind in "KV":
                    yield lambda: bars["full"][i % NS].passes((i // NS) & 1)
                    check(seq[i % NS] == (kind, s, j), f"{kind}({s},{j}) handed on as {seq[i % NS]}")
                    if kind == "V":
                        bars["v_ready"][v & 7].arrive()
                        v += 1
                    bars["empty"][i % NS].arrive()
                    i += 1

    def mma():
        kpos, vpos, sb, pb, vi, nq = 0, 1, 0, 0, 0, 0
        for s in range(len(items) + 1):
            yield from get(s)
            n, two = items[s] if s < len(items) else (0, False)
            if n == 0:
                continue
            steps = 2 * n if two else n
            yield lambda: bars["q_full"].passes(nq & 1)
            nq += 1

            def scores(q, s=s, two=two, steps=steps):
                nonlocal kpos, sb
                j, slot, b = q >> 1 if two else q, kpos % NS, sb % NB
                yield lambda: bars["full"][slot].passes((kpos // NS) & 1)

                def start():
                    check(seq[slot] == ("K", s, j) and st["Q"] == s, f"S({s},{q}) read {seq[slot]}, queries {st['Q']}")
                    check(st["sread"][b] == 0, f"S({s},{q}) overwrote scores still read")
                    use[slot] += 1
                    st["quse"] += 1

                def finish():
                    use[slot] -= 1
                    st["quse"] -= 1
                    st["S"][b], st["P"][b] = (s, q), [None] * 8
                    bars["s_full"][b].arrive()
                    if not two or q & 1:
                        bars["empty"][slot].arrive()
                    if q == steps - 1:
                        bars["q_empty"].arrive()
                issue(start, finish)
                sb += 1
                if not two or q & 1:
                    kpos += 2
            for q in range(min(NB, steps)):
                yield from scores(q)
            if nq > 1:
                yield lambda: bars["o_free"].passes(nq & 1)
            for q in range(steps):
                w, j, b, slot, par = q & 1, q >> 1 if two else q, pb % NB, vpos % NS, (pb // NB) & 1
                yield lambda: bars["v_ready"][vi & 7].passes((vi >> 3) & 1)
                for h in (0, 1):
                    if h == 0 or second_half:
                        yield lambda: bars["p_full"][b][h].passes(par)
                    if h == 0:
                        st["pend"][w] += 1

                    def start(w=w, j=j, b=b, slot=slot, q=q, s=s, h=h):
                        check(seq[slot] == ("V", s, j), f"O({s},{q}) read {seq[slot]}")
                        check(st["P"][b][4 * h:4 * h + 4] == [(s, q)] * 4, f"O({s},{q}) read half {h}: {st['P'][b]}")
                        if h == 0:
                            use[slot] += 1
                        if h == 0 and q < 2:
                            check(st["O"][w] in ([], [None] * 4), f"O({s},{q}) overwrote {st['O'][w]} before it was written")
                            st["O"][w] = []

                    def finish(w=w, j=j, slot=slot, q=q, s=s, h=h, two=two, steps=steps):
                        if h == 0:
                            return
                        use[slot] -= 1
                        st["O"][w].append((s, j))
                        st["pend"][w] -= 1
                        bars["o_done"][w].arrive()
                        if q + 2 >= steps:
                            bars["o_last"][w].arrive()
                        if not two or w == 1:
                            bars["empty"][slot].arrive()
                    issue(start, finish)
                pb += 1
                if not two or w == 1:
                    vpos += 2
                    vi += 1
                if q + NB < steps:
                    yield from scores(q + NB)

    written = {0: 0, 1: 0}  # warps that have written an accumulator's rows

    def softmax(w, q4):
        base = cnt = lasts = singles = filled = 0
        for s in range(len(items) + 1):
            yield lambda: bars["item_full"][s & 1].passes((s >> 1) & 1)
            check(ring[s & 1] == s, f"item {s} read as {ring[s & 1]}")
            if s == len(items):
                return
            if not in_place:
                bars["item_empty"][s & 1].arrive()
            n, two = items[s]
            steps = 2 * n if two else n
            mine = list(range(w, steps, 2))
            for k, q in enumerate(mine):
                b = (base + q) % NB
                yield lambda: bars["s_full"][b].passes(((base + q) // NB) & 1)
                check(st["S"][b] == (s, q), f"softmax ({s},{q}) read {st['S'][b]}")
                st["sread"][b] += 1
                yield None
                st["sread"][b] -= 1
                if k > 0 and rnd.random() < 0.3:  # a row's maximum is raised
                    yield lambda: bars["o_done"][w].passes((cnt - 1) & 1)
                    check(st["pend"][w] == 0 and len(st["O"][w]) == k, f"rescale at ({s},{q}) with an MMA pending")
                for h in (0, 1):
                    yield None
                    st["P"][b][4 * h + q4] = (s, q)
                    bars["p_full"][b][h].arrive()
                cnt += 1
            base += steps
            if mine:
                yield lambda: bars["o_last"][w].passes(lasts & 1)
                lasts += 1
            if w == 1 and n > 0 and state_wait:
                yield lambda: bars["o_free"].passes((filled & 1) ^ 1)
            if not two and n > 0:
                if w == 1:
                    st["ml"][q4] = s
                    bars["merge"].arrive()
                else:
                    yield lambda: bars["merge"].passes(singles & 1)
                    yield None
                    check(st["ml"][q4] == s, f"item {s} merged with the state of {st['ml'][q4]}")
                singles += 1
            if w == 1 and n > 0 and one_step_wait:
                yield lambda: bars["o_last"][0].passes(filled & 1)
            filled += n > 0
            yield None
            check(ring[s & 1] == s, f"rows of item {s} by item {ring[s & 1]}")
            if in_place:
                bars["item_empty"][s & 1].arrive()
            want = [[(s, j) for j in range(n)]] * 2 if two else [[(s, j) for j in range(x, n, 2)] for x in (0, 1)]
            read = [x for x in ((w,) if two else (0, 1) if w == 0 else ()) if want[x]]
            for again in (0, 1):
                for x in read:
                    check(st["pend"][x] == 0 and st["O"][x] == want[x], f"item {s}: O_{x} written holding {st['O'][x]}")
                yield None
            for x in read:
                written[x] += 1
                if written[x] == 4:
                    written[x], st["O"][x] = 0, [None] * 4
            if n > 0:
                bars["o_free"].arrive()

    go([schedule(), tma(), hand(), mma(), *(softmax(w, q4) for w in (0, 1) for q4 in range(4))])


def _items(rnd):
    return [(rnd.choice([0, 1, 2, 3, rnd.randint(1, 7)]), rnd.random() < 0.6) for _ in range(rnd.randint(1, 6))]


@pytest.mark.parametrize("NS,NB", [(5, 2), (8, 3)])
def test_random_schedules(NS, NB):
    rnd = random.Random(700 + NS)
    for trial in range(200):
        run(_items(rnd), NS, NB, seed=trial)


@pytest.mark.parametrize("NS,NB", [(5, 2), (8, 3)])
@pytest.mark.parametrize("planted", ["ring_wait", "in_place", "second_half", "state_wait", "every_reader"])
def test_planted_slips_are_caught(NS, NB, planted):
    rnd, found = random.Random(701), 0
    for trial in range(300):
        try:
            run(_items(rnd), NS, NB, seed=trial, **{planted: False})
        except (Violation, AssertionError):
            found += 1
    assert found > 0, planted


def test_the_wait_of_items_of_one_step_is_caught():
    rnd, found = random.Random(702), 0
    for trial in range(600):
        try:
            run(_items(rnd), 5, 2, seed=trial, one_step_wait=False)
        except (Violation, AssertionError):
            found += 1
    assert found > 0
