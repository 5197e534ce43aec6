"""CPU models of the barrier protocols of the multi-head cross attention's kernels
(csrc/sa_cross_fwd.cu, csrc/sa_cross_bwd.cu), in the style of the other kernels' models: each
role of one CTA runs as a coroutine over a list of items, TMA landings and tensor-pipe
completions (one in-order pipe) come in random order, and barriers follow mbarrier phase and
parity semantics: a wait passes when the phase before the current one has the awaited parity, so
it tells adjacent phases apart only. A wait for a phase whose predecessor was never waited for
can therefore pass early, or miss a phase that came and went; such slips are planted here and must be caught.

Checked: no deadlock; every MMA reads its own tiles, scores and weights; no TMA load, MMA or
store overwrites what is still to be read; an accumulator is rescaled and written with none of
its MMAs pending, holds exactly its item's tiles, and is not overwritten before it was written.
"""
import random

import pytest

from test_fwd_barrier_protocol import Bar, Violation, check
from test_stca_barrier_protocol import _engine


def _tma(later, bars, slot_use, slot, what, seq):
    """One load of `what` into a slot: the caller has waited for the slot's empty barrier."""
    bars["full"][slot].arrive_expect_tx(1)

    def land():
        check(slot_use[slot] == 0, f"load of {what} into slot {slot} in use")
        seq[slot] = what
        bars["full"][slot].complete_tx(1)
    later(land, 1, 90)


def run_forward(items, NS, NB, seed, hand_waits_k=True, hand_frees=True, last_output=True, one_step_wait=True, empty_phases=False):
    """items: (key tiles, two tiles of rows). NS ring stages, NB score buffers."""
    rnd = random.Random(seed)
    later, issue, run = _engine(rnd)
    bars = dict(full=[Bar(1) for _ in range(NS)], empty=[Bar(2 if hand_frees else 1) for _ in range(NS)],
                v_ready=[Bar(1) for _ in range(8)], s_full=[Bar(1) for _ in range(NB)],
                p_full=[Bar(4) for _ in range(NB)], o_done=[Bar(1), Bar(1)], o_last=[Bar(1), Bar(1)],
                q_full=Bar(1), q_empty=Bar(1), o_free=Bar(2), merge=Bar(1))
    use, seq = [0] * NS, [None] * NS
    st = dict(Q=None, quse=0, S=[None] * NB, sread=[0] * NB, P=[None] * NB, ready=set(), O=[[], []], pend=[0, 0],
              ml=None)

    def tma():
        i = nq = 0
        for s, (n, two) in enumerate(items):
            if n == 0:
                continue
            p = (nq & 1) ^ 1
            yield lambda: bars["q_empty"].passes(p)
            nq += 1
            bars["q_full"].arrive_expect_tx(1)

            def land(s=s):
                check(st["quse"] == 0, "Q overwritten in use")
                st["Q"] = s
                bars["q_full"].complete_tx(1)
            later(land)
            for x in range(2 * n):
                slot, p = i % NS, ((i // NS) & 1) ^ 1
                yield lambda: bars["empty"][slot].passes(p)
                _tma(later, bars, use, slot, ("KV"[x & 1], s, x >> 1), seq)
                i += 1

    def hand():
        base = v = 0
        for s, (n, two) in enumerate(items):
            for j in range(n):
                i = base + 2 * j + 1
                if hand_waits_k:
                    yield lambda: bars["full"][(i - 1) % NS].passes(((i - 1) // NS) & 1)
                if hand_frees:
                    bars["empty"][(i - 1) % NS].arrive()
                yield lambda: bars["full"][i % NS].passes((i // NS) & 1)
                check(seq[i % NS] == ("V", s, j), f"V({s},{j}) handed on before it landed")
                bars["v_ready"][v & 7].arrive()
                if hand_frees:
                    bars["empty"][i % NS].arrive()
                v += 1
            base += 2 * n

    def mma():
        kpos, vpos, sb, pb, vi, nq, free = 0, 1, 0, 0, 0, 0, 0
        for s, (n, two) in enumerate(items):
            if n == 0:
                free += 1 if empty_phases else 0
                continue
            steps = 2 * n if two else n
            yield lambda: bars["q_full"].passes(nq & 1)
            nq += 1

            def scores(q, s=s, two=two, steps=steps):
                nonlocal kpos, sb
                j = q >> 1 if two else q
                slot, par, b = kpos % NS, (kpos // NS) & 1, sb % NB
                yield lambda: bars["full"][slot].passes(par)

                def start():
                    check(seq[slot] == ("K", s, j), f"S({s},{q}) read {seq[slot]}")
                    check(st["Q"] == s, f"S({s},{q}) read the queries of {st['Q']}")
                    check(st["sread"][b] == 0, f"S({s},{q}) overwrote scores still read")
                    use[slot] += 1
                    st["quse"] += 1

                def finish():
                    use[slot] -= 1
                    st["quse"] -= 1
                    st["S"][b], st["P"][b] = (s, q), None
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
            if free > 0:
                yield lambda: bars["o_free"].passes((free - 1) & 1)
            free += 1
            for q in range(steps):
                w, j, b, par = q & 1, q >> 1 if two else q, pb % NB, (pb // NB) & 1
                slot, v = vpos % NS, vi
                yield lambda: bars["v_ready"][v & 7].passes((v >> 3) & 1)
                yield lambda: bars["p_full"][b].passes(par)
                st["pend"][w] += 1

                def start(w=w, j=j, b=b, slot=slot, q=q, s=s):
                    check(seq[slot] == ("V", s, j), f"O({s},{q}) read {seq[slot]}")
                    check(st["P"][b] == (s, q), f"O({s},{q}) read the weights of {st['P'][b]}")
                    use[slot] += 1
                    if q < 2:
                        check(st["O"][w] in ([], "written"), f"O({s},{q}) overwrote {st['O'][w]} before it was written")
                        st["O"][w] = []

                def finish(w=w, j=j, b=b, slot=slot, q=q, s=s, two=two, steps=steps):
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

    def softmax(w):
        base = cnt = singles = lasts = filled = 0
        for s, (n, two) in enumerate(items):
            steps = 2 * n if two else n
            mine = list(range(w, steps, 2))
            for k, q in enumerate(mine):
                b, par = (base + q) % NB, ((base + q) // NB) & 1
                yield lambda: bars["s_full"][b].passes(par)
                check(st["S"][b] == (s, q), f"softmax ({s},{q}) read {st['S'][b]}")
                st["sread"][b] += 1
                yield None
                if k > 0 and rnd.random() < 0.3:  # the maximum is raised
                    yield lambda: bars["o_done"][w].passes((cnt - 1) & 1)
                    check(st["pend"][w] == 0 and len(st["O"][w]) == k, f"rescale at ({s},{q}) with an MMA pending")
                st["sread"][b] -= 1
                st["P"][b] = (s, q)
                cnt += 1
                bars["p_full"][b].arrive(4)
            base += steps
            if mine:
                if last_output:
                    yield lambda: bars["o_last"][w].passes(lasts & 1)
                else:
                    yield lambda: bars["o_done"][w].passes((cnt - 1) & 1)
                lasts += 1
            if n == 0 and not empty_phases:
                continue
            if w == 1 and filled > 0:
                yield lambda: bars["o_free"].passes((filled - 1) & 1)
            filled += 1
            want = [[(s, j) for j in range(n)]] * 2 if two else [[(s, j) for j in range(x, n, 2)] for x in (0, 1)]
            if w == 1 and one_step_wait:
                yield lambda: bars["o_last"][0].passes((filled - 1) & 1)
            read = (w,) if two else (0, 1) if w == 0 else ()
            if not two:
                if w == 1:
                    st["ml"] = s
                    bars["merge"].arrive()
                else:
                    yield lambda: bars["merge"].passes(singles & 1)
                    check(st["ml"] == s, f"item {s} merged with the state of {st['ml']}")
                singles += 1
            for x in read:
                if want[x]:
                    check(st["pend"][x] == 0 and st["O"][x] == want[x],
                          f"item {s}: O_{x} written holding {st['O'][x]}, {st['pend'][x]} pending")
            yield None
            for x in read:
                if want[x]:
                    check(st["O"][x] == want[x], f"item {s}: O_{x} changed while written")
                    st["O"][x] = "written"
            bars["o_free"].arrive()

    run([tma(), hand(), mma(), softmax(0), softmax(1)])


def _items(rnd, most=7):
    return [(rnd.choice([0, 1, 2, 3, rnd.randint(1, most)]), rnd.random() < 0.6) for _ in range(rnd.randint(1, 5))]


@pytest.mark.parametrize("NS,NB", [(5, 2), (8, 3)])
def test_forward_protocol_random_schedules(NS, NB):
    rnd = random.Random(900 + NS)
    for trial in range(250):
        run_forward(_items(rnd), NS, NB, seed=trial)


@pytest.mark.parametrize("NS,NB,planted", [(5, 2, "hand_waits_k"), (5, 2, "hand_frees"), (8, 3, "last_output"),
                                           (5, 2, "one_step_wait"), (5, 2, "empty_phases")])
def test_forward_model_catches_waits_that_skip_a_phase(NS, NB, planted):
    rnd = random.Random(901)
    found = 0
    for trial in range(600):
        try:
            run_forward(_items(rnd), NS, NB, seed=trial, **{planted: planted == "empty_phases"})
        except (Violation, AssertionError):  # the latter: an arrival that the barrier does not expect
            found += 1
    assert found > 0, planted


def run_backward(items, NK, NV, NB, seed, stats_wait=True, acc_wait=True, v_wait=True, hand_frees=True, own_p_full=True,
                 empty_phases=False):
    """items: ("dkv" | "dq", steps). NK long-held and NV short-held slots, NB S^T buffers of dK/dV."""
    rnd = random.Random(seed)
    later, issue, run = _engine(rnd)
    slots = NK + NV
    bars = dict(full=[Bar(1) for _ in range(slots)], empty=[Bar(2 if hand_frees and x >= NK else 1) for x in range(slots)],
                ready=[Bar(1) for _ in range(8)], own=Bar(1), own_empty=Bar(1), s_full=[Bar(1), Bar(1)],
                dp_full=Bar(1), p_full=[Bar(2), Bar(2)], ds_full=[Bar(2), Bar(2)], done=Bar(1), acc_free=Bar(2))
    use, seq = [0] * slots, [None] * slots
    st = dict(own=None, ownuse=0, S=[None, None], sread=[0, 0], P=[None, None], dP=None, dpread=0, dS=None,
              dSq=[None, None], stat=[None, None], acc=None, acc_read=0, pend=0)

    def tma():
        used, own = [0] * slots, 0
        for s, (kind, n) in enumerate(items):
            if n == 0:
                continue
            yield lambda: bars["own_empty"].passes((own & 1) ^ 1)
            own += 1
            bars["own"].arrive_expect_tx(1)

            def land(s=s):
                check(st["ownuse"] == 0, "own tiles overwritten in use")
                st["own"] = s
                bars["own"].complete_tx(1)
            later(land)
            for x in range(n):
                for v in (0, 1):
                    slot = NK + x % NV if v else x % NK
                    yield lambda: bars["empty"][slot].passes((used[slot] & 1) ^ 1)
                    _tma(later, bars, use, slot, ("xy"[v], s, x), seq)
                    used[slot] += 1

    def hand():
        loaded, step = [0] * slots, 0
        for s, (kind, n) in enumerate(items):
            for i in range(n):
                x, y = i % NK, NK + i % NV
                px, py = loaded[x] & 1, loaded[y] & 1
                loaded[x] += 1
                loaded[y] += 1
                yield lambda: bars["full"][x].passes(px)
                check(seq[x] == ("x", s, i), f"slot {x} handed on holding {seq[x]}")
                if kind == "dkv":
                    yield lambda: bars["full"][y].passes(py)
                    check(seq[y] == ("y", s, i), f"slot {y} handed on holding {seq[y]}")
                    if step >= 2 and stats_wait:
                        yield lambda: bars["ds_full"][step & 1].passes(((step >> 1) & 1) ^ 1)
                    check(st["stat"][step & 1] in (None, "read"), f"statistics of {st['stat'][step & 1]} overwritten")
                    st["stat"][step & 1] = (s, i)
                bars["ready"][step & 7].arrive()
                if kind == "dq" and v_wait:
                    yield lambda: bars["full"][y].passes(py)
                if hand_frees:
                    bars["empty"][y].arrive()
                step += 1

    def mma():
        own = steps = free = 0
        pcnt = [0, 0]
        loaded = [0] * slots
        for s, (kind, n) in enumerate(items):
            if n == 0:
                free += 1 if empty_phases else 0
                continue
            yield lambda: bars["own"].passes(own & 1)
            own += 1
            dkv = kind == "dkv"
            nb = NB if dkv else 2

            def scores(i, s=s, n=n, nb=nb, steps=steps):
                b, slot = (i & 1) if nb == 2 else 0, i % NK
                k = steps + i
                yield lambda: bars["ready"][k & 7].passes((k >> 3) & 1)

                def start():
                    check(st["own"] == s and seq[slot] == ("x", s, i), f"S({s},{i}) read {seq[slot]}, own {st['own']}")
                    check(st["sread"][b] == 0, f"S({s},{i}) overwrote scores still read")
                    use[slot] += 1
                    st["ownuse"] += 1

                def finish():
                    use[slot] -= 1
                    st["ownuse"] -= 1
                    st["S"][b], st["P"][b], st["dSq"][b] = (s, i), None, None
                    bars["s_full"][b].arrive()
                issue(start, finish)

            def dprob(i, s=s, n=n, dkv=dkv):
                slot = NK + i % NV
                if not dkv:
                    par = loaded[slot] & 1
                    yield lambda: bars["full"][slot].passes(par)
                loaded[slot] += 1

                def start():
                    check(st["own"] == s and seq[slot] == ("y", s, i), f"dP({s},{i}) read {seq[slot]}")
                    check(st["dpread"] == 0, f"dP({s},{i}) overwrote values still read")
                    check(dkv or st["acc"] is None or st["acc"][0] == s, f"dP({s},{i}) overwrote the sums of {st['acc']}")
                    use[slot] += 1
                    st["ownuse"] += 1

                def finish():
                    use[slot] -= 1
                    st["ownuse"] -= 1
                    st["dP"], st["dS"] = (s, i), None
                    bars["dp_full"].arrive()
                    if not dkv:
                        bars["empty"][slot].arrive()
                    if i == n - 1:
                        bars["own_empty"].arrive()
                issue(start, finish)

            def wait_acc():
                nonlocal free
                if free > 0 and acc_wait:
                    yield lambda: bars["acc_free"].passes((free - 1) & 1)
                free += 1

            def accumulate(i, slot, what, read, s=s, kind=kind):
                st["pend"] += 1

                def start():
                    check(seq[slot] == (what, s, i), f"{kind} accumulate ({s},{i}) read {seq[slot]}")
                    check(read() == (s, i), f"{kind} accumulate ({s},{i}) read the packed tile of {read()}")
                    check(st["acc"] is None or st["acc"][0] == s, f"item {s} overwrote the sums of {st['acc']}")
                    st["acc"] = (s, "sums")
                    use[slot] += 1

                def finish():
                    use[slot] -= 1
                    st["pend"] -= 1
                    bars["empty"][slot].arrive()
                issue(start, finish)

            yield from scores(0)
            if dkv:
                yield from dprob(0)
                if nb == 2 and n > 1:
                    yield from scores(1)
                yield from wait_acc()
            else:
                yield from wait_acc()
                yield from dprob(0)
                if n > 1:
                    yield from scores(1)
            for i in range(n):
                k = steps + i
                b = (i & 1) if nb == 2 else 0
                if dkv:
                    pb = b if own_p_full else 0
                    yield lambda: bars["p_full"][pb].passes(pcnt[pb] & 1)
                    pcnt[pb] += 1
                    accumulate(i, NK + i % NV, "y", lambda b=b: st["P"][b])
                    if i + nb < n:
                        yield from scores(i + nb)
                yield lambda: bars["ds_full"][k & 1].passes((k >> 1) & 1)
                if dkv:
                    accumulate(i, i % NK, "x", lambda: st["dS"])
                    if i + 1 < n:
                        yield from dprob(i + 1)
                else:
                    if i + 1 < n:
                        yield from dprob(i + 1)
                    accumulate(i, i % NK, "x", lambda b=b: st["dSq"][b])
                    if i + 2 < n:
                        yield from scores(i + 2)
            steps += n
            issue(lambda: None, lambda: bars["done"].arrive())

    def elementwise(w):
        own = steps = 0
        uses = [0, 0]
        for s, (kind, n) in enumerate(items):
            dkv = kind == "dkv"
            nb = NB if dkv else 2
            for i in range(n):
                b = (i & 1) if nb == 2 else 0
                if dkv:
                    yield lambda: bars["ready"][steps & 7].passes((steps >> 3) & 1)
                yield lambda: bars["s_full"][b].passes(uses[b] & 1)
                uses[b] += 1
                check(st["S"][b] == (s, i), f"elementwise ({s},{i}) read S of {st['S'][b]}")
                st["sread"][b] += 1
                if dkv:
                    check(st["stat"][steps & 1] == (s, i), f"elementwise ({s},{i}) read {st['stat'][steps & 1]}")
                yield None
                if dkv:  # (each warpgroup its own columns; the tile counts once both have arrived)
                    st["sread"][b] -= 1
                    st["P"][b] = (s, i)
                    bars["p_full"][b if own_p_full else 0].arrive()
                yield lambda: bars["dp_full"].passes(steps & 1)
                check(st["dP"] == (s, i), f"elementwise ({s},{i}) read dP of {st['dP']}")
                st["dpread"] += 1
                if dkv:
                    check(st["stat"][steps & 1] == (s, i), f"elementwise ({s},{i}) read {st['stat'][steps & 1]}")
                yield None
                st["dpread"] -= 1
                if dkv:
                    st["dS"] = (s, i)
                    if bars["ds_full"][steps & 1].pend == 1:
                        st["stat"][steps & 1] = "read"
                else:
                    st["sread"][b] -= 1
                    st["dSq"][b] = (s, i)
                bars["ds_full"][steps & 1].arrive()
                steps += 1
            if n > 0:
                yield lambda: bars["done"].passes(own & 1)
                own += 1
                check(st["acc"] == (s, "sums") and st["pend"] == 0, f"item {s} written from {st['acc']}, {st['pend']} pending")
                yield None
                check(st["acc"] == (s, "sums"), f"item {s}: sums changed while written")
                st["acc_read"] += 1
                if st["acc_read"] == 2:
                    st["acc"], st["acc_read"] = None, 0
            if n > 0 or empty_phases:
                bars["acc_free"].arrive()

    run([tma(), hand(), mma(), elementwise(0), elementwise(1)])


def _bwd_items(rnd):
    return [(rnd.choice(["dkv", "dq"]), rnd.choice([0, 1, 2, 3, rnd.randint(1, 8)])) for _ in range(rnd.randint(1, 5))]


@pytest.mark.parametrize("NK,NV,NB", [(3, 2, 1), (5, 3, 2)])
def test_backward_protocol_random_schedules(NK, NV, NB):
    rnd = random.Random(950 + NK)
    for trial in range(250):
        run_backward(_bwd_items(rnd), NK, NV, NB, seed=trial)


@pytest.mark.parametrize("NK,NV,NB,planted", [(5, 3, 2, "stats_wait"), (3, 2, 1, "acc_wait"), (3, 2, 1, "v_wait"),
                                              (3, 2, 1, "hand_frees"), (5, 3, 2, "own_p_full"),
                                              (3, 2, 1, "empty_phases")])
def test_backward_model_catches_planted_races(NK, NV, NB, planted):
    rnd = random.Random(951)
    found = 0
    for trial in range(800):
        try:
            run_backward(_bwd_items(rnd), NK, NV, NB, seed=trial, **{planted: planted == "empty_phases"})
        except (Violation, AssertionError):  # the latter: an arrival that the barrier does not expect
            found += 1
    assert found > 0, planted
