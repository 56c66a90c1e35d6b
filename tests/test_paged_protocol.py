"""Model of the barrier protocol of paged_prompt_kernel (k_paged.cu), checked under random schedules (no GPU): which
mbarrier each role waits on, for which use of it, and what it arrives on, with copies completing in random order and
products in the order of their issue for one accumulator, in any order for several.  Checked: every wait ends after the phase that it means and no other, no schedule
stalls, and no buffer is written while it is still read."""

import random

import pytest

from test_protocol_models import Bar, run_agents, waitable


def prompt_cta(items, stages, rnd, skip=None):
    """items: (key tiles of row tile 0, of row tile 1, whether tile 1 has rows).  skip: a wait that is left out (planted)."""
    q_full, q_empty, drain = Bar("q_full", 1), Bar("q_empty", 1), Bar("drain", 1)
    kf, ke, vf, ve = ([Bar(f"{x}{s}", 1) for s in range(stages)] for x in ("k_full", "k_empty", "v_full", "v_empty"))
    sf, pf, pv = ([Bar(f"{x}{t}", c) for t in range(2)] for x, c in (("s_full", 1), ("p_full", 8), ("pv_done", 1)))
    pending, tensor = [], []
    held_q = [None]
    held_k, held_v = [None] * stages, [None] * stages  # key tile that each stage holds
    s_of = [None, None]   # (item, step) whose S, then P, lies in S_t: ("s" or "p", k, j)
    o_of = [None, None]   # item that O_t accumulates, and the steps it has
    o_read = [set(), set()]
    out = [dict(), dict()]

    def waits(bar, phase, name=None):
        if name is not None and name == skip:
            return
        while not waitable(bar, phase):
            yield

    def complete_tensor():
        firsts = {}
        for op in tensor:
            if not op["done"]:
                firsts.setdefault(op["acc"], op)
        op = rnd.choice(list(firsts.values()))
        op["effect"]()
        op["done"] = True
        while tensor and tensor[0]["done"]:  # a commit covers all that was issued before it
            for b in tensor.pop(0)["bars"]:
                b.arrive()

    def issue_op(acc, effect, bars):
        tensor.append(dict(acc=acc, effect=effect, bars=bars, done=False))
        pending.append(complete_tensor)

    def producer():
        g = 0
        for k, (n0, n1, _) in enumerate(items):
            if k >= 1:
                yield from waits(q_empty, k - 1, "q_empty")

            def q_lands(k=k):
                held_q[0] = k
                q_full.arrive()

            pending.append(q_lands)
            for j in range(max(n0, n1)):
                s, use = g % stages, g // stages
                for full, empty, held, name in ((kf, ke, held_k, "k_empty"), (vf, ve, held_v, "v_empty")):
                    if g >= stages:
                        yield from waits(empty[s], use - 1, name)
                    held[s] = None  # (the copy may write from now on)

                    def lands(full=full, held=held, s=s, g=g):
                        held[s] = g
                        full[s].arrive()

                    pending.append(lands)
                    yield
                g += 1

    def mma():
        g = 0
        par_s, par_pv = [0, 0], [0, 0]  # products of either kind so far
        todo = [None, None]

        def issue(t, k, j, act, q_last):
            if todo[t]:
                pk, pj, v = todo[t]
                s = v % stages
                yield from waits(pf[t], par_pv[t], "p_full")
                yield from waits(vf[s], v // stages, "v_full")

                def effect(s=s):
                    assert s_of[t] == ("p", pk, pj), ("P V of another tile", s_of[t], pk, pj)
                    assert held_v[s] == v, "V is not there"
                    if pj == 0:
                        assert o_of[t] is None or o_of[t][0] in o_read[t], "O overwritten before it was read"
                        o_of[t] = (pk, 0)
                    assert o_of[t] == (pk, pj)
                    o_of[t] = (pk, pj + 1)
                    s_of[t] = None

                issue_op(("o", t), effect, [pv[t]] + ([ve[s]] if t == 1 or not todo[1] else []))
                par_pv[t] += 1
                yield
            if not act[t]:
                return
            s = g % stages
            yield from waits(kf[s], g // stages, "k_full")
            if par_s[t]:
                yield from waits(pv[t], par_s[t] - 1, "pv_done")

            def effect(g=g, s=s):
                assert s_of[t] is None, ("S overwrites", s_of[t])
                assert held_q[0] == k and held_k[s] == g, "Q or K is not there"
                s_of[t] = ("s", k, j)

            last = t == 1 or not act[1]
            issue_op(("s", t), effect, [sf[t]] + ([ke[s]] if last else []) + ([q_empty] if last and q_last else []))
            par_s[t] += 1
            yield

        for k, (n0, n1, _) in enumerate(items):
            yield from waits(q_full, k, "q_full")
            for j in range(max(n0, n1)):
                act = (j < n0, j < n1)
                for t in range(2):
                    yield from issue(t, k, j, act, j + 1 == max(n0, n1))
                todo = [(k, j, g) if act[t] else None for t in range(2)]
                g += 1
        for t in range(2):
            yield from issue(t, 0, 0, (False, False), False)
        issue_op("end", lambda: None, [drain])
        yield from waits(drain, 0)

    def softmax(t):
        g0 = n = 0
        for k, (n0, n1, two) in enumerate(items):
            nk = (n0, n1)[t]
            if t == 0 or two:
                for j in range(nk):
                    yield from waits(sf[t], n, "s_full")
                    assert s_of[t] == ("s", k, j), ("read another S", s_of[t], k, j)
                    if j:
                        assert o_of[t] == (k, j), "O rescaled before its products"
                    yield
                    if j + 1 == max(n0, n1) and rnd.random() < 0.5:  # the last tile's V rows past the end
                        v = g0 + j
                        yield from waits(vf[v % stages], v // stages)
                        assert held_v[v % stages] == v
                    s_of[t] = ("p", k, j)
                    pf[t].arrive(8)
                    yield
                    n += 1
                if nk:
                    yield from waits(pv[t], n - 1, "pv_last")
                    assert o_of[t] == (k, nk), "output read before its last product"
                    out[t][k] = nk
                    yield
                    o_read[t].add(k)
            g0 += max(n0, n1)

    run_agents([producer(), mma(), softmax(0), softmax(1)], pending, rnd)
    assert out == [{k: i[t] for k, i in enumerate(items) if i[t]} for t in range(2)]


def draw(rnd, most=6):
    items = []
    for _ in range(rnd.randint(1, 6)):
        n1 = rnd.randint(1, most)
        if rnd.random() < 0.3:
            items.append((n1, 0, False))            # one row tile only
        else:
            items.append((rnd.randint(0, n1), n1, True))  # tile 0 sees no more than tile 1
    return items


@pytest.mark.parametrize("stages", [2, 4])
@pytest.mark.parametrize("seed", range(150))
def test_prompt_protocol(seed, stages):
    rnd = random.Random(seed)
    prompt_cta(draw(rnd, rnd.choice([1, 2, 6])), stages, rnd)


@pytest.mark.parametrize("skip", ["q_empty", "k_empty", "v_empty", "p_full", "v_full", "pv_done", "k_full", "q_full",
                                  "s_full", "pv_last"])
def test_a_wait_left_out_is_found(skip):
    found = 0
    for seed in range(200):
        rnd = random.Random(1000 + seed)
        try:
            prompt_cta(draw(rnd, rnd.choice([1, 2, 6])), rnd.choice([2, 4]), rnd, skip)
        except AssertionError:
            found += 1
    assert found
