"""Model of the barrier protocol of paged_prompt_kernel (k_paged.cu), checked under random schedules (no GPU): which
mbarrier each role waits on, for which use of it, and what it arrives on, with copies completing in random order and
products in the order in which their thread issued them.  Checked: every wait ends after the phase that it means and no
other, no schedule stalls, and no buffer is written while it is still read."""

import random

import pytest

from test_protocol_models import Bar, run_agents, waitable


def prompt_cta(items, stages, rnd, skip=None):
    """items: (key tiles of row tile 0, of row tile 1, whether tile 1 has rows).  skip: a wait left out (planted)."""
    qf, qe = Bar("q_full", 1), Bar("q_empty", 2)
    full, empty = ([[Bar(f"{kv}_{x}{s}", c) for s in range(stages)] for kv in "kv"]
                   for x, c in (("full", 1), ("empty", 2)))
    sf, pf = ([[Bar(f"{x}{t}{b}", c) for b in range(2)] for t in range(2)] for x, c in (("s_full", 1), ("p_full", 4)))
    od = [[Bar(f"o_done{t}{x}", 1) for x in range(2)] for t in range(2)]
    drain = [Bar(f"drain{t}", 1) for t in range(2)]
    pending, tensor = [], [[], []]  # tensor: the products of either MMA thread
    held_q = [None]
    held = [[None] * stages, [None] * stages]  # key tile that each stage of K and of V holds
    s_of = [[None, None], [None, None]]  # ("s" or "p", item, step) in the buffers of S_t
    o_of = [None, None]   # item that O_t accumulates, and the steps it has
    o_read = [set(), set()]
    out = [dict(), dict()]

    def waits(bar, phase, name=None):
        if name is not None and name == skip:
            return
        while not waitable(bar, phase):
            yield

    def issue(t, effect, bars):
        """A product: run in the order of its thread's, of the two threads' in any; its commits arrive behind it."""
        def complete():
            effect, bars = tensor[t].pop(0)
            effect()
            for b in bars:
                b.arrive()

        tensor[t].append((effect, bars))
        pending.append(complete)

    def producer(kv):
        """The thread that loads Q and K, or V."""
        g = 0
        for k, (n0, n1, _) in enumerate(items):
            if not kv:
                if k >= 1:
                    yield from waits(qe, k - 1, "q_empty")
                held_q[0] = None

                def q_lands(k=k):
                    held_q[0] = k
                    qf.arrive()

                pending.append(q_lands)
            for j in range(max(n0, n1)):
                s = g % stages
                if g >= stages:
                    yield from waits(empty[kv][s], g // stages - 1, "kv"[kv] + "_empty")
                held[kv][s] = None  # (the copy may write from now on)

                def lands(s=s, g=g):
                    held[kv][s] = g
                    full[kv][s].arrive()

                pending.append(lands)
                yield
                g += 1

    total = sum(max(n0, n1) for n0, n1, _ in items)

    def mma(t):
        """The thread of row tile t."""
        at = dict(k=0, j=0, g=0, n=0, ready=False)  # of S

        def next_s():
            last = at["j"] + 1 == max(items[at["k"]][:2])
            if last:
                issue(t, lambda: None, [qe])
                at["j"], at["k"] = -1, at["k"] + 1
            at["g"] += 1
            at["j"] += 1

        def prepare_s(end):
            while not at["ready"] and at["g"] < min(end, total):
                k, s = at["k"], at["g"] % stages
                yield from waits(full[0][s], at["g"] // stages, "k_full")
                if at["j"] == 0:
                    yield from waits(qf, k, "q_full")
                at["ready"] = at["j"] < items[k][t]
                if not at["ready"]:
                    empty[0][s].arrive()
                    next_s()
                yield

        def issue_s():
            k, j, g, s, b = at["k"], at["j"], at["g"], at["g"] % stages, at["n"] & 1

            def effect():
                assert s_of[t][b] is None, ("S overwrites", s_of[t][b])
                assert held_q[0] == k and held[0][s] == g, "Q or K is not there"
                s_of[t][b] = ("s", k, j)

            issue(t, effect, [sf[t][b], empty[0][s]])
            at["n"] += 1
            at["ready"] = False
            next_s()

        np, g = 0, 0
        for k, item in enumerate(items):
            item_end = g + max(item[0], item[1])
            for j in range(max(item[0], item[1])):
                while True:
                    yield from prepare_s(total if skip == "lead" else min(g + stages, item_end))
                    if not at["ready"] or at["n"] >= np + 2:
                        break
                    issue_s()
                    yield
                s, b = g % stages, np & 1
                yield from waits(full[1][s], g // stages, "v_full")
                if j >= item[t]:
                    empty[1][s].arrive()
                    g += 1
                    continue
                yield from waits(pf[t][b], np >> 1, "p_full")

                def effect(g=g, s=s, k=k, j=j, b=b):
                    assert s_of[t][b] == ("p", k, j), ("P V of another tile", s_of[t][b], k, j)
                    assert held[1][s] == g, "V is not there"
                    if j == 0:
                        assert o_of[t] is None or o_of[t][0] in o_read[t], "O overwritten before it was read"
                        o_of[t] = (k, 0)
                    assert o_of[t] == (k, j)
                    o_of[t] = (k, j + 1)
                    s_of[t][b] = None

                issue(t, effect, [empty[1][s]] + ([od[t][j == item[t] - 1]] if j >= item[t] - 2 else []))
                if at["ready"]:
                    issue_s()
                np += 1
                g += 1
                yield
        issue(t, lambda: None, [drain[t]])
        yield from waits(drain[t], 0)

    def softmax(t):
        g0 = n = 0
        n_o = [0, 0]

        for k, (n0, n1, two) in enumerate(items):
            nk = (n0, n1)[t]
            if t == 0 or two:
                for j in range(nk):
                    b = n & 1
                    yield from waits(sf[t][b], n >> 1, "s_full")
                    assert s_of[t][b] == ("s", k, j), ("read another S", s_of[t][b], k, j)
                    yield
                    if j and rnd.random() < 0.3:  # a row's maximum grew: O is rescaled
                        if j + 1 < nk:
                            yield from waits(sf[t][b ^ 1], (n + 1) >> 1, "s_rescale")
                        else:
                            yield from waits(od[t][0], n_o[0], "o_rescale")
                        assert o_of[t] == (k, j), "O rescaled before its products"
                    if j + 1 == max(n0, n1) and rnd.random() < 0.5:  # the last tile's V rows past the end
                        v = g0 + j
                        yield from waits(full[1][v % stages], v // stages)
                        assert held[1][v % stages] == v
                    s_of[t][b] = ("p", k, j)
                    pf[t][b].arrive(4)
                    yield
                    n += 1
                if nk:
                    for x in range(0 if nk >= 2 else 1, 2):
                        yield from waits(od[t][x], n_o[x], "o_done")
                        n_o[x] += 1
                    assert o_of[t] == (k, nk), "output read before its last product"
                    out[t][k] = nk
                    yield
                    o_read[t].add(k)
            g0 += max(n0, n1)

    run_agents([producer(0), producer(1), mma(0), mma(1), softmax(0), softmax(1)], pending, rnd)
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


@pytest.mark.parametrize("stages", [3, 4, 8])
@pytest.mark.parametrize("seed", range(150))
def test_prompt_protocol(seed, stages):
    rnd = random.Random(seed)
    prompt_cta(draw(rnd, rnd.choice([1, 2, 6])), stages, rnd)


@pytest.mark.parametrize("skip", ["q_empty", "k_empty", "v_empty", "p_full", "k_full", "v_full", "q_full", "s_full",
                                  "s_rescale", "o_rescale", "o_done", "lead"])
def test_a_wait_left_out_is_found(skip):
    for seed in range(200):
        rnd = random.Random(1000 + seed)
        try:
            prompt_cta(draw(rnd, rnd.choice([1, 2, 6])), rnd.choice([3, 4]), rnd, skip)
        except AssertionError:
            return
    assert False, "no schedule shows it"
