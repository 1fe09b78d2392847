"""Models of the latent-attention kernels' pipelines on the CPU: every role (TMA, product issuers, softmax and
correction warps) as a coroutine, every mbarrier with its arrival count, every buffer with the tile whose
contents it holds. Roles advance in random order, some much slower than others. A model fails where an arrival
or a wait by parity meets another phase than its own, where a buffer is read with other contents than meant or
written while it is still needed, and where nothing can advance."""

import os
import random
import re

import pytest

from sparse_attention_token_04_b200.build import CSRC


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self, phase):
        assert phase == self.phase, "an arrival counts for another phase"
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, phase):
        assert self.phase <= phase + 1, "a wait by parity takes a later phase for its own"
        return self.phase == phase + 1


class Ring:
    """Barriers used in turn: use n is phase n // len of barrier n % len."""

    def __init__(self, size, count):
        self.bars = [Barrier(count) for _ in range(size)]

    def arrive(self, n):
        self.bars[n % len(self.bars)].arrive(n // len(self.bars))

    def wait(self, n):
        while not self.bars[n % len(self.bars)].done(n // len(self.bars)):
            yield


def run(roles, rng):
    roles = list(roles)
    speed = {id(r): rng.choice([1, 1, 1, 0.3, 0.03]) for r in roles}
    steps = 0
    while roles:
        r = rng.choices(roles, [speed[id(x)] for x in roles])[0]
        try:
            next(r)
        except StopIteration:
            roles.remove(r)
        steps += 1
        assert steps < 400_000, "no progress"


def _code(file):
    with open(os.path.join(CSRC, file)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def decode_roles(segments, n_soft, stages, n_p, rng, lead=4, scores=3):
    """latent_decode_kernel of one CTA: `segments` key tiles of each of its requests."""
    tiles = [(s, i == 0, i == n - 1) for s, n in enumerate(segments) for i in range(n)]
    T = len(tiles)
    full, empty = Ring(stages, 1), Ring(stages, 1)
    q_full, s_full = Ring(1, 4), Ring(scores, 1)
    m_ready, p_ready = Ring(lead, n_soft), Ring(n_p, n_soft + 4)
    seg_ready, seg_done = Ring(1, n_soft), Ring(1, 4)
    ring, S = [None] * stages, [[None] * n_soft for _ in range(scores)]
    P, fac = [[None] * n_soft for _ in range(2)], [[None] * n_soft for _ in range(lead)]
    q, inv = [None] * 4, [None] * n_soft
    done = dict(corr=[-1] * 4, pv_start=-1, pv_end=-1, epilogue=[-1] * 4)

    def tma():
        for t in range(T):
            if t >= stages:
                yield from empty.wait(t - stages)
            ring[t % stages] = ("coming", t)
            yield
            ring[t % stages] = t
            full.arrive(t)

    def qk():
        for t, (seg, first, _) in enumerate(tiles):
            if first:
                yield from q_full.wait(seg)
            if t >= scores:
                yield from m_ready.wait(t - scores)
            yield from full.wait(t)
            for step in range(2):
                assert ring[t % stages] == t and q == [seg] * 4
                S[t % scores] = [("coming", t)] * n_soft
                if step == 0:
                    yield
            S[t % scores] = [t] * n_soft
            s_full.arrive(t)
            yield

    def pv():
        for t in range(T):
            yield from p_ready.wait(t)
            done["pv_start"] = t
            for step in range(2):
                assert ring[t % stages] == t and P[t & 1] == [t] * n_soft
                assert min(done["corr"]) >= t and (t == 0 or min(done["epilogue"]) >= tiles[t][0] - 1)
                if step == 0:
                    yield
            done["pv_end"] = t
            empty.arrive(t)
            yield

    def softmax(w):
        for t, (seg, _, last) in enumerate(tiles):
            yield from s_full.wait(t)
            assert S[t % scores][w] == t
            yield
            assert S[t % scores][w] == t
            fac[t % lead][w] = t
            m_ready.arrive(t)
            yield
            if t >= 2:
                yield from empty.wait(t - 2)
            P[t & 1][w] = t
            yield
            p_ready.arrive(t)
            yield
            if last:
                if seg > 0:
                    yield from seg_done.wait(seg - 1)
                inv[w] = seg
                yield
                seg_ready.arrive(seg)
                yield

    def correction(c):
        q[c] = 0
        yield
        q_full.arrive(0)
        for t, (seg, first, last) in enumerate(tiles):
            yield from m_ready.wait(t)
            assert fac[t % lead] == [t] * n_soft
            if not first and rng.random() < 0.3:              # O is rescaled
                yield from empty.wait(t - 1)
                assert done["pv_end"] == t - 1 == done["pv_start"]
                yield
                assert done["pv_start"] == t - 1 and fac[t % lead] == [t] * n_soft
            if last or rng.random() < 0.1:                    # rows of V are cleared
                yield from full.wait(t)
                assert ring[t % stages] == t and done["pv_start"] < t
                yield
            done["corr"][c] = t
            p_ready.arrive(t)
            yield
            if last:
                if t + 1 < T:
                    q[c] = seg + 1
                    yield
                    q_full.arrive(seg + 1)
                    yield
                yield from seg_ready.wait(seg)
                yield from empty.wait(t)
                for _ in range(2):
                    assert done["pv_end"] == t == done["pv_start"] and inv == [seg] * n_soft
                    yield
                done["epilogue"][c] = seg
                seg_done.arrive(seg)
                yield

    return [tma(), qk(), pv()] + [softmax(w) for w in range(n_soft)] + [correction(c) for c in range(4)]


def _decode_runs(n_p, runs, seed):
    rng = random.Random(seed)
    for _ in range(runs):
        segments = [rng.choice([1, 1, 2, 3, 7]) for _ in range(rng.choice([1, 2, 5]))]
        n_soft = rng.choice([1, 2, 4])
        run(decode_roles(segments, n_soft, 4 if n_soft == 4 else 5, n_p, rng), rng)


def test_decode_pipeline():
    code = _code("latent_decode.cu")
    # what the model takes from the kernel
    assert re.search(r"kLdScores = 3;", code) and re.search(r"kLdLead = 4;", code)
    assert "kStages = HT == 64 ? 4 : 5;" in code and "kSoft = HT / 16;" in code
    assert "mbar_init(&sm.p_ready[i], kSoft + 4);" in code and "m_ready[kLdLead], p_ready[kLdLead]" in code
    assert "mbar_init(&sm.q_full, 4);" in code and "mbar_init(&sm.seg_ready, kSoft);" in code
    assert "mbar_init(&sm.seg_done, 4);" in code and "mbar_init(&sm.m_ready[i], kSoft);" in code
    _decode_runs(4, 150, 1)


@pytest.mark.parametrize("n_p", [1, 2])
def test_decode_pipeline_with_fewer_barriers_fails(n_p):
    """A warp that drifts two tiles ahead of another meets its phase where two barriers alternate."""
    with pytest.raises(AssertionError):
        _decode_runs(n_p, 150, 1)


def prefill_roles(nt, rng, k_ring=4):
    """latent_prefill_kernel of one CTA: nt[w] key tiles of query tile w."""
    T = max(nt)
    both = nt[0] > 0 and nt[1] > 0
    q_full = [Ring(1, 1), Ring(1, 1)]
    k_full, k_free, v_full, v_free = Ring(k_ring, 1), Ring(k_ring, 1), Ring(2, 1), Ring(2, 1)
    s_full = [Ring(1, 1), Ring(1, 1)]
    p_ready = [[Ring(1, 4), Ring(1, 4)], [Ring(1, 4), Ring(1, 4)]]
    o_done = [Ring(1, 1), Ring(1, 1)]
    K, V = [None] * k_ring, [None] * 2
    SP = [[None] * 4, [None] * 4]                     # what a warp's lanes of S / P hold
    pv_start, pv_end = [-1, -1], [-1, -1]
    cleared = [set(), set()]

    def tma():
        loads = []
        for g in range(3 * T):
            j, c = divmod(g, 3)
            loads.append(("k", g))
            if g == 2:
                if nt[1] > 0:
                    loads.append(("q", 1))
                loads.append(("v", 0))
            elif g > 2 and c == 0:
                loads.append(("v", j))
        if nt[0] > 0:
            q_full[0].arrive(0)
        for kind, n in loads:
            if kind == "k":
                if n >= k_ring:
                    yield from k_free.wait(n - k_ring)
                K[n % k_ring] = None
                yield
                K[n % k_ring] = n
                k_full.arrive(n)
            elif kind == "v":
                if n >= 2:
                    yield from v_free.wait(n - 2)
                V[n & 1] = None
                yield
                V[n & 1] = n
                v_full.arrive(n)
            else:
                q_full[n].arrive(0)
            yield

    def mma():
        # the tensor pipe runs in issue order: each piece of work is done before the next one starts
        def qk(w, j, first, last):
            for c in range(3):
                g = 3 * j + c
                if first:
                    yield from k_full.wait(g)
                assert K[g % k_ring] == g
                SP[w] = [("coming", j)] * 4
                yield
                assert K[g % k_ring] == g
                if last:
                    k_free.arrive(g)
            SP[w] = [("s", j)] * 4
            s_full[w].arrive(j)
            yield

        def pv(w, j):
            for half in range(2):
                yield from p_ready[w][half].wait(j)
                pv_start[w] = j
                for _ in range(2):
                    assert V[j & 1] == j and all(x[0] == "p" and x[1] == j and x[2] >= half for x in SP[w])
                    assert j != T - 1 or len(cleared[w]) == 4
                    yield
            pv_end[w] = j

        for w in range(2):
            if nt[w]:
                yield from q_full[w].wait(0)
                yield from qk(w, 0, w == 0 or not both, w == 1 or not both)
        for j in range(T):
            yield from v_full.wait(j)
            two, two_next = j < nt[0] and j < nt[1], j + 1 < nt[0] and j + 1 < nt[1]
            for w in range(2):
                if j < nt[w]:
                    yield from pv(w, j)
                    o_done[w].arrive(j)
                    if w == 1 or not two:
                        v_free.arrive(j)
                if j + 1 < nt[w]:
                    yield from qk(w, j + 1, w == 0 or not two_next, w == 1 or not two_next)

    def softmax(w, c):
        for j in range(nt[w]):
            yield from s_full[w].wait(j)
            assert SP[w][c] == ("s", j)
            yield
            assert SP[w][c] == ("s", j)
            if j > 0 and rng.random() < 0.3:          # O is rescaled
                yield from o_done[w].wait(j - 1)
                assert pv_end[w] == j - 1
                yield
                assert pv_start[w] == j - 1
            if j == T - 1:                            # rows of V are cleared
                yield from v_full.wait(j)
                assert V[j & 1] == j and pv_start[w] < j
                cleared[w].add(c)
                yield
            for half in range(2):
                SP[w][c] = ("p", j, half)
                yield
                p_ready[w][half].arrive(j)
                yield
        if nt[w]:
            yield from o_done[w].wait(nt[w] - 1)
            assert pv_end[w] == nt[w] - 1

    return [tma(), mma()] + [softmax(w, c) for w in range(2) for c in range(4)]


def test_prefill_pipeline():
    code = _code("latent_prefill.cu")
    assert "kLpKRing = 4;" in code and "mbar_init(&sm.p_ready[i][0], 4);" in code and "mbar_init(&sm.p_ready[i][1], 4);" in code
    rng = random.Random(2)
    for _ in range(120):
        n = rng.choice([1, 1, 2, 3, 6, 9])
        # causal: the second tile of queries sees as many key tiles as the first or one more; either may be empty
        nt = rng.choice([[n, n], [n, n + 1], [n, 0], [0, n]])
        run(prefill_roles(nt, rng), rng)
