"""Orderings between the threads of the latent-attention kernels that no run shows reliably, read in the
sources (no GPU)."""

import os
import re

from sparse_attention_token_04_b200.build import CSRC


def _code(file: str) -> str:
    with open(os.path.join(CSRC, file)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_scores_are_fenced_before_their_buffer_is_released():
    """latent_decode: the softmax's arrival at m_ready lets the QK issuer overwrite the scores that have just
    been read from TMEM, so a tcgen05 fence stands in front of it, behind that read."""
    code = _code("latent_decode.cu")
    arrivals = [m.start() for m in re.finditer(r"mbar_arrive\(&sm\.m_ready\[", code)]
    assert arrivals
    for at in arrivals:
        read = code.rindex("tmem_wait_ld_regs(s", 0, at)
        assert "tc_fence_before();" in code[read:at]


def test_a_warps_wait_orders_the_memory_of_all_its_lanes():
    """Where one lane waits on a barrier for its warp, the others learn of it by a shuffle, which orders no
    memory: a warp barrier follows. And no lane's test of a barrier stands for the warp's."""
    code = _code("common.cuh")
    at = code.index("bool mbar_wait_warp(")
    body = code[at:code.index("\n}\n", at)]
    assert "__syncwarp();" in body[body.rindex("__shfl_sync("):]
    for file in ("latent_decode.cu", "latent_prefill.cu"):
        for test in re.finditer(r"[^\n]*mbar_test\([^\n]*", _code(file)):
            assert "__all_sync(" in test.group(), (file, test.group())


class _Barrier:
    """An mbarrier whose arrivals and waits name the phase that they mean."""

    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self, phase):
        assert phase == self.phase, "an arrival counts for another tile's phase"
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, phase):
        assert self.phase <= phase + 1, "a wait by parity takes a later phase for its own"
        return self.phase == phase + 1


def _decode_pipeline(tiles, n_soft, n_stages, n_p, rng):
    """The hand-overs of latent_decode between its warps (one segment), in a random order of steps in which
    some warps are much slower than others: raises where an arrival or a wait meets another tile's phase."""
    lead, scores = 4, 3
    s_full = [_Barrier(1) for _ in range(scores)]
    m_ready = [_Barrier(n_soft) for _ in range(lead)]
    p_ready = [_Barrier(n_soft + 4) for _ in range(n_p)]
    empty = [_Barrier(1) for _ in range(n_stages)]
    of = lambda bars, t: (bars[t % len(bars)], t // len(bars))

    def wait(bars, t):
        bar, phase = of(bars, t)
        while not bar.done(phase):
            yield

    def arrive(bars, t):
        bar, phase = of(bars, t)
        bar.arrive(phase)

    def qk():
        for t in range(tiles):
            if t >= n_stages:
                yield from wait(empty, t - n_stages)     # the TMA's wait for the tile's place
            if t >= scores:
                yield from wait(m_ready, t - scores)
            arrive(s_full, t)
            yield

    def pv():
        for t in range(tiles):
            yield from wait(p_ready, t)
            yield
            arrive(empty, t)

    def softmax():
        for t in range(tiles):
            yield from wait(s_full, t)
            yield
            arrive(m_ready, t)
            yield
            if t >= 2:
                yield from wait(empty, t - 2)
            arrive(p_ready, t)
            yield

    def correction():
        for t in range(tiles):
            yield from wait(m_ready, t)
            yield
            arrive(p_ready, t)
            yield

    roles = [qk(), pv()] + [softmax() for _ in range(n_soft)] + [correction() for _ in range(4)]
    speed = {id(r): rng.choice([1, 1, 1, 0.05]) for r in roles}
    idle = 0
    while roles:
        r = rng.choices(roles, [speed[id(x)] for x in roles])[0]
        try:
            next(r)
        except StopIteration:
            roles.remove(r)
        idle += 1
        assert idle < 200_000, "no progress"


def test_decode_arrivals_meet_their_own_tiles_phase():
    """The decode kernel's barriers, as many as it has of each: no warp's arrival counts for another tile,
    however far the warps drift apart. (With two p_ready barriers it does, which the model shows.)"""
    import random

    code = _code("latent_decode.cu")
    lead = int(re.search(r"kLdLead = (\d+);", code).group(1))
    declared = re.search(r"p_ready\[(\w+)\]", code).group(1)
    n_p = lead if declared == "kLdLead" else int(declared)
    assert lead == 4 and int(re.search(r"kLdScores = (\d+);", code).group(1)) == 3
    uses = re.findall(r"p_ready\[([^\]]*)\]", code)[1:]
    assert all(u in ("i", "t % kLdLead", "done % kLdLead") for u in uses), uses
    rng = random.Random(1)

    def run(n):
        for _ in range(40):
            _decode_pipeline(24, rng.choice([1, 2, 4]), rng.choice([4, 5]), n, rng)

    run(n_p)
    try:
        run(2)
    except AssertionError as e:
        assert "another tile" in str(e) or "later phase" in str(e)
    else:
        raise AssertionError("the model misses the drift of two barriers")
