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
