"""The joins of split attention calls are programmatic dependents of the kernel in front of them: what follows
a join on the stream waits for the join only, so every CTA of it has to wait for that kernel before it exits
(read in the sources, no GPU)."""

import os
import re

import pytest

from sparse_attention_token_04_b200.build import CSRC


def _kernel_body(source: str, name: str) -> str:
    """Text between the braces of kernel `name`."""
    at = re.search(rf"__global__[^;{{]*\b{name}\(", source)
    assert at, name
    start = source.index("{", at.end())
    depth = 0
    for i in range(start, len(source)):
        depth += {"{": 1, "}": -1}.get(source[i], 0)
        if depth == 0:
            return source[start:i]
    raise AssertionError(name)


@pytest.mark.parametrize("file,kernel", [("latent_decode.cu", "latent_combine_kernel"),
                                         ("latent_prefill.cu", "latent_prefill_combine_kernel")])
def test_joins_wait_before_any_of_their_ctas_exits(file, kernel):
    with open(os.path.join(CSRC, file)) as f:
        body = re.sub(r"//[^\n]*", "", _kernel_body(f.read(), kernel))
    assert body.count("grid_dependency_wait();") == 1
    before = body[:body.index("grid_dependency_wait();")]
    assert not re.search(r"\breturn\s*;", before)
    assert before.count("{") == before.count("}") + 1      # not inside a branch or a loop
