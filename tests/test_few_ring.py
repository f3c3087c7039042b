"""The expert kernel's ring, read from its source: what a run on the GPU cannot show.

Token rows come into a stage by cp.async (generic proxy), weights by bulk copies
(async proxy).  Where a stage's next weights may lie over its token rows, a barrier
does not order the two; the side that gives the stage back issues a proxy fence."""

import os
import re

import pytest

import sparse_mixture_experts_22_b200 as M

SOURCE = os.path.join(os.path.dirname(M.__file__), "csrc", "few.cu")


def body(text, head):
    """The braces' text after the first match of head."""
    at = text.index("{", re.search(head, text).end())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(head)


def test_fence_between_token_rows_and_weights():
    text = open(SOURCE).read()
    assert "fence.proxy.async.shared::cta" in body(text, r"void fence_proxy_async\(\)")
    done = body(text, r"template <bool FENCE>\s+__device__ __forceinline__ void done\(\)")
    fence, arrive = done.index("if (FENCE) fence_proxy_async();"), done.index("mbar_arrive(&empty")
    assert fence < arrive
    up = body(text, r"void up_q4\(Consumer& c")
    assert re.findall(r"c\.done<(\w+)>\(\)", up) == ["true"]
    # nothing else gives a stage back
    assert text.count("mbar_arrive(&empty") == 1


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("blocks", [1, 2])
def test_where_the_fence_is_needed(group, blocks):
    """Bytes of a 4-bit stage: where token rows begin, and how far eight panels of the
    second half reach (layout of few.h); bf16 stages end below by a static assertion."""
    rows_begin = 4 * blocks * (4096 + 128 * (128 // group))
    groups = 8 if group == 32 else 8 * 32 // group + 1
    reach = 2 * 8 * 2048 + 2 * groups * 256
    assert (reach > rows_begin) == (blocks == 1 or group != 32)
