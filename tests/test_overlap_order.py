"""Kernels that may start beside the caller's previous kernel wait for it
before they touch device memory (read from the sources: no GPU needed)."""
import os
import re

import pytest

from speculative_decoding_drafting_gb300 import _build

# first kernels of an entry point that are launched with the overlap
KERNELS = [("attn_paged.cu", "attn_paged_kernel"), ("attn_prompt.cu", "attn_prompt_kernel")]

# what reads or writes device memory there: the workspace's header and status,
# the requests, lists, descriptors and results
DEVICE = re.compile(r"ws_wait_limit|ws_test_withhold|raise_status|check_requests|row_range|pairs_of|entry_of|get_item|"
                    r"load4|load16|plan_request|tma_load|cp_async|__ld\w+\(|p\.(ws|desc|part|out|lse|list|count)\b")


def _body(name, kernel):
    with open(os.path.join(_build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = re.search(r"__global__[^;{]*\b" + kernel + r"\(", text).end()
    at = text.index("{", at)
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            return text[at:end]
        end += 1


@pytest.mark.parametrize("name,kernel", KERNELS)
def test_nothing_is_touched_before_the_wait(name, kernel):
    body = _body(name, kernel)
    assert body.count("pdl_wait()") == 1
    before, after = body.split("pdl_wait()")
    assert not DEVICE.findall(before)
    assert "ws_wait_limit(p.ws)" in after
