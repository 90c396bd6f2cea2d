"""The order in which the kernels that hold tensor memory wait, allocate and let their dependents
start, read from their sources (no GPU).

An allocation waits for columns without a limit.  A CTA that held columns while it waited for the
kernel before it could keep them from a CTA of that kernel, and a dependent that starts before this
kernel has its own columns could take them: both would wait for good.  So: the dependency wait, the
allocation, a barrier of the CTA, and only then the dependents.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_attention_stief_b200", "csrc")


def _body(name, kernel):
    """The kernel's body in the file, without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    at = text.index("{", re.search(kernel + r"\(const __grid_constant__", text).start())
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
        if depth == 0:
            return text[at:end]


@pytest.mark.parametrize("name,kernel", [("shared_decode.cu", "stief_shared_decode_kernel"),
                                         ("shared_expand.cu", "stief_shared_expand_kernel"),
                                         ("prefill_attention.cu", "stief_prefill_kernel"),
                                         ("prefill_one_tile.cu", "stief_prefill_one_tile_kernel")])
def test_wait_then_allocate_then_let_dependents_start(name, kernel):
    body = _body(name, kernel)
    wait, alloc = body.index("pdl_wait();"), [m.start() for m in re.finditer(r"tmem_alloc(?:_pair)?\(", body)]
    starts = [m.start() for m in re.finditer(r"pdl_launch_dependents\(\);", body)]
    assert len(alloc) == 1 and starts and wait < alloc[0]
    for at in starts:
        assert alloc[0] < at
        assert re.search(r"__syncthreads\(\);|cluster_sync\(\);", body[alloc[0]:at])
