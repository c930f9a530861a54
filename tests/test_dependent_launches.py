"""Kernels that are launched while the one before still runs (launch_after) wait
before they touch memory, and read what it wrote by plain loads: loads through
the read-only path are promised memory that nothing writes from the kernel's launch
on, and may be moved ahead of the wait. Read from the sources; no GPU shows it
reliably."""
import re

import pytest

from quantized_lora_merge_b200.build import CSRC

DEPENDENT = {"embedding_kernels.cu": ["embedding_join_first_kernel", "embedding_join_runs_kernel",
                                      "embedding_chunks_kernel", "embedding_touched_kernel"],
             "layer_norm_backward_kernels.cu": ["layer_norm_reduce_kernel"],
             "grad_norm_kernels.cu": ["grad_norm_finish_kernel", "grad_clip_kernel"]}


def _body(text, kernel):
    """From the kernel's name in its definition to the brace that closes it."""
    at = re.search(r"__global__[^;{]*\b" + kernel + r"\(", text).end()
    begin = text.index("{", at)
    depth = 0
    for k in range(begin, len(text)):
        depth += {"{": 1, "}": -1}.get(text[k], 0)
        if depth == 0:
            return text[begin:k]
    raise AssertionError(kernel)


@pytest.mark.parametrize("file", sorted(DEPENDENT))
def test_every_dependent_kernel_is_listed_and_waits(file):
    text = (CSRC / file).read_text()
    launched = set(re.findall(r"launch_after\(\s*(\w+)", text)) - {"kernel"} | set(re.findall(r"launch\((\w+_kernel)", text))
    assert launched == set(DEPENDENT[file])
    for kernel in DEPENDENT[file]:
        body = _body(text, kernel)
        before = body[:body.index("wait_for_previous();")]
        # declarations and index arithmetic alone: no parameter that points to memory is used
        assert not re.search(r"\b(norm|partial|key|pos|key_out|pos_out|dweight|dbias)\b|load_elem|__ldg",
                             before), kernel


def test_lists_and_partial_sums_are_read_by_plain_loads():
    text = (CSRC / "embedding_kernels.cu").read_text()
    written = [m for m in re.findall(r"__ldg\(([^;]*);", text) if re.search(r"\b(key|pos|partial)\b", m)]
    assert not written
    # rows of fp32 single columns: dy, or the chunks' sums
    load = text[text.index("struct RawStrip"):text.index("void add_to(S& s)")]
    assert not re.search(r"__ldg\(static_cast<const uint32_t\*>", load)
