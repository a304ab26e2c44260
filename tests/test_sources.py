"""Properties of the kernel sources that no run can show."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_nf4_quantized_dq_b200", "csrc")


def kernels():
    """(name, parameters, body) of every __global__ function."""
    for f in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        for part in text.split("__global__")[1:]:
            m = re.search(r"(\w+)\s*\(((?:[^(){}]|\([^(){}]*\))*)\)\s*\{", part)
            if m:
                depth, end = 1, m.end()
                while depth and end < len(part):
                    depth += {"{": 1, "}": -1}.get(part[end], 0)
                    end += 1
                yield m.group(1), m.group(2), part[m.end():end]


def test_kernels_that_start_before_their_inputs_are_written_make_no_promise_about_them():
    """A kernel launched on the heels of the one before it waits for that grid's results.  A parameter of
    const __restrict__ type promises memory that never changes while the kernel runs, which lets the
    compiler load it ahead of the wait."""
    found = {name: params for name, params, body in kernels() if "griddepcontrol.wait" in body}
    assert {"column_sum_bf16_kernel", "dq_mean_groups_kernel", "few_token_join_kernel", "few_token_kernel",
            "few_token_ragged_kernel"} <= set(found)
    for name, params in found.items():
        assert "__restrict__" not in params, name
