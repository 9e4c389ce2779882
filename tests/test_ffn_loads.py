"""The product kernel and the kernel that joins its parts may become resident while the kernel
before them in the stream still writes what they read (launch_after, await_before): nothing
there goes through the read-only path, whose loads a compiler may move in front of the wait.
Read from the source, without a GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "non_linear_matrix_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_products_read_nothing_as_constant():
    text = source("m2rnn_gemm.cuh")
    assert "__ldg" not in text and ".nc." not in text
    assert not re.search(r"\bload_vec<", text)  # (through the read-only path)
    loads = re.findall(r"raw_load<([^>]*)>", text)
    assert loads and all(args.split(",")[-1].strip() == "false" for args in loads)


def test_kernels_that_wait_read_nothing_before():
    """await_before comes first in what is launched by launch_after (or with its attribute)."""
    text = source("m2rnn_gemm.cuh")
    join = text[text.index("join_parts_kernel(const"):]
    assert join.index("await_before") < join.index("p.parts")
    kernel = text[text.index("gemm_kernel(const"):text.index("join_parts_kernel(const")]
    first_use = min(kernel.index(s) for s in ("issue_tile<", "block_load(", "finish_bf16<", "prefetch_map("))
    assert kernel.index("await_before") < first_use
