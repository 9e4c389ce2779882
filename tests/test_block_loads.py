"""Which loads of the block operators may take the read-only path
(``ld.global.nc``): memory that nobody writes while the kernel is resident.  A
kernel that ``await_before`` holds back is resident while the kernels before it
still write, and a state that is updated in place is written by its own kernel:
there the compiler must not be told that the memory is constant (it may move
such loads in front of the wait, or behind a store), whatever the results look
like with one compiler.  Read from the source, without a GPU; the GPU tests
below check the bits where such memory is used again at once."""
import os
import re

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "non_linear_matrix_gb300", "csrc")


def body(file, name):
    """The text from the definition of ``name`` to its closing brace, comments
    left out."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    start = re.search(rf"\b{name}\([^;{{]*\)\s*(?:const\s*)?{{", text)
    assert start, name
    depth = 0
    for i in range(start.end() - 1, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start.start():i + 1]
    raise AssertionError(name)


@pytest.mark.parametrize("file,name", [
    ("m2rnn_scan.cuh", "state_load"),         # states and decays of the kernels before
    ("m2rnn_scan_states.cu", "join_kernel"),  # segments' ends and decays
    ("m2rnn_scan_bwd.cu", "add_shares_kernel"),
    ("m2rnn_vec.cuh", "sum_parts_kernel"),
    ("m2rnn_scan_step.cu", "scan_step_kernel"),
    ("m2rnn_conv.cu", "conv_step_kernel"),
])
def test_written_memory_is_not_read_as_constant(file, name):
    text = body(file, name)
    assert "__ldg" not in text and ".nc." not in text
    if name == "conv_step_kernel":  # the state may be state_out
        assert re.findall(r"row_of<([^>]*)>", text) == ["F32, VEC, W, false"]


def rn(seed, *s, dtype=torch.bfloat16):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_step_in_place(m, W, dtype):
    """A run of tokens with the state in place and between two buffers: the
    same bits."""
    B, C = 37, 136
    w, x = rn(1, C, W, dtype=dtype), rn(2, 50, B, C, dtype=dtype)
    apart, here = rn(3, B, W - 1, C, dtype=dtype), rn(3, B, W - 1, C, dtype=dtype)
    for t in range(50):
        y, apart = m.conv_step(x[t], w, apart)
        y2, same = m.conv_step(x[t], w, here, state_out=here)
        assert same is here and torch.equal(y, y2) and torch.equal(apart, here)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [700, 130, 64])  # segments, one segment, one chunk
def test_scan_workspace_used_again_at_once(m, T, dtype):
    """Calls on different inputs through the same scratch, back to back: the
    bits of calls with scratch of their own."""
    B, N, K, V = 2, 4, 64, 16
    par = [rn(s, N, dtype=dtype) for s in (1, 2)]
    ins, own = [], []
    for i in range(6):
        q, k = rn(10 + i, B, T, 1, K, dtype=dtype) * 0.1, rn(20 + i, B, T, 1, K, dtype=dtype)
        ins.append((q, k, rn(30 + i, B, T, N, V, dtype=dtype), rn(40 + i, B, T, N, dtype=dtype)))
    dy = rn(3, B, T, N, V, dtype=dtype)
    ws = [torch.empty(32 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for x in ins:
        own.append((*m.scan_fwd(*x, *par)[:2], m.scan_bwd(*x, *par, dy)))
        torch.cuda.synchronize()
    got = [(*m.scan_fwd(*x, *par, workspace=ws[0])[:2], m.scan_bwd(*x, *par, dy, workspace=ws[1]))
           for x in ins]
    for (y, H, g), (y2, H2, g2) in zip(own, got):
        assert torch.equal(y, y2) and torch.equal(H, H2)
        assert all(torch.equal(t, g2[n]) for n, t in g.items() if t is not None)
