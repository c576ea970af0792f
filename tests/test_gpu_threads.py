"""Calls from a thread that has not touched the CUDA runtime (as autograd's workers may not have)."""
import threading

import pytest
import torch

import tiled_exact_attention_forward_b200 as fa
import workloads
from gpu_helpers import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


def in_new_thread(f):
    got = []

    def run():
        try:
            got.append(f())
        except Exception as e:  # handed to the caller
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


def test_forward_from_a_new_thread():
    q, k, v = workloads.forward_inputs(1, 2, 300, 128, torch.bfloat16, seed=1, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(1, 2, 300, device="cuda")
    torch.cuda.synchronize()
    in_new_thread(lambda: fa.forward(q, k, v, causal=True, out=o, lse=lse))
    torch.cuda.synchronize()
    assert torch.equal(o, fa.forward(q, k, v, causal=True)[0])


def test_autograd_without_a_torch_kernel_before_the_backward():
    q, k, v, do = workloads.forward_inputs(1, 2, 300, 128, torch.bfloat16, seed=2, device="cuda", with_dout=True)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    fa.attention(*leaves, causal=True).backward(do)
    torch.cuda.synchronize()
    assert all(torch.isfinite(t.grad).all() and t.grad.any() for t in leaves)
