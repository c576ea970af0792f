"""Calls from a thread that has not touched the CUDA runtime (as autograd's workers may not have)."""
import threading

import pytest
import torch

import tiled_exact_attention_forward_b200 as fa
import workloads
from gpu_helpers import requires_cuda
from paged_helpers import paged_cache, rope_table

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


def paged_inputs():
    """A small cache and its calls' arguments, outputs and workspace: nothing is left for torch to allocate."""
    kp, vp, table, cu, lens = paged_cache([2, 40], [100, 300], 2, 16, torch.bfloat16, seed=3)
    x = torch.randn(42, 8, 128, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    dev = [t.cuda() for t in (kp, vp, table, lens, cu)]
    out = torch.empty(42, 4, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(42, 4, device="cuda")
    ws = torch.empty(fa.extend_paged_workspace_size(42, 4, 2, 128), dtype=torch.uint8, device="cuda")
    return x[:, :4], x[:, 4:6], x[:, 6:], dev, out, lse, ws


@pytest.mark.parametrize("which", ["norm_rope", "append_paged", "extend_paged"])
def test_paged_operators_from_a_new_thread(which):
    q, k, v, (kp, vp, table, lens, cu), out, lse, ws = paged_inputs()
    rope = rope_table(300, 128).cuda()

    def call():
        if which == "norm_rope":
            fa.norm_rope(q, rope=rope, q_out=out)
        elif which == "append_paged":
            fa.append_paged(k, v, kp, vp, table, lens, cu, rope, q, q_out=out)
        else:
            fa.extend_paged(q, kp, vp, table, lens, cu, workspace=ws, out=out, lse=lse)
        return [t.clone().nan_to_num(9.0) for t in (out, lse, kp, vp)]

    lse.zero_()
    torch.cuda.synchronize()
    got = in_new_thread(call)
    torch.cuda.synchronize()
    out.zero_()
    assert all(torch.equal(a, b) for a, b in zip(got, call()))
    assert fa.device_status() == fa.FA_OK


def test_rotated_autograd_without_a_torch_kernel_before_the_backward():
    q, k, v, do = workloads.forward_inputs(1, 2, 300, 128, torch.bfloat16, seed=5, device="cuda", with_dout=True)
    leaves = [t.requires_grad_() for t in (q, k, torch.ones(128, dtype=q.dtype, device="cuda"))]
    rope = rope_table(300, 128).cuda()
    y = fa.qk_norm_rope(leaves[0], leaves[1], leaves[2], rope=rope)
    torch.autograd.backward(y, (do, v))
    torch.cuda.synchronize()
    want = fa.norm_rope_backward(q.detach(), k.detach(), do, v, leaves[2].detach(), rope=rope)
    assert all(torch.equal(t.grad, w) for t, w in zip(leaves, want))


def test_two_threads_at_once():
    """Calls of two threads, each on a stream of its own, give what they give alone."""
    ins = [paged_inputs() for _ in range(2)]
    ins[1][0].mul_(0.5)
    want = [fa.extend_paged(q, kp, vp, table, lens, cu) for q, _, _, (kp, vp, table, lens, cu), *_ in ins]
    torch.cuda.synchronize()
    got = [[], []]

    def run(i):
        q, _, _, (kp, vp, table, lens, cu), *_ = ins[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got[i].append(fa.extend_paged(q, kp, vp, table, lens, cu))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in (0, 1):
        assert len(got[i]) == 50 and all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))
    assert fa.device_status() == fa.FA_OK
