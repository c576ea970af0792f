"""The norm-and-rotate, append and chunk attention calls among torch's other operations and Python's
other threads: versions of tensors written in place, calls that wait for the device."""
import threading
import time

import pytest
import torch

import tiled_exact_attention_forward_b200 as fa
from gpu_helpers import requires_cuda
from paged_helpers import paged_cache, rope_table

pytestmark = [pytest.mark.gpu, requires_cuda]

BF16 = torch.bfloat16


def small_cache():
    """(q, k, v, kpool, vpool, block_table, seqlens, cu_tokens) of two sequences, seven new tokens."""
    kp, vp, table, cu, lens = paged_cache([2, 5], [20, 33], 2, 16, BF16, seed=40, pad=0.0)
    x = torch.randn(7, 8, 128, generator=torch.Generator().manual_seed(41)).to(BF16).cuda()
    return x[:, :4].clone(), x[:, 4:6].clone(), x[:, 6:].clone(), *(t.cuda() for t in (kp, vp, table, lens, cu))


def test_an_overwritten_tensor_is_missed_by_the_backward_that_saved_it():
    leaf = torch.randn(1, 2, 8, 64, device="cuda").requires_grad_()
    x = leaf * 2.0
    y = x.square().sum()
    x = x.detach()
    fa.norm_rope(x, q_out=x)
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.backward()


def test_versions_of_what_a_call_writes():
    q, k, v, kp, vp, table, lens, cu = small_cache()
    rope = rope_table(40, 128).cuda()
    out, lse = torch.empty(7, 4, 128, dtype=BF16, device="cuda"), torch.empty(7, 4, device="cuda")
    calls = [
        (lambda: fa.norm_rope(q, k, q_out=out, k_out=k), [out, k], [q]),
        (lambda: fa.norm_rope(q, k), [], [q, k]),
        (lambda: fa.append_paged(k, v, kp, vp, table, lens, cu, rope, q, q_out=out), [kp, vp, out], [v, table, lens, cu]),
        (lambda: fa.append_paged(k, v, kp[:], vp[:], table, lens, cu), [kp, vp], [v]),
        (lambda: fa.extend_paged(q, kp, vp, table, lens, cu, out=out, lse=lse), [out, lse], [q, kp, vp]),
    ]
    for call, writes, reads in calls:
        before = [t._version for t in writes], [t._version for t in reads]
        call()
        assert all(t._version > a for t, a in zip(writes, before[0]))
        assert all(t._version == a for t, a in zip(reads, before[1]))


def test_inference_tensors_have_no_version():
    with torch.inference_mode():
        q, k, v, kp, vp, table, lens, cu = small_cache()
        want = fa.norm_rope(q)
        assert torch.equal(fa.norm_rope(q, q_out=q), want)
        fa.append_paged(k, v, kp, vp, table, lens, cu)
        assert torch.equal(fa.extend_paged(q, kp, vp, table, lens, cu, out=torch.empty_like(q))[0],
                           fa.extend_paged(q, kp, vp, table, lens, cu)[0])
    assert fa.device_status() == fa.FA_OK


@pytest.mark.parametrize("which", ["norm_rope", "norm_rope_backward", "append_paged", "extend_paged"])
def test_other_threads_run_while_a_launch_waits(which):
    """The device is busy for about a second and its queue of launches fills up: a call then waits in the
    driver, and another thread goes on meanwhile (it sleeps a millisecond a turn)."""
    q, k, v, kp, vp, table, lens, cu = small_cache()
    g, w = torch.ones_like(q), torch.ones(128, dtype=BF16, device="cuda")
    call = {"norm_rope": lambda: fa.norm_rope(q),
            "norm_rope_backward": lambda: fa.norm_rope_backward(q, None, g, None, w),
            "append_paged": lambda: fa.append_paged(k, v, kp, vp, table, lens, cu),
            "extend_paged": lambda: fa.extend_paged(q, kp, vp, table, lens, cu)}[which]
    call()
    torch.cuda.synchronize()
    turns, done = [], threading.Event()

    def tick():
        while not done.is_set():
            time.sleep(0.001)
            turns.append(time.perf_counter())

    t = threading.Thread(target=tick)
    t.start()
    torch.cuda._sleep(2_000_000_000)
    begin = time.perf_counter()
    for _ in range(1500):
        call()
    took = time.perf_counter() - begin
    torch.cuda.synchronize()
    done.set()
    t.join()
    assert took > 0.4, "the queue did not fill up"
    during = [x for x in turns if begin <= x <= begin + took]
    assert len(during) > 100
    assert max(b - a for a, b in zip(during, during[1:])) < 0.25
