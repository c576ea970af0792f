"""The norm-and-rotate, append and chunk attention calls among torch's other operations and Python's
other threads: given outputs, versions of tensors written in place, frozen inputs of the differentiable form, calls
that wait for the device."""
import itertools
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


def test_given_outputs_at_their_strides():
    """Outputs into parts of larger tensors, in another order of dimensions, and onto the inputs where a
    fused projection left them: the same bits, and nothing beside them is touched."""
    gen = torch.Generator().manual_seed(44)
    x = torch.randn(2, 30, 10, 128, generator=gen).to(BF16).cuda()   # [B, N, Hq + Hk + 2, d]
    rope, w = rope_table(30, 64).cuda(), 1 + 0.3 * torch.randn(128, generator=gen).to(BF16).cuda()
    q, k = x[:, :, 1:6].transpose(1, 2), x[:, :, 6:8].transpose(1, 2)
    want = fa.norm_rope(q, k, w, None, rope)
    wide = torch.full((2, 30, 10, 128), 7.0, dtype=BF16, device="cuda")
    got = fa.norm_rope(q, k, w, None, rope, q_out=wide[:, :, 1:6].transpose(1, 2), k_out=wide[:, :, 6:8].transpose(1, 2))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (wide[:, :, 0] == 7.0).all() and (wide[:, :, 8:] == 7.0).all()
    before = x.clone()
    got = fa.norm_rope(q, k, w, None, rope, q_out=q, k_out=k)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(x[:, :, 0], before[:, :, 0]) and torch.equal(x[:, :, 8:], before[:, :, 8:])


def test_queries_turned_where_they_lie_and_pools_inside_larger_ones():
    q, k, v, kp, vp, table, lens, cu = small_cache()
    rope = rope_table(40, 128).cuda()
    big = [torch.cat([p[:1], p, p[:1]]) for p in (kp, vp)]
    edges = [(p[0].clone(), p[-1].clone()) for p in big]
    want = fa.append_paged(k, v, kp, vp, table, lens, cu, rope, q)
    o, lse = fa.extend_paged(want, kp, vp, table, lens, cu)
    fa.append_paged(k, v, big[0][1:-1], big[1][1:-1], table, lens, cu, rope, q, q_out=q)
    assert torch.equal(q, want)
    for p, small, (a, b) in zip(big, (kp, vp), edges):
        assert torch.equal(p[1:-1], small) and torch.equal(p[0], a) and torch.equal(p[-1], b)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = fa.extend_paged(q, big[0][1:-1], big[1][1:-1], table, lens, cu)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    assert fa.device_status() == fa.FA_OK


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


def allocations(f):
    """(f's result, how many blocks of device memory it asked for)."""
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    r = f()
    return r, torch.cuda.memory_stats()["allocation.all.allocated"] - before


@pytest.mark.parametrize("trains", [t for t in itertools.product([False, True], repeat=4) if any(t)])
def test_frozen_inputs_cost_nothing(trains):
    """Gradients of the inputs that train are norm_rope_backward's; a frozen side is not computed, a
    frozen weight's gradient not summed."""
    gen = torch.Generator().manual_seed(42)
    q, gq = (torch.randn(2, 4, 30, 64, generator=gen).to(BF16).cuda() for _ in range(2))
    k, gk = (torch.randn(2, 2, 30, 64, generator=gen).to(BF16).cuda() for _ in range(2))
    qw, kw = (1 + 0.3 * torch.randn(64, generator=gen).to(BF16).cuda() for _ in range(2))
    rope = rope_table(30, 64).cuda()
    want = fa.norm_rope_backward(q, k, gq, gk, qw, kw, rope)
    ins = [t.clone().requires_grad_(r) for t, r in zip((q, k, qw, kw), trains)]
    y = fa.qk_norm_rope(*ins, rope=rope)
    leaves = [t for t in ins if t.requires_grad]
    got, blocks = allocations(lambda: torch.autograd.grad(y, leaves, (gq, gk)))
    for g, w in zip(got, [w for w, r in zip(want, trains) if r]):
        if g.dim() == 4:
            assert torch.equal(g, w)
        else:  # one side alone is summed in another order: the rounding to bf16 may be the next one
            assert ((g.float() - w.float()).abs() <= torch.finfo(BF16).eps * w.float().abs()).all()
    sides = [s for s in (0, 1) if trains[s] or trains[2 + s]]
    sums = trains[2] + trains[3]
    assert blocks == len(sides) + sums + (sums > 0)  # rows' gradients, weights', the sums' workspace


@pytest.mark.parametrize("eps", [1e-6, None])
@pytest.mark.parametrize("with_k", [False, True])
def test_a_table_that_wants_a_gradient_gets_none(eps, with_k):
    """Frozen rows under a rotation table that is a parameter: the backward runs and leaves it without one."""
    q = torch.randn(1, 2, 8, 64, device="cuda")
    rope = rope_table(8, 64).cuda().requires_grad_()
    y = fa.qk_norm_rope(q, q if with_k else None, rope=rope, eps=eps)
    sum(t.sum() for t in (y if with_k else (y,))).backward()
    assert rope.grad is None


@pytest.mark.parametrize("layout", ["projection", "slice", "expanded"])
@pytest.mark.parametrize("frozen", [None, 0, 1])
def test_rotation_alone_does_not_keep_its_rows(layout, frozen):
    """Without the norm the inputs can be freed before the backward, whose gradients are laid out as if
    they were there."""
    gen = torch.Generator().manual_seed(43)
    rope = rope_table(400, 64).cuda()

    def rows(H):
        if layout == "projection":
            return torch.randn(2, 400, H, 64, generator=gen).cuda(), lambda t: t.transpose(1, 2)
        if layout == "slice":
            return torch.randn(2, 400, 3 * H, 64, generator=gen).cuda(), lambda t: t[:, :, H:2 * H].transpose(1, 2)
        return torch.randn(2, 1, 400, 64, generator=gen).cuda(), lambda t: t.expand(2, H, 400, 64)

    leaves, xs, want = [], [], []
    grads = [torch.randn(2, H, 400, 64, generator=gen).cuda() for H in (4, 2)]
    for s, H in enumerate((4, 2)):
        t, view = rows(H)
        leaves.append(t.requires_grad_(s != frozen))
        xs.append(view(t * 2.0))
        x = view(t.detach())
        dx = fa.norm_rope_backward(x, None, grads[s], None, rope=rope, eps=None)[0]
        assert torch.equal(dx, fa.norm_rope_backward(None, None, grads[s], None, rope=rope, eps=None)[0])
        if layout != "expanded":
            assert dx.stride() == torch.empty_like(x).stride()
        again = t.detach().clone().requires_grad_()
        want.append(torch.autograd.grad(view(again * 2.0), again, dx)[0])
    y = fa.qk_norm_rope(*xs, rope=rope, eps=None)
    before = torch.cuda.memory_allocated()
    size = sum(t.numel() * 4 for t in leaves)
    del xs
    assert before - torch.cuda.memory_allocated() >= size
    torch.autograd.backward(y, grads)
    for s, t in enumerate(leaves):
        assert t.grad is None if s == frozen else torch.allclose(t.grad, want[s], rtol=1e-6, atol=1e-6)


def test_backward_of_the_rotation_alone_takes_rows_or_none():
    g = torch.randn(1, 2, 8, 64, device="cuda")
    rope = rope_table(8, 64).cuda()
    with pytest.raises(TypeError, match="q must be a tensor"):
        fa.norm_rope_backward(None, None, g, None, rope=rope)
    with pytest.raises(TypeError, match="q must be a tensor"):
        fa.norm_rope_backward(None, g, g, g, rope=rope, eps=None)
    with pytest.raises(ValueError, match="go together"):
        fa.norm_rope_backward(g, None, g, g, rope=rope, eps=None)
    dq, dk, _, _ = fa.norm_rope_backward(None, None, g, g, rope=rope, eps=None)
    assert torch.equal(dq, dk) and torch.equal(dq, fa.norm_rope_backward(g, None, g, None, rope=rope, eps=None)[0])


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
