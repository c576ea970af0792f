"""Per-head norm and position rotation on the GPU against plain 64-bit forms."""
import pytest
import torch

import tiled_exact_attention_forward_b200 as fa
from gpu_helpers import requires_cuda
from paged_helpers import assert_within, norm_rotate, norm_rotate_grads, rope_table, turn

pytestmark = [pytest.mark.gpu, requires_cuda]

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def make(B, Hq, Hk, N, d, rot, dtype, seed, wdtype=None, rows=None):
    """Inputs as a projection leaves them ([B, N, H, d] seen as [B, H, N, d]), gradients contiguous."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, N, Hq, d, generator=g).to(dtype).transpose(1, 2)
    k = torch.randn(B, N, Hk, d, generator=g).to(dtype).transpose(1, 2)
    dq = torch.randn(B, Hq, N, d, generator=g).to(dtype)
    dk = torch.randn(B, Hk, N, d, generator=g).to(dtype)
    qw = (1 + 0.3 * torch.randn(d, generator=g)).to(wdtype or dtype)
    kw = (1 + 0.3 * torch.randn(d, generator=g)).to(wdtype or dtype)
    return q, k, dq, dk, qw, kw, rope_table(rows or N, rot) if rot else None


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check(q, k, dq, dk, qw, kw, rope, eps, inter, positions=None, table=None):
    """Forward and backward against the 64-bit forms; `table`: the rope rows of every position."""
    q_, k_, dq_, dk_, qw_, kw_, rope_ = cuda(q, k, dq, dk, qw, kw, rope)
    pos_ = None if positions is None else positions.cuda()
    yq, yk = fa.norm_rope(q_, k_, qw_, kw_, rope_, pos_, eps, inter)
    gq, gk, gqw, gkw = fa.norm_rope_backward(q_, k_, dq_, dk_, qw_, kw_, rope_, pos_, eps, inter)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    assert yq.is_contiguous() and yk.is_contiguous() and gq.stride() == q_.stride()
    for name, x, dz, w, y, gx, gw in (("q", q, dq, qw, yq, gq, gqw), ("k", k, dk, kw, yk, gk, gkw)):
        z, b = norm_rotate(x, w, table, eps, inter)
        assert_within(y, z, b, f"{name} out")
        dx, b, dw, wb = norm_rotate_grads(x, dz, w, table, eps, inter)
        assert_within(gx, dx, b, f"d{name}")
        if dw is None:
            assert gw is None
        else:
            assert gw.dtype == w.dtype
            assert_within(gw, dw, wb, f"d{name}_weight")


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("part", ["norm", "rope", "both"])
def test_forward_and_backward(dtype, d, inter, part):
    rot = 0 if part == "norm" else d
    q, k, dq, dk, qw, kw, rope = make(2, 5, 2, 37, d, rot, dtype, seed=1)
    if part == "rope":
        qw = kw = None
    check(q, k, dq, dk, qw, kw, rope, None if part == "rope" else 1e-6, inter, table=rope)


@pytest.mark.parametrize("rot", [16, 48, 96, 112])
@pytest.mark.parametrize("inter", [False, True])
def test_partial_rotation(rot, inter):
    q, k, dq, dk, qw, kw, rope = make(1, 3, 3, 50, 128, rot, BF16, seed=rot)
    check(q, k, dq, dk, qw, kw, rope, 1e-6, inter, table=rope)


@pytest.mark.parametrize("B,Hq,Hk,N", [(1, 1, 1, 1), (3, 4, 4, 16), (1, 7, 1, 17), (2, 9, 3, 333), (5, 8, 2, 129)])
def test_sizes(B, Hq, Hk, N):
    q, k, dq, dk, qw, kw, rope = make(B, Hq, Hk, N, 128, 128, BF16, seed=N)
    check(q, k, dq, dk, qw, kw, rope, 1e-5, False, table=rope)


@pytest.mark.parametrize("Hq,Hk", [(1, 2500), (2500, 1)])
def test_lopsided_heads(Hq, Hk):
    q, k, dq, dk, qw, kw, rope = make(1, Hq, Hk, 3, 64, 64, BF16, seed=20)
    check(q, k, dq, dk, qw, kw, rope, 1e-6, False, table=rope)


def test_float32_weights_with_16_bit_rows():
    q, k, dq, dk, qw, kw, rope = make(2, 4, 2, 40, 128, 64, BF16, seed=3, wdtype=FP32)
    check(q, k, dq, dk, qw, kw, rope, 1e-6, False, table=rope)


def test_weight_of_one_side_only():
    q, k, dq, dk, qw, kw, rope = make(1, 4, 2, 40, 128, 128, FP16, seed=4)
    check(q, k, dq, dk, qw, None, rope, 1e-6, False, table=rope)
    check(q, k, dq, dk, None, kw, rope, 1e-6, False, table=rope)


@pytest.mark.parametrize("shared", [False, True])
def test_given_positions(shared):
    """Positions in any order, the same one twice, the table's last row."""
    B, N, rows = 3, 21, 5000
    q, k, dq, dk, qw, kw, rope = make(B, 4, 2, N, 128, 128, BF16, seed=5, rows=rows)
    pos = torch.randint(0, rows, (N,) if shared else (B, N), generator=torch.Generator().manual_seed(6), dtype=torch.int32)
    pos[..., 0] = rows - 1
    pos[..., 1] = pos[..., 2]
    table = rope[pos.long()] if shared else rope[pos.long()][:, None]
    check(q, k, dq, dk, qw, kw, rope, 1e-6, False, positions=pos, table=table)


def test_packed_tokens_from_a_fused_projection():
    T, Hq, Hk, rows = 45, 6, 2, 900
    g = torch.Generator().manual_seed(7)
    x = torch.randn(T, Hq + 2 * Hk, 128, generator=g).to(BF16)
    rope, pos = rope_table(rows, 128), torch.randint(0, rows, (T,), generator=g, dtype=torch.int32)
    xd = x.cuda()
    yq, yk = fa.norm_rope(xd[:, :Hq], xd[:, Hq:Hq + Hk], rope=rope.cuda(), positions=pos.cuda())
    for y, part in ((yq, x[:, :Hq]), (yk, x[:, Hq:Hq + Hk])):
        z, b = norm_rotate(part, None, rope[pos.long()][:, None], 1e-6, False)
        assert y.is_contiguous()
        assert_within(y, z, b, "packed")
    assert torch.equal(xd.cpu(), x)


def test_in_place_and_query_only():
    q, k, dq, dk, qw, kw, rope = make(2, 4, 4, 33, 128, 128, BF16, seed=8)
    want = fa.norm_rope(q.cuda(), None, qw.cuda(), rope=rope.cuda())
    x = q.cuda()
    got = fa.norm_rope(x, None, qw.cuda(), rope=rope.cuda(), q_out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
    g1 = fa.norm_rope_backward(q.cuda(), None, dq.cuda(), None, qw.cuda(), rope=rope.cuda())
    assert g1[1] is None and g1[3] is None
    dx, b, dw, wb = norm_rotate_grads(q, dq, qw, rope, 1e-6, False)
    assert_within(g1[0], dx, b, "dq")
    assert_within(g1[2], dw, wb, "dq_weight")


def test_rows_of_zeros_and_large_values():
    """A row of zeros stays zero (eps keeps it finite); rows whose squares pass float16's range."""
    q, k, dq, dk, qw, kw, rope = make(1, 2, 2, 8, 128, 128, FP16, seed=9)
    q, k = q.clone(), k.clone()
    q[0, 0, 3] = 0
    k[0, 1, 5] *= 8000
    check(q, k, dq, dk, qw, kw, rope, 1e-6, False, table=rope)


@pytest.mark.parametrize("size,eps", [(1e15, 1e-6), (1e-15, 0.0), (1e-3, 0.0)])
def test_rows_far_from_one(size, eps):
    """1/|x| cubed leaves float32's range at the first two sizes; the gradients do not."""
    q, k, dq, dk, qw, kw, rope = make(1, 2, 2, 8, 128, 128, FP32, seed=19)
    check(q * size, k * size, dq, dk, qw, kw, rope, eps, False, table=rope)


def test_non_finite_rows_stay_in_their_rows():
    q, k, dq, dk, qw, kw, rope = make(1, 4, 2, 20, 128, 128, BF16, seed=10)
    want, _ = fa.norm_rope(q.cuda(), k.cuda(), qw.cuda(), kw.cuda(), rope.cuda())
    bad = q.cuda().clone()
    bad[0, 1, 7] = float("nan")
    bad[0, 2, 9, 5] = float("inf")
    got, _ = fa.norm_rope(bad, k.cuda(), qw.cuda(), kw.cuda(), rope.cuda())
    keep = torch.ones(1, 4, 20, dtype=torch.bool)
    keep[0, 1, 7] = keep[0, 2, 9] = False
    assert torch.equal(got.cpu()[keep], want.cpu()[keep]) and got[0, 1, 7].isnan().all()


@pytest.mark.parametrize("where", [-1, 30, 2 ** 31 - 1])
def test_position_outside_the_table(where):
    q, k, dq, dk, qw, kw, rope = make(1, 2, 2, 10, 128, 64, BF16, seed=11, rows=30)
    pos = torch.arange(10, dtype=torch.int32)
    good = fa.norm_rope(q.cuda(), k.cuda(), rope=rope.cuda(), positions=pos.cuda())[0]
    assert fa.device_status() == fa.FA_OK
    pos[4] = where
    y = fa.norm_rope(q.cuda(), k.cuda(), rope=rope.cuda(), positions=pos.cuda())[0]
    assert fa.device_status() == fa.FA_ERR_INVALID and fa.device_status() == fa.FA_OK
    assert y[:, :, 4, :64].isnan().all() and torch.equal(y[:, :, 4, 64:], good[:, :, 4, 64:])
    keep = torch.arange(10) != 4
    assert torch.equal(y[:, :, keep], good[:, :, keep])


def test_weight_gradients_are_the_same_bits_every_time():
    q, k, dq, dk, qw, kw, rope = cuda(*make(2, 16, 4, 700, 128, 128, BF16, seed=12, wdtype=FP32))
    first = fa.norm_rope_backward(q, k, dq, dk, qw, kw, rope)
    for _ in range(3):
        again = fa.norm_rope_backward(q, k, dq, dk, qw, kw, rope)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_gradients_against_differences():
    """Central differences of the 64-bit forward along random directions, and float32 gradients."""
    q, k, dq, dk, qw, kw, rope = make(1, 2, 1, 6, 64, 32, FP32, seed=13)
    gq, gk, gqw, gkw = fa.norm_rope_backward(*cuda(q, k, dq, dk, qw, kw, rope), None, 1e-6, True)
    g = torch.Generator().manual_seed(14)
    for x, w, dz, gx, gw in ((q, qw, dq, gq, gqw), (k, kw, dk, gk, gkw)):
        def loss(x_, w_):
            y = x_ / (x_.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w_
            return (turn(y, rope, True) * dz.double()).sum()

        vx, vw = torch.randn(x.shape, generator=g).double(), torch.randn(w.shape, generator=g).double()
        h = 1e-5  # the difference's error is O(h^2), about 1e-10 of the third derivative
        dx = (loss(x.double() + h * vx, w.double()) - loss(x.double() - h * vx, w.double())) / (2 * h)
        dw = (loss(x.double(), w.double() + h * vw) - loss(x.double(), w.double() - h * vw)) / (2 * h)
        n = x.numel()
        scale_x = float((gx.cpu().double().abs() * vx.abs()).sum())
        scale_w = float((gw.cpu().double().abs() * vw.abs()).sum())
        # float32 gradients carry at most 64 U (dx) and 128 U (dw) of their terms, a few times themselves.
        assert abs(float((gx.cpu().double() * vx).sum() - dx)) <= 1e-4 * scale_x, n
        assert abs(float((gw.cpu().double() * vw).sum() - dw)) <= 1e-4 * scale_w, n


def test_autograd_before_attention():
    """qk_norm_rope, attention and both backward passes as one graph, against the calls made by hand."""
    B, H, N = 1, 2, 200
    q, k, dq, dk, qw, kw, rope = make(B, H, H, N, 128, 128, BF16, seed=15)
    v = torch.randn(B, H, N, 128, generator=torch.Generator().manual_seed(16)).to(BF16).cuda()
    leaves = [t.cuda().requires_grad_() for t in (q, k, qw, kw)]
    rq, rk = fa.qk_norm_rope(*leaves, rope=rope.cuda())
    o = fa.attention(rq, rk, v, causal=True)
    do = dq.cuda()
    o.backward(do)
    with torch.no_grad():
        yq, yk = fa.norm_rope(*leaves, rope=rope.cuda())
        o2, lse = fa.forward(yq, yk, v, causal=True)
        gq, gk, _ = fa.backward(yq, yk, v, o2, do, lse, causal=True)
        want = fa.norm_rope_backward(leaves[0], leaves[1], gq, gk, leaves[2], leaves[3], rope=rope.cuda())
    assert torch.equal(o, o2)
    # fa.backward adds dQ tiles in the order in which they finish: dq and its weight's gradient
    # agree to the roundings of that sum, dk's to the bit.
    for leaf, w in zip(leaves, want):
        assert torch.allclose(leaf.grad.float(), w.float(), rtol=0.03, atol=0.02 * float(w.float().abs().max()))
    assert torch.equal(leaves[1].grad, want[1]) and torch.equal(leaves[3].grad, want[3])


def test_broadcast_head_gets_its_gradient():
    """One key head expanded over four: read through its zero stride, its gradient the sum."""
    g = torch.Generator().manual_seed(17)
    q = torch.randn(1, 4, 30, 64, generator=g).cuda()
    k1 = torch.randn(1, 1, 30, 64, generator=g).cuda().requires_grad_()
    dk = torch.randn(1, 4, 30, 64, generator=g)
    rope = rope_table(30, 64)
    _, yk = fa.qk_norm_rope(q, k1.expand(1, 4, 30, 64), rope=rope.cuda())
    yk.backward(dk.cuda())
    dx, b, _, _ = norm_rotate_grads(k1.detach().cpu().expand(1, 4, 30, 64), dk, None, rope, 1e-6, False)
    # torch adds the four float32 gradients: three roundings of partial sums more.
    assert_within(k1.grad, dx.sum(1, keepdim=True), (b + 4 * 2.0 ** -24 * dx.abs()).sum(1, keepdim=True), "shared head")


@pytest.mark.parametrize("how", ["sum", "narrow", "offset", "turned"])
def test_gradients_as_autograd_lays_them_out(how):
    """Expanded, sliced, misaligned and transposed gradients of the outputs."""
    x = torch.randn(2, 3, 20, 64, generator=torch.Generator().manual_seed(20)).to(BF16).cuda()
    rope = rope_table(20, 64).cuda()
    w = torch.ones(64, dtype=BF16, device="cuda")
    leaf, lw = x.clone().requires_grad_(), w.clone().requires_grad_()
    y = fa.qk_norm_rope(leaf, None, lw, None, rope)
    c = torch.randn(2, 3, 20, 64, generator=torch.Generator().manual_seed(21)).to(BF16).cuda()
    if how == "sum":
        g = torch.ones_like(x)
        y.sum().backward()
    elif how == "narrow":  # rows 65 elements apart
        g = c
        torch.cat([y, y.new_zeros(2, 3, 20, 1)], -1).backward(torch.cat([c, c[..., :1]], -1))
    elif how == "offset":  # rows that begin 2 bytes past a boundary
        g = c
        y.backward(torch.cat([c.new_zeros(1), c.flatten()])[1:].view_as(c))
    else:
        g = c
        y.transpose(2, 3).backward(c.transpose(2, 3).contiguous())
    want = fa.norm_rope_backward(x, None, g, None, w, None, rope)
    assert torch.equal(leaf.grad, want[0]) and torch.equal(lw.grad, want[2])


def test_statuses_become_errors():
    """What the C ABI refuses raises FAError and leaves the next call unharmed."""
    x = torch.randn(1, 2, 4, 96, device="cuda")
    with pytest.raises(fa.FAError) as e:
        fa.norm_rope(x)
    assert e.value.status == fa.FA_ERR_UNSUPPORTED
    y = torch.randn(1, 2, 4, 66, device="cuda")[..., :64]  # rows 66 elements apart: not a multiple of 16 bytes
    with pytest.raises(fa.FAError) as e:
        fa.norm_rope(y)
    assert e.value.status == fa.FA_ERR_INVALID
    with pytest.raises(fa.FAError):
        fa.norm_rope(torch.empty(1, 2, 0, 64, device="cuda"))
    x = torch.ones(1, 2, 4, 64, device="cuda")
    assert torch.allclose(fa.norm_rope(x, eps=0.0), x, atol=1e-6)


def test_second_derivatives_are_refused():
    x = torch.randn(1, 1, 4, 64, device="cuda").requires_grad_()
    y = fa.qk_norm_rope(x, rope=rope_table(4, 64).cuda())
    (g,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_captured_and_replayed():
    q, k, dq, dk, qw, kw, rope = cuda(*make(2, 4, 2, 64, 128, 128, BF16, seed=18))
    run = lambda: (*fa.norm_rope(q, k, qw, kw, rope), *fa.norm_rope_backward(q, k, dq, dk, qw, kw, rope))  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    q.mul_(0.5)
    dq.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, run()))


def test_row_offsets_past_32_bits():
    """Queries, outputs and gradients of more than 2^31 elements: the last rows are read and written at
    their places."""
    T, Hq = (1 << 31) // (32 * 128) + 70, 32
    x = torch.empty(T, Hq + 1, 128, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(22))
    q, k = x[:, :Hq], x[:, Hq:]
    assert q.numel() > 1 << 31
    pos = (torch.arange(T, device="cuda") % 100).int()
    rope = rope_table(100, 128).cuda()
    yq, yk = fa.norm_rope(q, k, rope=rope, positions=pos)
    gq, gk, _, _ = fa.norm_rope_backward(q, k, yq, yk, rope=rope, positions=pos)
    assert fa.device_status() == fa.FA_OK
    for part in (slice(0, 70), slice(T - 70, T)):
        want = fa.norm_rope(q[part], k[part], rope=rope, positions=pos[part])
        assert torch.equal(yq[part], want[0]) and torch.equal(yk[part], want[1])
        g = fa.norm_rope_backward(q[part], k[part], yq[part], yk[part], rope=rope, positions=pos[part])
        assert torch.equal(gq[part], g[0]) and torch.equal(gk[part], g[1])
    z, b = norm_rotate(q[-3:].cpu(), None, rope.cpu()[pos[-3:].cpu().long()][:, None], 1e-6, False)
    assert_within(yq[-3:], z, b, "last rows")
