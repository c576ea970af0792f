"""Appending new tokens to a paged cache on the GPU against plain 64-bit forms."""
import pytest
import torch

import tiled_exact_attention_forward_b200 as fa
from gpu_helpers import requires_cuda
from paged_helpers import assert_within, norm_rotate, paged_cache, rope_table

pytestmark = [pytest.mark.gpu, requires_cuda]

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def make(new, total, Hq, Hkv, block, dtype, seed, rot=128, extra=0):
    kp, vp, table, cu, lens = paged_cache(new, total, Hkv, block, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    T = sum(new) + extra
    x = torch.randn(T, Hq + 2 * Hkv, 128, generator=g).to(dtype)
    qw, kw = ((1 + 0.3 * torch.randn(128, generator=g)).to(dtype) for _ in range(2))
    return x, kp, vp, table, cu, lens, qw, kw, rope_table(max(total) + 1, rot) if rot else None


def check(new, total, Hq, Hkv, block, dtype, seed=0, rot=128, inter=False, eps=1e-6, with_q=True, no_cu=False, extra=0):
    x, kp, vp, table, cu, lens, qw, kw, rope = make(new, total, Hq, Hkv, block, dtype, seed, rot, extra)
    if eps is None:
        qw = kw = None
    T = x.shape[0]
    xd = x.cuda()
    kd, vd = kp.cuda(), vp.cuda()
    q_out = torch.full((T, Hq, 128), 7.0, dtype=dtype, device="cuda") if with_q else None
    put = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = fa.append_paged(xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], kd, vd, table.cuda(), lens.cuda(),
                          cu_tokens=None if no_cu else cu.cuda(), rope=put(rope), q=xd[:, :Hq] if with_q else None,
                          q_weight=put(qw), k_weight=put(kw), eps=eps, interleaved=inter, q_out=q_out)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    want_k, want_v, bound = kp.double(), vp.double(), torch.zeros(kp.shape, dtype=torch.float64)
    for b in range(len(new)):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        at = torch.arange(total[b] - new[b], total[b])
        phys, off = table[b].long()[at // block], at % block
        r = None if rope is None else rope[at][:, None]
        if not len(at):
            continue
        z, bd = norm_rotate(x[t0:t1, Hq:Hq + Hkv], kw, r, eps, inter)
        if rope is None and eps is None:
            bd.zero_()
        want_k[phys, :, off], bound[phys, :, off] = z, bd
        want_v[phys, :, off] = x[t0:t1, Hq + Hkv:].double()
        if with_q:
            z, bd = norm_rotate(x[t0:t1, :Hq], qw, r, eps, inter)
            assert_within(got[t0:t1], z, bd, f"q of sequence {b}")
    assert_within(kd, want_k, bound, "key pool")
    assert_within(vd, want_v, torch.zeros_like(bound), "value pool")
    if with_q:
        assert (got[sum(new):] == 7.0).all()  # tokens behind the last sequence
    assert torch.equal(xd.cpu(), x)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("block", [1, 4, 16, 128, 4096])
def test_ragged_batch(dtype, inter, block):
    check([3, 0, 1, 40, 17], [3, 9, 50, 41, 300], 6, 2, block, dtype, seed=block, inter=inter)


@pytest.mark.parametrize("rot", [0, 16, 96, 128])
@pytest.mark.parametrize("eps", [None, 1e-5])
@pytest.mark.parametrize("with_q", [False, True])
def test_parts(rot, eps, with_q):
    check([5, 2], [20, 33], 8, 4, 16, BF16, seed=rot, rot=rot, eps=eps, with_q=with_q)


@pytest.mark.parametrize("B", [1, 2, 15, 16, 17, 64, 257, 1000])
def test_one_token_each(B):
    total = [1 + (7 * b) % 40 for b in range(B)]
    check([1] * B, total, 4, 1, 16, BF16, seed=B)
    check([1] * B, total, 4, 1, 16, BF16, seed=B, no_cu=True)


@pytest.mark.parametrize("B", [3, 16, 40, 300])
def test_many_sequences_some_empty(B):
    new = [(5 * b) % 4 for b in range(B)]
    check(new, [n + (3 * b) % 30 for b, n in enumerate(new)], 2, 3, 8, FP16, seed=B, extra=9)


def test_heads_that_do_not_fill_a_group():
    check([9, 30], [12, 64], 7, 5, 32, BF16, seed=3)
    check([9, 30], [12, 64], 1, 1, 32, BF16, seed=4)


def test_tokens_without_a_place_are_left_out():
    """A block id outside the pool, a position past the cache, one below 0, one past the table."""
    new, total, Hkv, block = [4, 4, 4, 4], [20, 20, 20, 20], 2, 8
    x, kp, vp, table, cu, lens, qw, kw, rope = make(new, total, 2, Hkv, block, BF16, seed=5)
    table[0, 2] = kp.shape[0]                # sequence 0's last block (positions 16 .. 19)
    lens[1] = 26                             # positions 22 .. 25: two past the 24 the table holds
    lens[2] = 2                              # positions -2 .. 1: two below 0
    rope = rope[:18]                         # sequence 3's positions 16 .. 19: two past the table
    xd, kd, vd = x.cuda(), kp.cuda(), vp.cuda()
    table[1] = table[3]                      # sequence 1's writes 22, 23 lie in sequence 3's last block, unused
    rope_long = rope_table(30, 128)
    for r, bad in ((rope, True), (rope_long, True)):
        kd.copy_(kp), vd.copy_(vp)
        fa.append_paged(xd[:, 2:4], xd[:, 4:], kd, vd, table.cuda(), lens.cuda(), cu_tokens=cu.cuda(), rope=r.cuda())
        assert (fa.device_status() == fa.FA_ERR_INVALID) == bad
        want_v = vp.clone()
        for b in range(4):
            for i in range(4):
                pos = int(lens[b]) - 4 + i
                if b == 0 or pos < 0 or pos >= 24 or pos >= r.shape[0]:
                    continue
                want_v[int(table[b, pos // block]), :, pos % block] = x[int(cu[b]) + i, 4:]
        assert torch.equal(vd.cpu().nan_to_num(9.0), want_v.nan_to_num(9.0))


@pytest.mark.parametrize("rot,eps", [(128, 1e-6), (64, None), (0, 1e-6)])
def test_a_token_without_a_place_has_no_query_either(rot, eps):
    """A block id outside the pool, a position below 0 and one past the cache: the token's key and value
    are not written and its query is NaN where it would be turned; all else is as without them."""
    new, total, Hq, Hkv, block = [4, 4, 4, 3], [20, 20, 20, 9], 6, 2, 8
    x, kp, vp, table, cu, lens, qw, kw, rope = make(new, total, Hq, Hkv, block, FP16, seed=6, rot=rot)
    rope = rope_table(32, rot) if rot else None
    if eps is None:
        qw = kw = None
    put = lambda t: None if t is None else t.cuda()  # noqa: E731

    def run(table, lens):
        kd, vd, xd = kp.cuda(), vp.cuda(), x.cuda()
        q = fa.append_paged(xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], kd, vd, table.cuda(), lens.cuda(), cu_tokens=cu.cuda(),
                            rope=put(rope), q=xd[:, :Hq], q_weight=put(qw), k_weight=put(kw), eps=eps)
        return fa.device_status(), q.cpu(), kd.cpu(), vd.cpu()

    status, q, kd, vd = run(table, lens)
    assert status == fa.FA_OK
    for bad_id in (-1, kp.shape[0], 2 ** 31 - 1):
        t2, l2 = table.clone(), lens.clone()
        t2[0, 2] = bad_id                # sequence 0's tokens, positions 16 .. 19
        l2[1] = 2                        # sequence 1: positions -2 .. 1, two below 0
        l2[2] = 26                       # sequence 2: positions 22 .. 25, two past the 24 that the table holds
        status, q2, kd2, vd2 = run(t2, l2)
        assert status == fa.FA_ERR_INVALID
        lost = [0, 1, 2, 3, 4, 5, 10, 11]
        moved = [6, 7, 8, 9]             # written at other positions than before
        same = [12, 13, 14]
        assert torch.equal(q2[same], q[same]) and q2[moved].isfinite().all()
        if rot:
            assert q2[lost][..., :rot].isnan().all()
        if rot < 128:
            assert torch.equal(q2[lost][..., rot:], q[lost][..., rot:])
        want_k, want_v = kp.clone(), vp.clone()
        for t, b, pos in ((6, 1, 0), (7, 1, 1), (8, 2, 22), (9, 2, 23), (12, 3, 6), (13, 3, 7), (14, 3, 8)):
            at = (int(table[b, pos // block]), slice(None), pos % block)
            r = None if rope is None else rope[pos]
            z, bound = norm_rotate(x[t, Hq:Hq + Hkv], kw, r, eps, False)
            assert_within(kd2[at], z, bound, f"key of token {t}")
            want_k[at], want_v[at] = kd2[at], x[t, Hq + Hkv:]
        assert torch.equal(kd2.nan_to_num(9.0), want_k.nan_to_num(9.0))
        assert torch.equal(vd2.nan_to_num(9.0), want_v.nan_to_num(9.0))


def test_pool_offsets_past_32_bits():
    """A pool of more than 2^31 elements: the last block is written at its place."""
    block, Hkv = 4096, 8
    num = (1 << 31) // (block * Hkv * 128) + 2
    kp = torch.zeros(num, Hkv, block, 128, dtype=BF16, device="cuda")
    vp = torch.zeros_like(kp)
    x = torch.randn(3, 2 * Hkv, 128, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    table = torch.tensor([[num - 1]], dtype=torch.int32, device="cuda")
    fa.append_paged(x[:, :Hkv], x[:, Hkv:], kp, vp, table, torch.tensor([4096], dtype=torch.int32, device="cuda"),
                    cu_tokens=torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    assert fa.device_status() == fa.FA_OK
    assert torch.equal(kp[num - 1, :, 4093:], x[:, :Hkv].transpose(0, 1))
    assert torch.equal(vp[num - 1, :, 4093:], x[:, Hkv:].transpose(0, 1))
    assert int(kp[num - 1].count_nonzero()) == int(x[:, :Hkv].count_nonzero()) and not kp[:num - 1].any()
