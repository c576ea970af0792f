"""Chunk attention over a paged cache on the GPU against a plain 64-bit form."""
import pytest
import torch

import tiled_exact_attention_forward_b200 as fa
from gpu_helpers import requires_cuda
from paged_helpers import assert_within, attend, paged_cache

pytestmark = [pytest.mark.gpu, requires_cuda]

BF16, FP16 = torch.bfloat16, torch.float16


def make(new, total, Hq, Hkv, block, dtype, seed=0, extra=0):
    kp, vp, table, cu, lens = paged_cache(new, [max(n, 0) for n in total], Hkv, block, dtype, seed)
    q = torch.randn(sum(new) + extra, Hq, 128, generator=torch.Generator().manual_seed(seed + 5)).to(dtype)
    return q, kp, vp, table, cu, lens


def check(new, total, Hq, Hkv, block, dtype=BF16, seed=0, extra=0, no_cu=False, **kw):
    q, kp, vp, table, cu, lens = make(new, total, Hq, Hkv, block, dtype, seed, extra)
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=None if no_cu else cu.cuda(),
                    out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    o_ref, l_ref, ob, lb = attend(q, kp, vp, table, cu, lens, **kw)
    T = sum(new)
    assert_within(out[:T], o_ref[:T], ob[:T], "o")
    assert_within(lse[:T], l_ref[:T], lb[:T], "lse")
    assert (out[T:] == 7.0).all() and (lse[T:] == 7.0).all()  # tokens behind the last sequence
    return out, lse


def test_one_token_one_tile():
    check([1], [100], 4, 1, 16)


@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 256, 257, 1000])
def test_one_token_lengths(n):
    check([1], [n], 8, 2, 16, seed=n)


@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 63, 64, 65, 100, 128, 200])
def test_chunk_lengths(m):
    check([m], [m + 150], 8, 2, 16, seed=m)
    check([m], [m], 8, 2, 16, seed=m)


@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 2), (3, 2), (5, 1), (7, 2), (12, 1), (32, 1), (100, 1), (128, 1)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_groups(G, Hkv, dtype):
    check([1, 5, 90], [70, 5, 333], G * Hkv, Hkv, 32, dtype, seed=G)


@pytest.mark.parametrize("block", [1, 2, 4, 8, 16, 32, 64, 128, 256, 4096])
def test_block_sizes(block):
    check([1, 70, 3], [300, 270, 517], 4, 2, block, seed=block)


@pytest.mark.parametrize("window", [1, 2, 17, 128, 200, 10000])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_windows(window, dtype):
    check([1, 300, 20], [500, 410, 20], 4, 2, 16, dtype, seed=window, window=window)


@pytest.mark.parametrize("window", [0, 100])
def test_not_causal(window):
    check([1, 150, 20], [500, 410, 20], 4, 2, 16, seed=3, causal=False, window=window)


def test_scale():
    check([9], [200], 4, 2, 16, seed=4, scale=0.02)


def test_ragged_batch_with_empty_sequences():
    new = [0, 1, 0, 260, 17, 1, 0, 64, 3, 0]
    total = [0, 1, 40, 900, 17, 2100, 0, 64, 131, 5]
    check(new, total, 8, 2, 16, seed=5, extra=3)
    check(new, total, 8, 8, 64, FP16, seed=6)


def test_one_token_each_without_cu_tokens():
    total = [1 + 37 * b % 700 for b in range(50)]
    a = check([1] * 50, total, 8, 2, 16, seed=7, no_cu=True)
    b = check([1] * 50, total, 8, 2, 16, seed=7)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("B", [511, 512, 513, 1100])
def test_more_sequences_than_threads(B):
    check([1 + (b % 3 == 0) for b in range(B)], [2 + 7 * b % 60 for b in range(B)], 2, 1, 16, seed=B)


@pytest.mark.parametrize("B", [40, 300])
def test_padded_decode_batch(B):
    """A batch padded with sequences of length zero, one token each, many of them in a row."""
    total = [0 if 3 < b < B - 2 else 50 + 90 * b for b in range(B)]
    total = [min(n, 700) for n in total]
    q, kp, vp, table, cu, lens = make([1] * B, total, 8, 2, 16, BF16, seed=31)
    o, lse = fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda())
    assert fa.device_status() == fa.FA_OK
    empty = lens == 0
    assert (o[empty] == 0).all() and lse[empty].isneginf().all()
    o_ref, l_ref, ob, lb = attend(q, kp, vp, table, cu, lens)
    assert_within(o[~empty], o_ref[~empty], ob[~empty], "o")
    assert_within(lse[~empty], l_ref[~empty], lb[~empty], "lse")


@pytest.mark.parametrize("order", [(1, 300, 1), (300, 1, 1, 300, 300, 5), (1, 1, 300, 1, 300)])
@pytest.mark.parametrize("n", [100, 129, 400, 650])
def test_one_and_two_tile_items_in_turn(order, n):
    """Items of one and of two row tiles after one another, with even and odd numbers of key tiles."""
    check(list(order), [m + n for m in order], 4, 1, 16, seed=n)
    check(list(order), [m + n for m in order], 4, 2, 64, FP16, seed=n + 1, window=300)


def test_long_cache_spread_over_the_whole_grid():
    check([1], [20000], 2, 1, 16, seed=8)
    check([3], [20000], 2, 1, 128, FP16, seed=9)


def test_long_chunk():
    check([1500], [1777], 4, 2, 16, seed=10)
    check([700, 1], [700, 3000], 1, 1, 16, seed=11)


def test_zero_length_and_more_tokens_than_keys():
    """Lengths below the new tokens: the first ones sit at negative positions and see nothing."""
    q, kp, vp, table, cu, lens = make([4, 200, 3], [4, 200, 3], 4, 2, 16, BF16, seed=12)
    lens = torch.tensor([0, 120, 2], dtype=torch.int32)
    o, lse = fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda())
    assert fa.device_status() == fa.FA_OK
    assert (o[:4] == 0).all() and lse[:4].isneginf().all()
    assert (o[4:84] == 0).all() and lse[4:84].isneginf().all()
    assert (o[204] == 0).all() and lse[204].isneginf().all()
    cu2 = torch.tensor([0, 120, 122], dtype=torch.int32)
    keep = torch.cat([torch.arange(84, 204), torch.arange(205, 207)])
    o_ref, l_ref, ob, lb = attend(q[keep], kp, vp, table[1:], cu2, lens[1:])
    assert_within(o[keep], o_ref, ob, "o")
    assert_within(lse[keep], l_ref, lb, "lse")


def test_lengths_are_clamped_to_the_table():
    q, kp, vp, table, cu, lens = make([2], [64], 4, 2, 16, BF16, seed=13)
    a = fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda())
    b = fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda() + 1000, cu_tokens=cu.cuda())
    assert fa.device_status() == fa.FA_OK and all(torch.equal(x, y) for x, y in zip(a, b))


def test_blocks_behind_the_window_are_never_read():
    """Their table entries may be anything: an id outside the pool, a block of another sequence."""
    new, total, window = [3, 150], [900, 700], 100
    q, kp, vp, table, cu, lens = make(new, total, 4, 2, 16, BF16, seed=14)
    want = attend(q, kp, vp, table, cu, lens, window=window)
    t2 = table.clone()
    for b, (m, n) in enumerate(zip(new, total)):
        first = max(0, n - m - window + 1) // 16
        t2[b, :first] = 1 << 30
    o, lse = fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), t2.cuda(), lens.cuda(), cu_tokens=cu.cuda(), window=window)
    assert fa.device_status() == fa.FA_OK
    assert_within(o, want[0], want[2], "o")
    assert_within(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("block", [2, 8, 16, 64, 256])
@pytest.mark.parametrize("bad_id", [-1, -2, 10 ** 9])
def test_bad_block_ids_are_skipped_and_reported(block, bad_id):
    new, total = [1, 140, 2], [600, 520, 900]
    q, kp, vp, table, cu, lens = make(new, total, 4, 2, block, BF16, seed=15)
    skip = [(0, 0), (0, 1), (1, 300 // block), (2, 899 // block)]
    for b, blk in skip:
        table[b, blk] = bad_id
    o, lse = fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda())
    assert fa.device_status() == fa.FA_ERR_INVALID and fa.device_status() == fa.FA_OK
    safe = table.clamp(0, kp.shape[0] - 1)
    o_ref, l_ref, ob, lb = attend(q, kp, vp, safe, cu, lens, skip=skip)
    assert_within(o, o_ref, ob, "o")
    assert_within(lse, l_ref, lb, "lse")


def test_all_blocks_bad_leaves_nothing():
    q, kp, vp, table, cu, lens = make([2], [40], 4, 2, 16, BF16, seed=16)
    table.fill_(-1)
    o, lse = fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda())
    assert fa.device_status() == fa.FA_ERR_INVALID
    assert (o == 0).all() and lse.isneginf().all()


def test_nan_row_stays_in_its_sequence_and_head():
    new, total = [2, 3], [200, 150]
    q, kp, vp, table, cu, lens = make(new, total, 4, 2, 16, BF16, seed=17)
    args = (vp.cuda(), table.cuda(), lens.cuda(), cu.cuda())
    want, wl = fa.extend_paged(q.cuda(), kp.cuda(), *args)
    k2 = kp.clone()
    k2[table[0, 3], 1, 5] = float("nan")  # sequence 0, key head 1: query heads 2 and 3
    o, lse = fa.extend_paged(q.cuda(), k2.cuda(), *args)
    assert o[:2, 2:].isnan().all() and lse[:2, 2:].isnan().all()
    assert torch.equal(o[:2, :2], want[:2, :2]) and torch.equal(o[2:], want[2:]) and torch.equal(lse[2:], wl[2:])


def test_masked_keys_may_be_non_finite():
    """Keys that a row does not see (later tokens of its chunk) may hold NaN or infinity."""
    q, kp, vp, table, cu, lens = make([130], [400], 2, 1, 16, BF16, seed=18)
    args = (vp.cuda(), table.cuda(), lens.cuda(), cu.cuda())
    want, _ = fa.extend_paged(q.cuda(), kp.cuda(), *args)
    k2 = kp.clone()
    k2[table[0, 399 // 16], 0, 399 % 16] = float("nan")
    k2[table[0, 398 // 16], 0, 398 % 16] = float("inf")
    o, _ = fa.extend_paged(q.cuda(), k2.cuda(), *args)
    assert torch.equal(o[:128], want[:128]) and o[129].isnan().all()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("causal,window,row", [
    (True, 100, 150),    # behind the window of the later tokens of the first group
    (True, 100, 290),    # before and behind tokens of the third
    (True, 0, 399),      # the last token's own
    (False, 100, 150),
    (True, 30, 169),     # behind every window: of the chunk's own group, no token sees it
])
def test_reach_of_a_non_finite_value_row(value, causal, window, row):
    """Tokens that see the row come out non-finite; others may within its group of 64 tokens and its key
    head; every other output, and every lse, keeps its bits."""
    m, n, G = 200, 400, 4                       # positions 200 .. 399; groups of 2 * 128 / G = 64 tokens
    q, kp, vp, table, cu, lens = make([m, 30], [n, 300], 2 * G, 2, 16, BF16, seed=34)
    run = lambda v: fa.extend_paged(q.cuda(), kp.cuda(), v.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda(),  # noqa: E731
                                    causal=causal, window=window)
    want, wl = run(vp)
    v2 = vp.clone()
    v2[table[0, row // 16], 1, row % 16] = value  # sequence 0, key head 1: query heads 4 .. 7
    o, lse = run(v2)
    assert fa.device_status() == fa.FA_OK
    place = torch.arange(n - m, n)
    sees = torch.ones(m, dtype=torch.bool)
    if causal:
        sees &= row <= place
    if window:
        sees &= row > place - window
    assert not o[:m, G:][sees.cuda()].isfinite().any()
    group = torch.arange(m) // 64
    near = torch.isin(group, group[sees])       # groups with a token that sees the row
    assert torch.equal(lse, wl)
    assert torch.equal(o[:, :G], want[:, :G]) and torch.equal(o[m:], want[m:])
    assert torch.equal(o[:m][~near.cuda()], want[:m][~near.cuda()])
    assert sees.any() == (window != 30)


def test_lowest_and_large_scores():
    """Queries scaled until one key takes all the weight, and scores far below zero."""
    q, kp, vp, table, cu, lens = make([5], [300], 4, 2, 16, BF16, seed=19)
    q = q * 60
    o, lse = fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda())
    o_ref, l_ref, ob, lb = attend(q, kp, vp, table, cu, lens)
    # Scores are 60 times those that the bounds count on, and so are their errors.
    assert_within(o, o_ref, ob + 60 * 4e-5 * 6, "o")
    assert_within(lse, l_ref, 60 * lb, "lse")


def test_strided_queries_of_a_fused_projection():
    q, kp, vp, table, cu, lens = make([3, 70], [80, 200], 6, 2, 16, BF16, seed=20)
    x = torch.full((q.shape[0], 10, 128), float("nan"), dtype=BF16)
    x[:, :6] = q
    a = fa.extend_paged(x.cuda()[:, :6], kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda())
    b = fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda())
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_one_token_matches_paged_decode():
    total = [1, 17, 700, 2500]
    q, kp, vp, table, cu, lens = make([1] * 4, total, 3, 3, 16, BF16, seed=21)
    dev = [t.cuda() for t in (q, kp, vp, table, lens)]
    o, lse = fa.extend_paged(*dev)
    o2, lse2 = fa.decode_paged(*dev)
    _, _, ob, lb = attend(q, kp, vp, table, cu, lens)
    assert_within(o, o2.cpu().double(), 2 * ob, "o")
    assert_within(lse, lse2.cpu().double(), 2 * lb, "lse")


def test_same_bits_every_time():
    q, kp, vp, table, cu, lens = make([1, 200, 7], [4000, 1000, 300], 8, 2, 16, BF16, seed=22)
    dev = [t.cuda() for t in (q, kp, vp, table, lens, cu)]
    first = fa.extend_paged(*dev)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, fa.extend_paged(*dev)))


def test_captured_and_replayed_with_new_lengths():
    """One captured call serves other lengths and tables: nothing of them is read on the host."""
    new, total = [1, 1, 1], [300, 20, 900]
    q, kp, vp, table, cu, lens = make(new, total, 8, 2, 16, BF16, seed=23)
    dev = [t.cuda() for t in (q, kp, vp, table, lens)]
    fa.extend_paged(*dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.extend_paged(*dev)
    for lengths in ([300, 20, 900], [5, 0, 17], [299, 1, 640]):
        dev[4].copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = fa.extend_paged(*dev)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert fa.device_status() == fa.FA_OK


def test_two_streams_at_once():
    cases = [make([1, 40], [3000, 700], 8, 2, 16, BF16, seed=s) for s in (24, 25)]
    dev = [[t.cuda() for t in (c[0], c[1], c[2], c[3], c[5], c[4])] for c in cases]
    want = [fa.extend_paged(*d) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    got = []
    for _ in range(5):
        for d, s in zip(dev, streams):
            with torch.cuda.stream(s):
                got.append(fa.extend_paged(*d))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


def test_pool_offsets_past_32_bits():
    """Pools of more than 2^31 elements each: blocks at their far ends are read at their places."""
    Hkv, block = 8, 4096
    num = (1 << 31) // (block * Hkv * 128) + 3
    g = torch.Generator().manual_seed(27)
    small = [torch.randn(2, Hkv, block, 128, generator=g).to(BF16) for _ in range(2)]
    q = torch.randn(3, Hkv, 128, generator=g).to(BF16)
    kp, vp = (torch.zeros(num, Hkv, block, 128, dtype=BF16, device="cuda") for _ in range(2))
    for pool, rows in ((kp, small[0]), (vp, small[1])):
        pool[num - 1], pool[num - 2] = rows[0].cuda(), rows[1].cuda()
    table = torch.tensor([[num - 1, num - 2]], dtype=torch.int32)
    lens, cu = torch.tensor([5000], dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32)
    o, lse = fa.extend_paged(q.cuda(), kp, vp, table.cuda(), lens.cuda(), cu_tokens=cu.cuda())
    assert fa.device_status() == fa.FA_OK
    o_ref, l_ref, ob, lb = attend(q, *small, torch.tensor([[0, 1]], dtype=torch.int32), cu, lens)
    assert_within(o, o_ref, ob, "o")
    assert_within(lse, l_ref, lb, "lse")


def test_query_offsets_past_32_bits():
    """Queries and outputs of more than 2^31 elements: 8193 sequences of 64 new tokens over shared blocks."""
    B, m, Hq, Hkv, block = 8193, 64, 32, 4, 16
    kp, vp, table, _, _ = paged_cache([1], [128], Hkv, block, BF16, seed=35)
    table = table.expand(B, 8).contiguous()
    lens = (m + torch.arange(B) * 7 % 65).int()
    cu = (torch.arange(B + 1) * m).int()
    q = torch.empty(B * m, Hq, 128, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(36))
    assert q.numel() > 1 << 31
    o, lse = fa.extend_paged(q, kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda())
    assert fa.device_status() == fa.FA_OK
    for b in (0, 4096, B - 1):
        part = slice(b * m, (b + 1) * m)
        o_ref, l_ref, ob, lb = attend(q[part].cpu(), kp, vp, table[:1], torch.tensor([0, m]), lens[b:b + 1])
        assert_within(o[part], o_ref, ob, f"o of sequence {b}")
        assert_within(lse[part], l_ref, lb, f"lse of sequence {b}")


def test_tokens_outside_every_sequence_and_shared_blocks():
    """cu_tokens that begins past 0, sequences that share their first blocks, the same block twice."""
    q, kp, vp, table, cu, lens = make([4, 6, 70], [100, 120, 200], 4, 2, 16, BF16, seed=28, extra=9)
    cu = cu + 5
    table[1, :6] = table[0, :6]
    table[2, 3] = table[2, 7]
    out = torch.full(q.shape, 7.0, dtype=BF16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda(), out=out, lse=lse)
    assert fa.device_status() == fa.FA_OK
    o_ref, l_ref, ob, lb = attend(q, kp, vp, table, cu, lens)
    assert_within(out[5:85], o_ref[5:85], ob[5:85], "o")
    assert_within(lse[5:85], l_ref[5:85], lb[5:85], "lse")
    assert (out[:5] == 7.0).all() and (out[85:] == 7.0).all() and (lse[85:] == 7.0).all()


def test_bad_token_bounds_stay_inside_the_batch():
    """cu_tokens below 0 and past T are clamped: nothing outside the outputs is touched."""
    q, kp, vp, table, cu, lens = make([3, 4], [50, 60], 4, 2, 16, BF16, seed=29)
    cu = torch.tensor([-5, 3, 1000], dtype=torch.int32)
    lens = torch.tensor([50, 60], dtype=torch.int32)
    guard = torch.full((3, 7, 4, 128), 7.0, dtype=BF16, device="cuda")
    fa.extend_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), cu_tokens=cu.cuda(), out=guard[1])
    assert fa.device_status() == fa.FA_OK
    o_ref, _, ob, _ = attend(q, kp, vp, table, torch.tensor([0, 3, 7]), lens)
    assert_within(guard[1], o_ref, ob, "o")
    assert (guard[0] == 7.0).all() and (guard[2] == 7.0).all()


def test_workspace_of_another_call_and_of_stale_bits():
    """The workspace's contents do not matter: NaN bits, or another call's partial results."""
    a = make([1, 200], [9000, 3000], 8, 2, 16, BF16, seed=30)
    b = make([130, 3], [700, 20000], 8, 2, 16, BF16, seed=32)
    size = fa.extend_paged_workspace_size(300, 8, 2, 128)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    run = lambda c, **kw: fa.extend_paged(*(t.cuda() for t in (c[0], c[1], c[2], c[3], c[5], c[4])), **kw)  # noqa: E731
    for c in (a, b, a):
        want, got = run(c), run(c, workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_right_after_the_kernel_that_writes_its_inputs():
    """The launch overlaps the end of the kernel ahead of it, but reads nothing before that is done."""
    q, kp, vp, table, cu, lens = make([1, 1, 90], [2000, 30, 400], 8, 2, 16, BF16, seed=33)
    dev = [t.cuda() for t in (q, kp, vp, table, lens, cu)]
    want = fa.extend_paged(*dev)
    work = [torch.zeros_like(t) for t in dev]
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        for t in work:
            t.zero_()
        big.fill_(1)  # keeps the stream busy while the launches below queue up
        for t, s in zip(work, dev):
            t.copy_(s)
        got = fa.extend_paged(*work)
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_a_serving_run():
    """Prompt pieces and single tokens of two sequences through append_paged, extend_paged and
    decode_paged, against the causal attention of the whole sequences."""
    from paged_helpers import norm_rotate, rope_table

    H, d, block, n = 4, 128, 16, [77, 150]
    g = torch.Generator().manual_seed(26)
    xs = [torch.randn(m, 3 * H, d, generator=g).to(BF16) for m in n]
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(BF16) for _ in range(2))
    rope = rope_table(256, d)
    table = torch.arange(20, dtype=torch.int32).view(2, 10).flip(1).contiguous().cuda()
    kp, vp = (torch.full((20, H, block, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    outs = [[], []]
    done = [0, 0]
    for step in ([30, 100], [46, 0], [0, 48], [1, 2]):
        x = torch.cat([xs[b][done[b]:done[b] + m] for b, m in enumerate(step)]).cuda()
        done = [a + m for a, m in zip(done, step)]
        cu = torch.tensor([0, step[0], sum(step)], dtype=torch.int32, device="cuda")
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        q = fa.append_paged(x[:, H:2 * H], x[:, 2 * H:], kp, vp, table, lens, cu_tokens=cu, rope=rope.cuda(), q=x[:, :H],
                            q_weight=qw.cuda(), k_weight=kw.cuda(), eps=1e-6)
        o, lse = fa.extend_paged(q, kp, vp, table, lens, cu_tokens=cu)
        outs[0].append(o[:step[0]]), outs[1].append(o[step[0]:])
    last, _ = fa.decode_paged(torch.stack([q[0], q[2]]), kp, vp, table, lens)
    assert fa.device_status() == fa.FA_OK
    for b, x in enumerate(xs):
        qk = [norm_rotate(x[:, i * H:(i + 1) * H], w, rope[:n[b]][:, None], 1e-6, False)[0].to(BF16)
              for i, w in ((0, qw), (1, kw))]
        pool = [t.transpose(0, 1)[None].contiguous() for t in (qk[1], x[:, 2 * H:])]
        o_ref, _, ob, _ = attend(qk[0], *pool, torch.zeros(1, 1, dtype=torch.int32), torch.tensor([0, n[b]]),
                                 torch.tensor([n[b]]))
        got = torch.cat(outs[b])
        # The kernel's queries and keys may round the other way in places (a step is 2^-7 of a value):
        # scores move by about 2^-8 * sqrt(2 / 128) * 11 per side at most a few 1e-3 each, weights alike.
        assert_within(got, o_ref, ob + 0.02, f"sequence {b}")
        assert_within(last[b], o_ref[-1], ob[-1] + 0.02, f"decode of sequence {b}")
