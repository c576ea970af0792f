"""Plain 64-bit forms of the norm and rotation, the paged append and the chunk attention,
and small paged caches to run them on.

Half a step of a type is torch.finfo(t).eps / 2 relative to the value (for float16 also
2^-25 absolute, half its smallest subnormal).  Each bound below counts the roundings of the
computation it belongs to; U is float32's half step, 2^-24.
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def rope_table(rows, rot, base=10000.0):
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def pairs(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(y, rope, interleaved, back=False, magnitude=False):
    """Rotation of y [..., d] by table rows rope [..., rot]; with magnitude, the sum of the
    terms' absolute values in place of the result (what roundings are relative to)."""
    if rope is None:
        return y.abs() if magnitude else y
    rot = rope.shape[-1]
    a, b = pairs(rot, interleaved)
    c, s = rope[..., :rot // 2].double(), rope[..., rot // 2:].double()
    if back:
        s = -s
    z = y.abs() if magnitude else y.clone()
    if magnitude:
        y, c, s = y.abs(), c.abs(), s.abs()
        z[..., a] = y[..., a] * c + y[..., b] * s
    else:
        z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    return z


def norm_rotate(x, w, rope, eps, interleaved):
    """(value, bound on |output - value| for an output of x's type) of the norm and rotation.

    float32 roundings: the sum of d <= 128 squares in a tree of 8 + 4 adds (12 U), mean and eps
    (2 U), square root and reciprocal (half of these, 2 U, counted whole), two products (2 U),
    two products and a sum in the rotation with a table entry (4 U with its own rounding counted):
    below 24 U of the terms' magnitude; then one rounding to the type.
    """
    y = x.double()
    if eps is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        if w is not None:
            y = y * w.double()
    z = turn(y, rope, interleaved)
    bound = half_step(x.dtype) * z.abs() + 25 * U * turn(y, rope, interleaved, magnitude=True) + floor_of(x.dtype)
    return z, bound


def norm_rotate_grads(x, dz, w, rope, eps, interleaved):
    """(dx, bound, dw, bound) for x, dz [..., d]; dw summed over every row.

    dx: g carries 4 U of its magnitude, u one more, the normalised row 17 U, mean(u x) a tree of
    12 adds over products with 5 + 17 + 1 U, the difference and the factor r 18 U more: below
    64 U of r (|u| + |x| mean|u x|).  dw: each term 22 U of |g x|; the terms are added one after
    another within a lane (few here), then over 16 or 32 lanes, then over the blocks: below
    128 U of the sum of the terms' magnitudes for the sizes tested.
    """
    g = turn(dz.double(), rope, interleaved, back=True)
    gm = turn(dz.double(), rope, interleaved, back=True, magnitude=True)
    t = x.dtype
    if eps is None:
        return g, half_step(t) * g.abs() + 5 * U * gm + floor_of(t), None, None
    xd = x.double()
    r = 1.0 / (xd.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    xh = xd * r
    wd = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    u, um = g * wd, gm * wd.abs()
    dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    mag = r * (um + xh.abs() * (um * xh.abs()).mean(-1, keepdim=True))
    bound = half_step(t) * dx.abs() + 64 * U * mag + floor_of(t)
    if w is None:
        return dx, bound, None, None
    axes = tuple(range(x.dim() - 1))
    dw = (g * xh).sum(axes)
    wbound = half_step(w.dtype) * dw.abs() + 128 * U * (gm * xh.abs()).sum(axes) + floor_of(w.dtype)
    return dx, bound, dw, wbound


def paged_cache(new, total, Hkv, block, dtype, seed, spare=3, pad=float("nan")):
    """A paged cache on the CPU for sequences with `new` new tokens of `total` in all.

    Blocks sit in a shuffled order; the rows past a length and `spare` blocks that no
    sequence uses hold `pad`; table entries past a sequence's blocks are -1.  Returns
    (kpool, vpool, table, cu_tokens, seqlens).
    """
    g = torch.Generator().manual_seed(seed)
    blocks = [-(-n // block) for n in total]
    num = max(1, sum(blocks)) + spare
    perm = torch.randperm(num, generator=g).int()
    table = torch.full((len(total), max(1, max(blocks))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    pools = []
    for _ in range(2):
        pool = torch.full((num, Hkv, block, 128), pad, dtype=dtype)
        for b, n in enumerate(total):
            rows = torch.randn(n, Hkv, 128, generator=g).to(dtype)
            j = torch.arange(n)
            pool[table[b].long()[j // block], :, j % block] = rows
        pools.append(pool)
    cu = torch.tensor([0] + list(new), dtype=torch.int64).cumsum(0).int()
    return pools[0], pools[1], table, cu, torch.tensor(total, dtype=torch.int32)


def attend(q, kpool, vpool, table, cu, lens, causal=True, window=0, scale=None, skip=()):
    """(o, lse, bound on o, bound on lse) of the chunk attention, q [T, Hq, 128], tokens outside
    every sequence NaN.  `skip`: (sequence, logical block) pairs left out.

    Bounds.  A score's float32 sum of 128 exact products: its terms' magnitudes sum to about
    82 for N(0, 1) rows, times 1/sqrt(128); 64 U of that (2.8e-5), the exponent's argument and
    2^x a few 1e-6 more: each weight is off by at most 4e-5 of itself, and by half a step of the
    16-bit type as the MMA takes it (float16 weights below 2^-14 by 2^-25 absolute, against a
    largest weight of at least 1).  Sums, joins and divisions in float32 are within the 4e-5.
    """
    T, Hq, d = q.shape
    block, Hkv = kpool.shape[2], kpool.shape[1]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.full((T, Hq, d), float("nan"), dtype=torch.float64)
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float64)
    ob, lb = o.clone(), lse.clone()
    u = half_step(q.dtype)
    for b in range(table.shape[0]):
        t0, t1, n = int(cu[b]), int(cu[b + 1]), int(lens[b])
        m = t1 - t0
        if m == 0:
            continue
        place = torch.arange(n - m, n)[:, None]
        j = torch.arange(n)
        seen = torch.ones(m, n, dtype=torch.bool)
        if causal:
            seen &= j <= place
        if window:
            seen &= j > place - window
        for sb, blk in skip:
            if sb == b:
                seen &= ~((j >= blk * block) & (j < (blk + 1) * block))
        used = seen.any(0)
        jj = j[used]
        phys, off = table[b].long()[jj // block], jj % block
        for h in range(Hkv):
            k, v = kpool[phys, h, off].double(), vpool[phys, h, off].double()
            qq = q[t0:t1, h * G:(h + 1) * G].double().transpose(0, 1)
            s = (qq @ k.T * scale).masked_fill(~seen[:, used], -math.inf)
            z = torch.logsumexp(s, -1) if len(jj) else torch.full((G, m), -math.inf, dtype=torch.float64)
            p = torch.exp(s - z[..., None]).nan_to_num(0.0)
            oo, mag = p @ v, p @ v.abs()
            o[t0:t1, h * G:(h + 1) * G] = oo.transpose(0, 1)
            lse[t0:t1, h * G:(h + 1) * G] = z.T
            sub = floor_of(q.dtype) * v.abs().sum(0)
            ob[t0:t1, h * G:(h + 1) * G] = (u * oo.abs() + (u + 4e-5) * mag + sub + floor_of(q.dtype)).transpose(0, 1)
            lb[t0:t1, h * G:(h + 1) * G] = 4e-5 + 4 * U * z.T.abs().nan_to_num(0.0, 0.0, 0.0)
    return o, lse, ob, lb


def assert_within(got, ref, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = (got == ref) | (got.isnan() & ref.isnan())
    err = (got - ref).abs()
    bad = ~(same | (err <= bound))
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {i}: "
                             f"{got[tuple(i)]:.8g} for {ref[tuple(i)]:.8g} +- {bound[tuple(i)]:.3g}")
