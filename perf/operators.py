"""The operators around the paged cache and the position rotation: cases, plain forms, exact values.

Four kinds of case, each one pass of an operator as a program calls it:

  rows    per-head norm and position rotation of the queries and keys of a batch of
          tokens, read as views of one fused projection output [T, Hq + 2 Hkv, d]
  train   the same over [B, H, N, d] with its gradients (input, weights): the step
          before attention and the step after its backward
  append  keys and values of new tokens put into a paged cache, keys (and the queries)
          rotated on the way; the caches come back
  chunk   attention of each sequence's new tokens over its paged cache

Lengths follow from the case alone (`lens` seeds them); values follow from the seed.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS = 1e-6
_BASE = 10000.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One token for each of 64 sequences (the paged decode workload's batch), grouped
        # heads: a decode step's queries and keys, a matter of latency.
        dict(name="rows_64_tokens", kind="rows", T=64, Hq=32, Hkv=8, d=128, rot=128, inter=False,
             norm=True, dtype="bf16"),
        # The training workload's shape (B 2, H 16, N 4096): norm, rotation and gradients.
        dict(name="train_4k_bf16", kind="train", B=2, Hq=16, Hkv=16, N=4096, d=128, rot=128, inter=False,
             norm=True, dtype="bf16"),
        # Odd length and head counts, float32, d = 64, half of the head rotated in adjacent pairs.
        dict(name="train_odd_fp32", kind="train", B=3, Hq=5, Hkv=1, N=1003, d=64, rot=32, inter=True,
             norm=True, dtype="fp32"),
        # The long-context shape (16K tokens), float16.
        dict(name="train_16k_fp16", kind="train", B=1, Hq=32, Hkv=8, N=16384, d=128, rot=128, inter=False,
             norm=True, dtype="fp16"),
        # One new token for each of 64 sequences: queries and keys normed and rotated, keys and
        # values into 16-row blocks.  A decode step.
        dict(name="append_64_tokens", kind="append", B=64, new_lo=1, new_hi=1, old_lo=0, old_hi=300, lens=1,
             Hq=32, Hkv=8, block=16, rot=128, inter=False, norm=True, with_q=True, dtype="bf16"),
        # Prompts of eight sequences, 16K tokens in all: the largest write.
        dict(name="append_prompts", kind="append", B=8, new_lo=2048, new_hi=2048, old_lo=0, old_hi=0, lens=2,
             Hq=32, Hkv=32, block=16, rot=128, inter=False, norm=False, with_q=False, dtype="bf16"),
        # Ragged chunks onto ragged caches, partial rotation in adjacent pairs, 64-row blocks.
        dict(name="append_ragged", kind="append", B=13, new_lo=1, new_hi=517, old_lo=0, old_hi=900, lens=3,
             Hq=24, Hkv=4, block=64, rot=64, inter=True, norm=True, with_q=True, dtype="fp16"),
        # One sequence, one token, a short cache: the smallest call.
        dict(name="chunk_one_token", kind="chunk", B=1, new_lo=1, new_hi=1, old_lo=511, old_hi=511, lens=4,
             Hq=32, Hkv=8, block=16, window=0, dtype="bf16"),
        # The paged decode workload's lengths with grouped heads: bound by reading the cache.
        dict(name="chunk_64_tokens", kind="chunk", B=64, new_lo=1, new_hi=1, old_lo=511, old_hi=8191, lens=5,
             Hq=32, Hkv=8, block=16, window=0, dtype="bf16"),
        # Five drafted tokens a sequence, scored in one call, one key head for each query head.
        dict(name="chunk_5_drafted", kind="chunk", B=24, new_lo=5, new_hi=5, old_lo=100, old_hi=4000, lens=6,
             Hq=16, Hkv=16, block=32, window=0, dtype="bf16"),
        # Ragged chunks (single tokens among prompt pieces) under a sliding window, float16.
        dict(name="chunk_ragged_window", kind="chunk", B=17, new_lo=1, new_hi=509, old_lo=0, old_hi=4000, lens=7,
             Hq=32, Hkv=8, block=16, window=1024, dtype="fp16"),
        # A 2048-token piece of a 16K prompt: bound by the tensor cores.
        dict(name="chunk_prompt_16k", kind="chunk", B=1, new_lo=2048, new_hi=2048, old_lo=14336, old_hi=14336,
             lens=8, Hq=32, Hkv=8, block=16, window=0, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rows", "train", "append", "append", "chunk", "chunk", "chunk"])
    c = dict(kind=kind)
    Hkv = rng.choice([1, 2, 4, 8, 16])
    c["Hkv"], c["Hq"] = Hkv, Hkv * rng.choice([1, 2, 3, 4, 7, 8])
    if kind in ("rows", "train"):
        c["d"] = rng.choice([64, 128])
        c["rot"] = 16 * rng.randint(1, c["d"] // 16)
        c["inter"], c["norm"] = rng.random() < 0.5, rng.random() < 0.75
        c["dtype"] = rng.choice(["bf16", "fp16", "fp32"])
        rows = _log_int(rng, 1, 16384 * 40 // (c["Hq"] + Hkv) // (2 if c["dtype"] == "fp32" else 1) // 2)
        if kind == "rows":
            c["T"] = rows
        else:
            c["B"] = rng.randint(1, 4)
            c["N"] = max(1, rows // c["B"])
        return c
    c["lens"] = rng.randrange(1 << 30)
    c["block"] = rng.choice([8, 16, 32, 64, 128, 256])
    c["dtype"] = rng.choice(["bf16", "fp16"])
    if kind == "append":
        c["rot"] = 16 * rng.randint(1, 8)
        c["inter"], c["norm"], c["with_q"] = rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5
        c["B"] = _log_int(rng, 1, 64)
        c["new_lo"] = 1
        c["new_hi"] = _log_int(rng, 1, max(1, 16384 * 32 // (c["Hq"] + 2 * Hkv) // c["B"]))
        c["old_lo"], c["old_hi"] = 0, _log_int(rng, 1, 1000)
        return c
    c["B"] = _log_int(rng, 1, 64)
    # ... and reads no more cache than the largest listed one.
    c["old_lo"], c["old_hi"] = 0, _log_int(rng, 16, min(16384, 2000000 // (c["B"] * Hkv)))
    c["new_lo"] = 1
    # A drawn chunk computes at most a quarter of the largest listed one, as if every chunk were the longest.
    most = 2048 * 16384 * 32 // 4 // (c["B"] * c["Hq"] * (c["old_hi"] + 1))
    c["new_hi"] = _log_int(rng, 1, max(1, min(1024, most)))
    c["window"] = rng.choice([0, 0, _log_int(rng, 1, 4096)])
    return c


def _lengths(c):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    r = random.Random(c["lens"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    return new, [n + r.randint(c["old_lo"], c["old_hi"]) for n in new]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, dtype, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _table(rows, rot):
    """cos | sin of position * base^(-2 i / rot), angles in 64 bits, kept as float32 [rows, rot]."""
    inv = _BASE ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _weight(g, dtype, d):
    return (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype)


def _paged(c, g, dtype):
    """Pools with every sequence's blocks in random places, the block table and the lengths."""
    new, total = _lengths(c)
    blocks = [-(-n // c["block"]) for n in total]
    perm = torch.randperm(sum(blocks), generator=g, device="cuda").int()
    table = torch.full((c["B"], max(blocks)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    pools = [_randn(g, dtype, sum(blocks), c["Hkv"], c["block"], 128) for _ in range(2)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return dict(kpool=pools[0], vpool=pools[1], table=table, T=cu[-1], max_new=max(new), max_len=max(total),
                cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                lens=torch.tensor(total, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    c, g = case, _gen(seed)
    dtype = _TYPES[c["dtype"]]
    s = dict(case=c)
    Hq, Hkv = c["Hq"], c["Hkv"]
    if c["kind"] == "rows":
        x = _randn(g, dtype, c["T"], Hq + 2 * Hkv, c["d"])
        s.update(q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], qw=_weight(g, dtype, c["d"]), kw=_weight(g, dtype, c["d"]),
                 rope=_table(8192, c["rot"]),
                 pos=torch.randint(0, 8192, (c["T"],), generator=g, device="cuda", dtype=torch.int32))
    elif c["kind"] == "train":
        # [B, N, H, d] as the projections leave it; the gradients come as attention's backward writes them.
        s.update(q=_randn(g, dtype, c["B"], c["N"], Hq, c["d"]).transpose(1, 2),
                 k=_randn(g, dtype, c["B"], c["N"], Hkv, c["d"]).transpose(1, 2),
                 dq=_randn(g, dtype, c["B"], Hq, c["N"], c["d"]), dk=_randn(g, dtype, c["B"], Hkv, c["N"], c["d"]),
                 qw=_weight(g, dtype, c["d"]), kw=_weight(g, dtype, c["d"]), rope=_table(c["N"], c["rot"]))
    else:
        s.update(_paged(c, g, dtype))
        if c["kind"] == "append":
            x = _randn(g, dtype, s["T"], Hq + 2 * Hkv, 128)
            s.update(q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], qw=_weight(g, dtype, 128),
                     kw=_weight(g, dtype, 128), rope=_table(s["max_len"], c["rot"]))
        else:
            s.update(q=_randn(g, dtype, s["T"], Hq, 128))
    if "norm" in c and not c["norm"]:
        s.update(qw=None, kw=None)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _RUN[s["case"]["kind"]](s)


def _eps(c):
    return _EPS if c["norm"] else None


def _run_rows(s):
    c = s["case"]
    if own:
        import tiled_exact_attention_forward_b200 as fa

        return fa.norm_rope(s["q"], s["k"], s["qw"], s["kw"], rope=s["rope"], positions=s["pos"], eps=_eps(c),
                            interleaved=c["inter"])
    pos = s["pos"].long()
    return [_norm_rotate(s[x], s[x + "w"], s["rope"][pos][:, None], c).to(s[x].dtype) for x in "qk"]


def _run_train(s):
    c = s["case"]
    if own:
        import tiled_exact_attention_forward_b200 as fa

        y = fa.norm_rope(s["q"], s["k"], s["qw"], s["kw"], rope=s["rope"], eps=_eps(c), interleaved=c["inter"])
        return y, fa.norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], s["qw"], s["kw"], rope=s["rope"],
                                        eps=_eps(c), interleaved=c["inter"])
    y = [_norm_rotate(s[x], s[x + "w"], s["rope"], c).to(s[x].dtype) for x in "qk"]
    (dq, dqw), (dk, dkw) = [_norm_rotate_grads(s[x], s["d" + x], s[x + "w"], s["rope"], c) for x in "qk"]
    return y, (dq, dk, dqw, dkw)


def _run_append(s):
    c = s["case"]
    if own:
        import tiled_exact_attention_forward_b200 as fa

        q = fa.append_paged(s["k"], s["v"], s["kpool"], s["vpool"], s["table"], s["lens"], cu_tokens=s["cu"],
                            rope=s["rope"], q=s["q"] if c["with_q"] else None, q_weight=s["qw"], k_weight=s["kw"],
                            eps=_eps(c), interleaved=c["inter"])
        return q, s["kpool"], s["vpool"]
    seq, at = _places(s)
    block = s["table"][seq, at // c["block"]].long()
    rope = s["rope"][at][:, None]
    s["kpool"][block, :, at % c["block"]] = _norm_rotate(s["k"], s["kw"], rope, c).to(s["k"].dtype)
    s["vpool"][block, :, at % c["block"]] = s["v"]
    q = _norm_rotate(s["q"], s["qw"], rope, c).to(s["q"].dtype) if c["with_q"] else None
    return q, s["kpool"], s["vpool"]


def _run_chunk(s):
    c = s["case"]
    if own:
        import tiled_exact_attention_forward_b200 as fa

        return fa.extend_paged(s["q"], s["kpool"], s["vpool"], s["table"], s["lens"], cu_tokens=s["cu"], causal=True,
                               window=c["window"])
    return _attend(s)


_RUN = dict(rows=_run_rows, train=_run_train, append=_run_append, chunk=_run_chunk)


# ------------------------------------------------------------------ plain forms

def _places(s):
    """Sequence and position of each packed token."""
    t = torch.arange(s["T"], device="cuda")
    cu, lens = s["cu"].long(), s["lens"].long()
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    return seq, lens[seq] - cu[seq + 1] + t


def _rotate(y, rope, inter, sign=1.0):
    """y's first rot elements turned by the table's angles (by their opposites for sign = -1)."""
    rot = rope.shape[-1]
    c, sn = rope[..., :rot // 2], rope[..., rot // 2:] * sign
    if inter:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([z, y[..., rot:]], -1)


def _norm_rotate(x, w, rope, c):
    y = x.float()
    if c["norm"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS) * w.float()
    return _rotate(y, rope, c["inter"])


def _norm_rotate_grads(x, dz, w, rope, c):
    """Gradients of the input (laid out as the input) and of the weight, summed in 64 bits."""
    g = _rotate(dz.float(), rope, c["inter"], -1.0)
    if not c["norm"]:
        return g.to(x.dtype), None
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + _EPS)
    xh = xf * r
    u = g * w.float()
    dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * xh).sum((0, 1, 2), dtype=torch.float64).to(w.dtype)


def _cached(pool, table, n):
    """A pool's rows in the sequences' own order: [B, H, n, d] in 32 bits."""
    x = pool[table.clamp(min=0).long()].transpose(1, 2)
    return x.flatten(2, 3)[:, :, :n].float()


def _attend(s):
    c = s["case"]
    B, Hkv, G = c["B"], c["Hkv"], c["Hq"] // c["Hkv"]
    n, mq = s["max_len"], s["max_new"]
    cu, lens = s["cu"].long(), s["lens"].long()
    k, v = _cached(s["kpool"], s["table"], n), _cached(s["vpool"], s["table"], n)
    at = (cu[:-1, None] + torch.arange(mq, device="cuda")).clamp(max=s["T"] - 1)
    q = s["q"][at].float().view(B, mq, Hkv, G, 128).transpose(1, 2).flatten(2, 3)
    x = q @ k.transpose(-1, -2) / math.sqrt(128.0)
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(mq, device="cuda")
    j = torch.arange(n, device="cuda")
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    x = x.view(B, Hkv, mq, G, n).masked_fill(~seen[:, None, :, None], -math.inf).flatten(2, 3)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (x - m).exp()
    z = p.sum(-1, keepdim=True)
    o = (p @ v) / z
    lse = m + z.log()
    seq, place = _places(s)
    i = place - pos[seq, 0]
    o = o.view(B, Hkv, mq, G, 128)[seq, :, i].flatten(1, 2)
    lse = lse.view(B, Hkv, mq, G)[seq, :, i].flatten(1, 2)
    return o.to(s["q"].dtype), lse


# ------------------------------------------------------------------ what a pass cannot do without

def _visible(c):
    """(key positions that some row sees, query-key pairs), over all sequences."""
    keys = pairs = 0
    for new, total in zip(*_lengths(c)):
        w = c["window"] or total
        keys += min(total, new + w - 1)
        first = total - new + 1  # keys that the first new token may see
        full = max(0, min(new, total - max(first, w) + 1))
        short = new - full
        pairs += full * w + short * first + short * (short - 1) // 2 if w < total else \
            new * first + new * (new - 1) // 2
    return keys, pairs


def work(case):
    c = case
    e = 4 if c["dtype"] == "fp32" else 2
    if c["kind"] in ("rows", "train"):
        rows = c["T"] if c["kind"] == "rows" else c["B"] * c["N"]
        x = rows * (c["Hq"] + c["Hkv"]) * c["d"]
        table = min(rows, 8192) * c["rot"] * 4 if c["kind"] == "rows" else c["N"] * c["rot"] * 4
        if c["kind"] == "rows":
            return dict(bytes=2 * x * e + table, flops=8 * x)
        # Forward: x in, y out.  Backward: dy in, dx out (x and the table are read already).
        return dict(bytes=4 * x * e + table, flops=24 * x)
    new, total = _lengths(c)
    T = sum(new)
    if c["kind"] == "append":
        x = T * (2 * c["Hkv"] + (c["Hq"] if c["with_q"] else 0)) * 128
        return dict(bytes=2 * x * e + T * c["rot"] * 4, flops=8 * x)
    keys, pairs = _visible(c)
    return dict(bytes=2 * keys * c["Hkv"] * 128 * e + T * c["Hq"] * (2 * 128 * e + 4), flops=4 * 128 * pairs * c["Hq"])


# ------------------------------------------------------------------ exact values

def _pairs64(c, rot):
    i = torch.arange(rot // 2, device="cuda")
    return (2 * i, 2 * i + 1) if c["inter"] else (i, i + rot // 2)


def _turn64(y, rope, c, back=False):
    rot = rope.shape[-1]
    a, b = _pairs64(c, rot)
    angle_c, angle_s = rope[..., :rot // 2].double(), rope[..., rot // 2:].double()
    if back:
        angle_s = -angle_s
    z = y.clone()
    z[..., a] = y[..., a] * angle_c - y[..., b] * angle_s
    z[..., b] = y[..., a] * angle_s + y[..., b] * angle_c
    return z


def _forward64(x, w, rope, c):
    x = x.double()
    if c["norm"]:
        x = w.double() * x / (x.pow(2).mean(-1, keepdim=True) + _EPS).sqrt()
    return _turn64(x, rope, c)


def _grads64(x, dz, w, rope, c):
    """By the chain rule through y = w x / s, s = sqrt(mean x^2 + eps)."""
    x, g = x.double(), _turn64(dz.double(), rope, c, back=True)
    if not c["norm"]:
        return g, None
    sd = (x.pow(2).mean(-1, keepdim=True) + _EPS).sqrt()
    gw = g * w.double()
    dx = gw / sd - x * (gw * x).sum(-1, keepdim=True) / (x.shape[-1] * sd.pow(3))
    return dx, (g * x / sd).sum((0, 1, 2))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "rows":
        rope = s["rope"][s["pos"].long()][:, None]
        return [_forward64(s["q"], s["qw"], rope, c), _forward64(s["k"], s["kw"], rope, c)]
    if c["kind"] == "train":
        dq, dqw = _grads64(s["q"], s["dq"], s["qw"], s["rope"], c)
        dk, dkw = _grads64(s["k"], s["dk"], s["kw"], s["rope"], c)
        y = [_forward64(s["q"], s["qw"], s["rope"], c), _forward64(s["k"], s["kw"], s["rope"], c)]
        return y, (dq, dk, dqw, dkw)
    new, total = _lengths(c)
    if c["kind"] == "append":
        pools = [s["kpool"].double(), s["vpool"].double()]
        out = s["q"].double().clone() if c["with_q"] else None
        t = 0
        for b in range(c["B"]):
            at = torch.arange(total[b] - new[b], total[b], device="cuda")
            blk, off, rope = s["table"][b].long()[at // c["block"]], at % c["block"], s["rope"][at][:, None]
            pools[0][blk, :, off] = _forward64(s["k"][t:t + new[b]], s["kw"], rope, c)
            pools[1][blk, :, off] = s["v"][t:t + new[b]].double()
            if out is not None:
                out[t:t + new[b]] = _forward64(s["q"][t:t + new[b]], s["qw"], rope, c)
            t += new[b]
        return out, pools[0], pools[1]
    G = c["Hq"] // c["Hkv"]
    o = torch.empty(s["T"], c["Hq"], 128, device="cuda", dtype=torch.float64)
    lse = torch.empty(s["T"], c["Hq"], device="cuda", dtype=torch.float64)
    t = 0
    for b in range(c["B"]):
        n = total[b]
        j = torch.arange(n, device="cuda")
        place = torch.arange(n - new[b], n, device="cuda")[:, None]
        hidden = j > place
        if c["window"]:
            hidden |= j <= place - c["window"]
        blk, off = s["table"][b].long()[j // c["block"]], j % c["block"]
        for h in range(c["Hkv"]):
            k, v = s["kpool"][blk, h, off].double(), s["vpool"][blk, h, off].double()
            q = s["q"][t:t + new[b], h * G:(h + 1) * G].double().transpose(0, 1)
            x = (q @ k.T / 128.0 ** 0.5).masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[t:t + new[b], h * G:(h + 1) * G] = z.T
            o[t:t + new[b], h * G:(h + 1) * G] = ((x - z[..., None]).exp() @ v).transpose(0, 1)
        t += new[b]
    return o, lse
