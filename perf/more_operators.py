"""Cases and plain forms of the operators that keep long and shared contexts in a block-scaled FP8 cache.

Four operators around a paged e4m3 pool whose every block of 16 tokens has a power-of-two scale per
KV head for K and one for V:

  axes    ``kv_rope_cache`` and ``kv_block_cache`` with rotary positions of several axes (time, height and
          width of image and video tokens), each rotated pair turned by its own axis's position, the
          positions given token by token.
  shared  ``fp8_block_shared_decode_attn``: one query per sequence; sequences of a group have the first
          tokens of their contexts in common, and the attention over those is computed for the group at once.
  weights ``fp8_block_attn_weights``: the attention weight that every cached key receives from a chunk of
          queries, summed over the queries and the heads of its group, added to what it received before.
  evict   ``kv_block_evict``: every KV head of a sequence keeps its first and last tokens and, of the others,
          those with the most weight; what is kept is copied to new blocks with new scales.

``run`` computes a case's operator either in its plain form (elementary torch operations, float32) or,
with ``own`` true, through the library's binding.
"""
import math

import torch

own = False

BLOCK = 16                 # tokens of a pool block
E4M3_MAX, E5M2_MAX = 448.0, 57344.0
MAX_POSITIONS = 131072     # rows of the rotary table


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # ---- axes
        # one decode step of 8 sequences (one layer of the Llama-3.1-8B-shaped model) behind prompts with
        # images, whose positions are not their places in the cache: latency, blocks that continue
        dict(name="axes append step", op="axes", form="append", batch=8, new_lo=1, new_hi=1, ctx_lo=16384, ctx_hi=24576,
             q_heads=32, kv_heads=8, head_dim=128, sections="16,24,24", assign="runs", style="half"),
        # a padded batch of text and image tokens of a layer kept in bf16, gpt-oss-20b-shaped heads
        dict(name="axes image tokens bf16", op="axes", form="slots", tokens=9001, pad=41, q_heads=64, kv_heads=8, head_dim=64,
             sections="12,10,10", assign="turns", style="half", pool="bf16"),
        # four long prompts with images, appended block by block
        dict(name="axes append fill", op="axes", form="append", batch=4, new_lo=12001, new_hi=16384, ctx_lo=16384, ctx_hi=16384,
             q_heads=32, kv_heads=8, head_dim=128, sections="16,24,24", assign="runs", style="half"),
        # ---- shared
        # four answers sampled from one prompt: latency
        dict(name="shared 4 x 2k", op="shared", groups="4", prefix="2048", own_lo=1, own_hi=150, q_heads=32, kv_heads=8,
             head_dim=128, window=0),
        # 32 requests behind one long document
        dict(name="shared 32 x 32k", op="shared", groups="32", prefix="32768", own_lo=16, own_hi=1024, q_heads=32, kv_heads=8,
             head_dim=128, window=0),
        # two system prompts of odd lengths and their requests, gpt-oss-20b-shaped heads
        dict(name="shared two prompts d64", op="shared", groups="13,43", prefix="8195,5000", own_lo=1, own_hi=2000, q_heads=64,
             kv_heads=8, head_dim=64, window=0),
        # ---- weights
        # one decode step under load, one layer: what each key of 8 long contexts received is added up
        dict(name="weights step", op="weights", batch=8, new_lo=1, new_hi=1, ctx_lo=16384, ctx_hi=24576, q_heads=32, kv_heads=8,
             head_dim=128, decay=1.0),
        # the last 32 queries of four prompts tell which of their keys matter
        dict(name="weights window", op="weights", batch=4, new_lo=32, new_hi=32, ctx_lo=7001, ctx_hi=16384, q_heads=32,
             kv_heads=8, head_dim=128, decay=0.0),
        # a whole prompt of odd length, every query of it, head_dim 256
        dict(name="weights prompt d256", op="weights", batch=1, new_lo=4001, new_hi=4001, ctx_lo=4001, ctx_hi=4001, q_heads=8,
             kv_heads=1, head_dim=256, decay=0.0),
        # ---- evict
        # two short contexts: latency
        dict(name="evict 2 x 1.5k", op="evict", batch=2, ctx_lo=1311, ctx_hi=1500, budget=512, sink=4, recent=64, kv_heads=8,
             head_dim=128),
        # the contexts of a loaded decode cut to a sixth
        dict(name="evict 8 x 16k-24k", op="evict", batch=8, ctx_lo=16384, ctx_hi=24576, budget=4096, sink=4, recent=512,
             kv_heads=8, head_dim=128),
        # one context of 131,072 tokens (the longest workload) cut to a quarter
        dict(name="evict 131k", op="evict", batch=1, ctx_lo=131072, ctx_hi=131072, budget=32768, sink=16, recent=1024,
             kv_heads=8, head_dim=128),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _cut(rng, total, parts):
    """`total` as a sum of `parts` positive numbers, as text."""
    at = sorted(rng.sample(range(1, total), parts - 1))
    return ",".join(str(b - a) for a, b in zip([0] + at, at + [total]))


def draw(rng):
    op = rng.choice(("axes", "shared", "weights", "evict"))
    most = [work(c) for c in listed() if c["op"] == op]
    while True:
        case = _drawn(rng, op)
        if all(work(case)[x] <= max(m[x] for m in most) for x in ("bytes", "flops")):
            return case


def _drawn(rng, op):
    head_dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 4, 8, 16) if head_dim <= 128 else (1, 2, 4, 8))
    if group * kv_heads > 64:
        kv_heads = 64 // group
    heads = dict(q_heads=group * kv_heads, kv_heads=kv_heads, head_dim=head_dim)
    if op == "axes":
        rot = rng.choice([r for r in (32, 64, 96, 128, 256) if r <= head_dim])
        how = dict(sections=_cut(rng, rot // 2, rng.choice((1, 2, 3, 3, 4))), assign=rng.choice(("runs", "turns")),
                   style=rng.choice(("half", "pairs")))
        most = min(65536, 65536 * 6144 // ((group + 2) * kv_heads * head_dim))          # tokens of the largest case's elements
        if rng.random() < 0.5:
            tokens = _log(rng, 1, most)
            return dict(op=op, form="slots", tokens=tokens, pad=rng.choice((0, 0, tokens // 7)),
                        pool=rng.choice(("e4m3", "bf16", "e5m2")), **heads, **how)
        batch = _log(rng, 1, 32)
        new_hi = _log(rng, 1, min(16384, most // batch))
        before = _log(rng, 1, 16384) - 1
        return dict(op=op, form="append", batch=batch, new_lo=rng.choice((1, (new_hi + 1) // 2, new_hi)), new_hi=new_hi,
                    ctx_lo=new_hi + before // 2, ctx_hi=new_hi + before, **heads, **how)
    if op == "shared":
        sizes = [_log(rng, 1, 64) for _ in range(rng.choice((1, 1, 2, 3)))]
        prefix = [_log(rng, 1, 32768 // len(sizes)) for _ in sizes]
        own_hi = _log(rng, 1, 4096)
        return dict(op=op, groups=",".join(map(str, sizes)), prefix=",".join(map(str, prefix)),
                    own_lo=rng.choice((0, own_hi // 3, own_hi)), own_hi=own_hi, window=rng.choice((0, 0, 0, _log(rng, 1, 8192))),
                    **heads)
    if op == "weights":
        while True:
            batch = _log(rng, 1, 16)
            new_hi = rng.choice((1, _log(rng, 1, 64), _log(rng, 1, 4096)))
            ctx_hi = new_hi + _log(rng, 1, 32768) - 1
            if batch * heads["q_heads"] * new_hi * ctx_hi <= 1 << 27:
                break
        return dict(op=op, batch=batch, new_lo=rng.choice((1, (new_hi + 1) // 2, new_hi)), new_hi=new_hi,
                    ctx_lo=(new_hi + ctx_hi) // 2, ctx_hi=ctx_hi, decay=rng.choice((0.0, 1.0, 0.875)), **heads)
    batch = _log(rng, 1, 32)
    ctx_hi = _log(rng, 1, 131072)
    budget = _log(rng, 1, ctx_hi)
    sink = rng.choice((0, min(4, budget)))
    return dict(op=op, batch=batch, ctx_lo=rng.choice((1, (ctx_hi + 1) // 2, ctx_hi)), ctx_hi=ctx_hi, budget=budget, sink=sink,
                recent=rng.choice((0, (budget - sink) // 5, budget - sink)), kv_heads=kv_heads, head_dim=head_dim)


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], the last of them hi, in an order without a pattern."""
    return [lo + int((hi - lo) * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(n - 1)] + [hi]


def _lens(c):
    """(new tokens, context lengths with the new tokens) of an append's or a weights case's sequences."""
    return _spread(c["new_lo"], c["new_hi"], c["batch"]), _spread(c["ctx_lo"], c["ctx_hi"], c["batch"])


def _ints(text):
    return [int(x) for x in text.split(",")]


def _pair_axes(c):
    """The axis of each rotated pair: the sections one after another, or dealt out in turns while they last."""
    n = _ints(c["sections"])
    if c["assign"] == "runs":
        return [a for a, m in enumerate(n) for _ in range(m)]
    return [a for turn in range(max(n)) for a, m in enumerate(n) if turn < m]


def _shared_lens(c):
    """(sequences of the groups, shared tokens of the groups, context lengths of the sequences)."""
    sizes, prefix = _ints(c["groups"]), _ints(c["prefix"])
    mine = _spread(c["own_lo"], c["own_hi"], sum(sizes))
    first = [p for p, n in zip(prefix, sizes) for _ in range(n)]
    return sizes, prefix, [a + b for a, b in zip(first, mine)]


# --------------------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _codes(g, shape):
    """Bytes left in a pool by earlier use: any e4m3 code."""
    return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)


def _int(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _fused(g, tokens, c):
    """The new tokens' q, k and v as slices of one projection's output, with K outlier channels."""
    hq, h, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    qkv = _randn(g, tokens, (hq + 2 * h) * d)
    k = qkv[:, hq * d:(hq + h) * d].view(tokens, h, d)
    k[:, :, torch.randperm(d, generator=g, device="cuda")[:4]] *= 8.0
    qkv = qkv.to(torch.bfloat16)
    return (qkv[:, :hq * d].view(tokens, hq, d), qkv[:, hq * d:(hq + h) * d].view(tokens, h, d),
            qkv[:, (hq + h) * d:].view(tokens, h, d))


def _table(rot_dim):
    """[position][rot_dim]: rot_dim / 2 cosines, then the sines."""
    inv = 500000.0 ** (-torch.arange(0, rot_dim, 2, device="cuda", dtype=torch.float64) / rot_dim)
    a = torch.arange(MAX_POSITIONS, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def _image_positions(g, tokens, axes):
    """Text tokens, whose axes count alike, and images of 7 rows of up to 9 patches among them."""
    at = torch.arange(tokens, device="cuda")
    start = torch.randint(0, MAX_POSITIONS - tokens - 16, (1,), generator=g, device="cuda")
    image = (at // 63) % 3 == 1
    in_image = torch.stack((torch.zeros_like(at), (at % 63) // 9, at % 9, at % 5))[:axes]
    return torch.where(image, start + at - at % 63 + in_image, (start + at).expand(axes, -1)).contiguous()


def _pages(g, lens):
    """A block table over sequences of `lens` tokens (a shuffled pool, unused entries -1) and the pool's blocks."""
    n = [(t + BLOCK - 1) // BLOCK for t in lens]
    perm = torch.randperm(sum(n) + 3, generator=g, device="cuda").to(torch.int32)
    tab = torch.full((len(n), max(1, *n)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(n):
        tab[i, :m] = perm[at:at + m]
        at += m
    return tab, sum(n) + 3


def _pow2_scale(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(amax > 0, torch.where(m > 0.875, e - 8, e - 9), -126).clamp(min=-126)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _block_pool(g, num_blocks, c):
    """K and V codes and scales of blocks filled from N(0, 1) tokens, K with outlier channels, V of
    differing size from block to block."""
    h, d = c["kv_heads"], c["head_dim"]
    pools = []
    for kind in range(2):
        x = _randn(g, num_blocks, h, BLOCK, d)
        if kind == 0:
            x[..., torch.randperm(d, generator=g, device="cuda")[:4]] *= 8.0
        else:
            x *= torch.exp2(_randn(g, num_blocks, h, 1, 1))
        s = _pow2_scale(x.abs().amax((2, 3)))
        pools += [(x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s]
    return pools[0], pools[2], pools[1], pools[3]


def _stale(g, s):
    """Whatever earlier use left behind each sequence's last token: any code, NaN among them."""
    for t, row in zip(s["lens"], s["table"]):
        if t % BLOCK:
            for pool in (s["k_pool"], s["v_pool"]):
                tail = pool[row[t // BLOCK].item(), :, t % BLOCK:]
                tail.copy_(_codes(g, tail.shape))


def _prepare_slots(s, g, c):
    h, d, n = c["kv_heads"], c["head_dim"], c["tokens"]
    nb = (n + BLOCK - 1) // BLOCK + 3
    slots = torch.randperm(nb, generator=g, device="cuda")[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    s["slots"] = slots.reshape(-1)[:n].contiguous()
    if c["pad"]:
        s["slots"][n - c["pad"]:] = -1
    shape = (nb, h, BLOCK, d)
    if c["pool"] == "bf16":
        s["k_pool"], s["v_pool"] = _randn(g, *shape).to(torch.bfloat16), _randn(g, *shape).to(torch.bfloat16)
        s["k_scale"] = s["v_scale"] = None
    else:
        # finite codes only, so that untouched rows compare
        s["k_pool"], s["v_pool"] = _codes(g, shape) & 0x7B, _codes(g, shape) & 0x7B
        top = E4M3_MAX if c["pool"] == "e4m3" else E5M2_MAX
        s["k_scale"] = s["k"].abs().amax((0, 2)).float() / top
        s["v_scale"] = s["v"].abs().amax((0, 2)).float() / top


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    h, d = c["kv_heads"], c["head_dim"]
    if c["op"] == "axes":
        slots = c["form"] == "slots"
        new, s["lens"] = ([c["tokens"]], None) if slots else _lens(c)
        n = sum(new)
        s["pair_axes"] = _pair_axes(c)
        s["q"], s["k"], s["v"] = _fused(g, n, c)
        s["positions"] = _image_positions(g, n, 1 + max(s["pair_axes"]))
        s["cos_sin"] = _table(2 * len(s["pair_axes"]))
        s["q_out"] = torch.zeros(n, c["q_heads"], d, dtype=torch.bfloat16, device="cuda")
        if slots:
            _prepare_slots(s, g, c)
            return s
    elif c["op"] == "shared":
        sizes, prefix, s["lens"] = _shared_lens(c)
        new, starts = None, [sum(sizes[:i]) for i in range(len(sizes) + 1)]
        s["starts"], s["shared"], s["max_group"] = _int(starts), _int(prefix), max(sizes)
        s["q"] = _randn(g, sum(sizes), c["q_heads"], d).to(torch.bfloat16)
        # whole shared blocks are one sequence's; a block that the shared tokens end in is every sequence's own
        mine = [t - p // BLOCK * BLOCK for t, p in zip(s["lens"], [p for p, n in zip(prefix, sizes) for _ in range(n)])]
        tab, nb = _pages(g, [p // BLOCK * BLOCK for p in prefix] + mine)
        full = [p // BLOCK for p in prefix]
        s["table"] = torch.full((sum(sizes), max(1, *((t + BLOCK - 1) // BLOCK for t in s["lens"]))), -1, dtype=torch.int32, device="cuda")
        for i, n in enumerate(sizes):
            for b in range(starts[i], starts[i] + n):
                own_blocks = (mine[b] + BLOCK - 1) // BLOCK
                s["table"][b, :full[i]] = tab[i, :full[i]]
                s["table"][b, full[i]:full[i] + own_blocks] = tab[len(sizes) + b, :own_blocks]
        s["workspace"] = torch.zeros(96 << 20, dtype=torch.uint8, device="cuda")
    elif c["op"] == "weights":
        new, s["lens"] = _lens(c)
        s["q"] = _randn(g, sum(new), c["q_heads"], d).to(torch.bfloat16)
    else:
        new, s["lens"] = None, _spread(c["ctx_lo"], c["ctx_hi"], c["batch"])
    if c["op"] != "shared":
        keep = [min(t, c["budget"]) for t in s["lens"]] if c["op"] == "evict" else []
        tab, nb = _pages(g, s["lens"] + keep)
        s["table"] = tab[:len(s["lens"]), :max(1, (max(s["lens"]) + BLOCK - 1) // BLOCK)].contiguous()
        if c["op"] == "evict":
            s["new_table"] = tab[len(s["lens"]):, :(max(keep) + BLOCK - 1) // BLOCK].contiguous()
    s["ctx"] = _int(s["lens"])
    if new is not None:
        s["cu"], s["max_new"] = _int([sum(new[:i]) for i in range(len(new) + 1)]), max(new)
    s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _block_pool(g, nb, c)
    if c["op"] in ("weights", "evict"):
        # what the keys received so far, as after a few steps: far apart, and nothing for many of them
        w = 2e-4 * torch.exp(2 * _randn(g, c["batch"], h, s["table"].shape[1] * BLOCK))
        s["weights"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.1, 0.0, w)
    if c["op"] == "weights":
        _stale(g, s)
        small = 4 * c["batch"] * c["q_heads"] * s["max_new"] * s["weights"].shape[2] if s["max_new"] * c["q_heads"] // h <= 16 else 0
        s["workspace"] = torch.zeros((96 << 20) + small, dtype=torch.uint8, device="cuda")
    if c["op"] == "evict":
        s["new_weights"] = torch.zeros(c["batch"], h, s["new_table"].shape[1] * BLOCK, device="cuda")
        s["new_lens"] = torch.zeros(c["batch"], dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros(c["batch"], h, c["budget"], dtype=torch.int32, device="cuda")
        # the blocks to come hold finite codes, so that slots behind the kept tokens compare
        s["k_pool"][s["new_table"][s["new_table"] >= 0].long()] &= 0x7B
        s["v_pool"][s["new_table"][s["new_table"] >= 0].long()] &= 0x7B
    if c["op"] == "shared":
        for i, (p, n) in enumerate(zip(prefix, sizes)):    # shared tokens in the sequences' own blocks are copies
            ids = s["table"][starts[i]:starts[i] + n, p // BLOCK].long() if p % BLOCK else []
            for pool, scale in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])):
                for x in ids[1:]:
                    pool[x, :, :p % BLOCK], scale[x] = pool[ids[0], :, :p % BLOCK], scale[ids[0]]
        _stale(g, s)
    return s


# --------------------------------------------------------------------------- plain forms

def _rotate(x, cs, style):
    """x [tokens][heads][head_dim] float, cs [tokens][rot_dim]: the first rot_dim elements of each head
    rotated, as the pairs (i, i + rot_dim / 2) or the neighbours (2 i, 2 i + 1)."""
    r = cs.shape[1]
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    if style == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat((a * c - b * s, b * c + a * s, x[..., r:]), -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat((torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2), x[..., r:]), -1)


def _f8(pool, fmt="e4m3"):
    return pool.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2)


def _axes_rows(s):
    """[token][rot_dim]: pair i's cosine and sine at the position of its axis."""
    at = s["positions"][_int(s["pair_axes"] * 2, torch.int64)].T               # [token][rot_dim]
    return s["cos_sin"].gather(0, at)


def _slots_plain(s):
    c = s["case"]
    cs, keep = _axes_rows(s), s["slots"] >= 0
    q = _rotate(s["q"].float(), cs, c["style"]).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(keep[:, None, None], q, s["q_out"]))
    slot = s["slots"][keep]
    k, v = _rotate(s["k"].float(), cs, c["style"])[keep], s["v"].float()[keep]
    if c["pool"] == "bf16":
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    else:
        dt, top = (torch.float8_e4m3fn, E4M3_MAX) if c["pool"] == "e4m3" else (torch.float8_e5m2, E5M2_MAX)
        k = (k * (1 / s["k_scale"])[:, None]).clamp(-top, top).to(dt).view(torch.uint8)
        v = (v * (1 / s["v_scale"])[:, None]).clamp(-top, top).to(dt).view(torch.uint8)
    s["k_pool"][slot // BLOCK, :, slot % BLOCK] = k
    s["v_pool"][slot // BLOCK, :, slot % BLOCK] = v


def _append_plain(s, x, pool, scale):
    """x [token][head][head_dim] float into a block-scaled pool, at the ends of the sequences."""
    at = torch.arange(x.shape[0], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], at, right=True) - 1
    pos = (s["ctx"][seq] - s["cu"][seq + 1] + at).long()
    block, off = s["table"][seq, pos // BLOCK].long(), pos % BLOCK
    # the first new slot of every block; a block begun here keeps nothing
    start = torch.full((pool.shape[0],), BLOCK, dtype=torch.int64, device="cuda")
    start.scatter_reduce_(0, block, off, "amin")
    amax = torch.zeros_like(scale).index_reduce_(0, block, x.abs().amax(2), "amax")
    held = torch.where(start[:, None] > 0, scale, 0.0)
    grown = torch.where(start[:, None] < BLOCK, torch.maximum(held, _pow2_scale(amax)), scale)
    # tokens already in the block that each sequence continues
    first = torch.unique(block[off == start[block]])
    kept = (_f8(pool)[first].float() * (held / grown)[first][:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    old = torch.arange(BLOCK, device="cuda") < start[first][:, None]
    pool[first] = torch.where(old[:, None, :, None], kept, pool[first])
    pool[block, :, off] = (x / grown[block][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(grown)


def _axes_plain(s):
    style = s["case"]["style"]
    cs = _axes_rows(s)
    s["q_out"].copy_(_rotate(s["q"].float(), cs, style))
    _append_plain(s, _rotate(s["k"].float(), cs, style), s["k_pool"], s["k_scale"])
    _append_plain(s, s["v"].float(), s["v_pool"], s["v_scale"])


def _gathered(table, pool, scale):
    """[sequence][KV head][key][head_dim] values of a table's blocks (-1: whatever block 0 holds)."""
    tab = table.clamp(min=0).long()
    return (_f8(pool[tab]).float() * scale[tab][..., None, None]).transpose(1, 2).flatten(2, 3)


def _shared_plain(s):
    c = s["case"]
    b, hq, d = s["q"].shape
    h, m, sizes = c["kv_heads"], s["max_group"], s["starts"].diff()
    ng, tau = sizes.shape[0], 1 / math.sqrt(d)
    lo = (s["ctx"] - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(s["ctx"])
    group = torch.searchsorted(s["starts"], torch.arange(b, device="cuda", dtype=torch.int32), right=True) - 1
    place = torch.arange(b, device="cuda") - s["starts"][group]                # in its group
    shared = s["shared"][group]
    q = s["q"].float().view(b, h, hq // h, d)
    # the shared keys, once per group, for all of its rows
    blocks = (max(_ints(c["prefix"])) + BLOCK - 1) // BLOCK
    tab = s["table"][s["starts"][:-1].long(), :blocks]
    rows = torch.zeros(ng, m, h, hq // h, d, device="cuda")
    rows[group, place] = q
    x = rows.permute(0, 2, 1, 3, 4).flatten(2, 3) @ _gathered(tab, s["k_pool"], s["k_scale"]).mT
    x = x.view(ng, h, m, hq // h, -1)[group, :, place] * tau                   # [B][H][G][key]
    key = torch.arange(x.shape[-1], device="cuda")
    seen = (key < torch.minimum(shared, s["ctx"])[:, None]) & (key >= lo[:, None])
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    # every sequence's own keys
    first = s["shared"] // BLOCK
    at = first[group][:, None] + torch.arange(int(c["own_hi"] + 2 * BLOCK) // BLOCK, device="cuda")
    mine = s["table"].gather(1, at.clamp(max=s["table"].shape[1] - 1).long())
    pos = at.repeat_interleave(BLOCK, 1) * BLOCK + torch.arange(BLOCK, device="cuda").repeat(at.shape[1])
    live = (pos >= torch.maximum(shared, lo)[:, None]) & (pos < s["ctx"][:, None])
    y = (q @ _gathered(mine, s["k_pool"], s["k_scale"]).mT) * tau
    y = y.masked_fill_(~live[:, None, None], -math.inf)
    top = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True)).clamp_(min=-1e30)
    x, y = x.sub_(top).exp_(), y.sub_(top).exp_()
    total = (x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)).clamp_(min=1e-30)
    p = torch.zeros(ng, m, h, hq // h, x.shape[-1], device="cuda")
    p[group, place] = x
    v = _gathered(tab, s["v_pool"], s["v_scale"])
    v = v.masked_fill_((key >= s["shared"][:, None])[:, None, :, None], 0.0)
    o = (p.permute(0, 2, 1, 3, 4).flatten(2, 3) @ v).view(ng, h, m, hq // h, d)[group, :, place]
    v = _gathered(mine, s["v_pool"], s["v_scale"]).masked_fill_(~live[:, None, :, None], 0.0)
    return ((o + y @ v) / total).reshape(b, hq, d).to(torch.bfloat16)


def _weights_plain(s):
    c = s["case"]
    n, hq, d = s["q"].shape
    h, b, m = c["kv_heads"], c["batch"], s["max_new"]
    k = _gathered(s["table"], s["k_pool"], s["k_scale"])
    # the ragged queries padded to the longest chunk
    row = s["cu"][:-1, None] + torch.arange(m, device="cuda")
    real = row < s["cu"][1:, None]
    q = s["q"].float()[row.clamp(max=n - 1).long()]                             # [B][m][Hq][D]
    q = q.view(b, m, h, hq // h, d).permute(0, 2, 1, 3, 4).flatten(2, 3)        # rows: token, then head of the group
    pos = s["ctx"][:, None] - s["cu"][1:, None] + row                           # [B][m]
    key = torch.arange(k.shape[2], device="cuda")
    seen = (key <= pos[:, :, None]) & real[:, :, None]
    seen = seen.repeat_interleave(hq // h, 1)[:, None]
    p = (q @ k.mT).mul_(1 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    p = (p / p.sum(-1, keepdim=True).clamp_(min=1e-30)).sum(2)                  # [B][H][key]
    old = key < (s["ctx"] - s["cu"].diff())[:, None]
    before = s["weights"] * c["decay"] if c["decay"] else torch.zeros_like(s["weights"])
    live = (key < s["ctx"][:, None])[:, None]
    s["weights"].copy_(torch.where(live, p + torch.where(old[:, None], before, 0.0), s["weights"]))
    return s["weights"]


def _recode(x):
    """[sequence][KV head][token][head_dim] values, whole blocks of them, as codes [..][block][16][D] and scales [..][block]."""
    x = x.unflatten(2, (-1, BLOCK))
    scale = _pow2_scale(x.abs().amax((3, 4)))
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _evict_plain(s):
    c = s["case"]
    b, h, keys = s["weights"].shape
    ctx, key = s["ctx"][:, None], torch.arange(keys, device="cuda")
    n = s["ctx"].clamp(max=c["budget"])
    always = (key < c["sink"]) | (key >= ctx - c["recent"])
    rank = torch.where(always[:, None], math.inf, s["weights"]).masked_fill((key >= ctx)[:, None], -math.inf)
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices
    room = s["new_table"].shape[1] * BLOCK
    wide = torch.nn.functional.pad(order, (0, max(0, room - keys)))[:, :, :room]
    live = torch.arange(room, device="cuda") < n[:, None]                       # [B][room]
    kept = torch.where(live[:, None], wide, keys).sort(2).values
    src = kept.clamp(max=keys - 1)
    kept32 = torch.where(live[:, None], kept, -1).to(torch.int32)
    s["kept"].copy_(torch.nn.functional.pad(kept32, (0, max(0, c["budget"] - room)), value=-1)[:, :, :c["budget"]])
    s["new_weights"].copy_(torch.where(live[:, None], s["weights"].gather(2, src), s["new_weights"]))
    s["new_lens"].copy_(n)
    block = s["table"].long()[torch.arange(b, device="cuda")[:, None, None], src // BLOCK].clamp(min=0)
    head = torch.arange(h, device="cuda")[:, None]
    live16 = live.unflatten(1, (-1, BLOCK))                                     # [B][block][16]
    used = live16.any(2)
    dst = s["new_table"][used].long()
    codes, scale = _recode((_f8(s["k_pool"][block, head, src % BLOCK]).float() * s["k_scale"][block, head][..., None])
                           .masked_fill(~live[:, None, :, None], 0.0))
    keep = live16[used][:, None, :, None]
    s["k_pool"][dst] = torch.where(keep, codes.transpose(1, 2)[used], s["k_pool"][dst])
    s["k_scale"][dst] = scale.transpose(1, 2)[used]
    codes, scale = _recode((_f8(s["v_pool"][block, head, src % BLOCK]).float() * s["v_scale"][block, head][..., None])
                           .masked_fill(~live[:, None, :, None], 0.0))
    s["v_pool"][dst] = torch.where(keep, codes.transpose(1, 2)[used], s["v_pool"][dst])
    s["v_scale"][dst] = scale.transpose(1, 2)[used]


# --------------------------------------------------------------------------- a pass

def _run_own(s):
    import fp8_kv_cache_quant_gb300 as f
    c = s["case"]
    if c["op"] == "axes":
        if "rope" not in s:    # a program keeps it
            s["rope"] = f.Rope(s["cos_sin"], interleaved=c["style"] == "pairs", axes=s["pair_axes"])
        if c["form"] == "slots":
            cache = f.LayerCache(s["k_pool"], s["v_pool"], f.KV_E5M2 if c["pool"] == "e5m2" else f.KV_E4M3)
            f.kv_rope_cache(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"], cache, s["k_scale"], s["v_scale"],
                            gran=f.SCALE_PER_HEAD, skip_layer_mask=[1] if c["pool"] == "bf16" else None, q_out=s["q_out"])
            return
    cache = f.BlockCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
    if c["op"] == "axes":
        f.kv_block_cache(s["k"], s["v"], s["cu"], s["max_new"], cache, s["table"], s["ctx"], rope=s["rope"], q=s["q"],
                         q_out=s["q_out"], positions=s["positions"])
    elif c["op"] == "shared":
        return f.fp8_block_shared_decode_attn(s["q"], cache, s["table"], s["ctx"], s["starts"], s["shared"],
                                              window=c["window"], workspace=s["workspace"])
    elif c["op"] == "weights":
        return f.fp8_block_attn_weights(s["q"], s["cu"], s["max_new"], cache, s["table"], s["ctx"], s["weights"],
                                        decay=c["decay"], workspace=s["workspace"])
    else:
        f.kv_block_evict(cache, s["table"], s["ctx"], s["weights"], c["budget"], s["new_table"], sink=c["sink"],
                         recent=c["recent"], new_weights=s["new_weights"], new_lens=s["new_lens"], kept=s["kept"])


def run(state):
    s, c = state, state["case"]
    if own:
        out = _run_own(s)
    elif c["op"] == "axes":
        out = _slots_plain(s) if c["form"] == "slots" else _axes_plain(s)
    elif c["op"] == "shared":
        out = _shared_plain(s)
    elif c["op"] == "weights":
        out = _weights_plain(s)
    else:
        out = _evict_plain(s)
    if c["op"] in ("shared", "weights"):
        return out
    if c["op"] == "axes" and c["form"] == "slots":
        bf16 = c["pool"] == "bf16"
        return {"q": s["q_out"], "k_pool": s["k_pool"] if bf16 else _f8(s["k_pool"], c["pool"]),
                "v_pool": s["v_pool"] if bf16 else _f8(s["v_pool"], c["pool"])}
    pools = {"k_pool": _f8(s["k_pool"]), "v_pool": _f8(s["v_pool"]), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if c["op"] == "axes":
        return {"q": s["q_out"], **pools}
    return {"kept": s["kept"], "new_lens": s["new_lens"], "new_weights": s["new_weights"], **pools}


# --------------------------------------------------------------------------- work

def work(case):
    c = case
    h, d = c["kv_heads"], c["head_dim"]
    if c["op"] == "evict":
        ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["batch"])
        keep = [min(t, c["budget"]) for t in ctx]
        # every weight once; the kept tokens' codes and scales; codes, scales, index and weight written
        by = 4 * h * sum(ctx) + h * sum(keep) * (2 * (2 * d + 8 / BLOCK) + 8) + 8 * c["batch"]
        return {"bytes": by, "flops": 3 * 2 * d * h * sum(keep)}
    hq = c["q_heads"]
    if c["op"] == "axes":
        n = c["tokens"] - c["pad"] if c["form"] == "slots" else sum(_lens(c)[0])
        pairs = sum(_ints(c["sections"]))
        out = 2 if c.get("pool") == "bf16" else 1
        by = n * (2 * (2 * hq + 2 * h) * d + out * 2 * h * d + 8 * pairs + 8 * len(_ints(c["sections"])))
        if c["form"] == "slots":
            by += 8 * n
        else:
            new, ctx = _lens(c)
            kept = sum((t - m) % BLOCK for m, t in zip(new, ctx))
            pages = sum((t + BLOCK - 1) // BLOCK - (t - m) // BLOCK for m, t in zip(new, ctx))
            by += 2 * h * (kept * d + 4 * pages)
        return {"bytes": by, "flops": n * (6 * pairs * (hq + h) + 2 * h * d)}
    if c["op"] == "shared":
        sizes, prefix, ctx = _shared_lens(c)
        w = c["window"] or max(ctx)
        pairs = sum(min(t, w) for t in ctx)
        at, keys = 0, 0
        for n, p in zip(sizes, prefix):
            mine = ctx[at:at + n]
            keys += max(0, p - max(0, min(mine) - w)) + sum(t - max(p, t - w) for t in mine)
            at += n
        return {"bytes": 2 * h * keys * (d + 4 / BLOCK) + 4 * sum(sizes) * hq * d, "flops": 4 * pairs * hq * d}
    new, ctx = _lens(c)
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, ctx))
    old = sum(t - n for n, t in zip(new, ctx)) if c["decay"] else 0
    return {"bytes": h * sum(ctx) * (d + 4 / BLOCK) + 2 * sum(new) * hq * d + 4 * h * (sum(ctx) + old), "flops": 2 * pairs * hq * d}


# --------------------------------------------------------------------------- 64 bits

def _grid64(x, bits, low, top):
    """x rounded to the nearest value (ties to even) of a float format with `bits` fraction bits, least
    normal exponent `low` and largest value `top`, saturating; float64."""
    e = (torch.frexp(x)[1] - 1).clamp(min=low)
    step = torch.exp2((e - bits).double())
    return (torch.round(x / step) * step).clamp(-top, top)


def _turn64(x, s):
    """Pair by pair: the two elements of pair i turned by the table's entry at its axis's position."""
    r, tab = len(s["pair_axes"]), s["cos_sin"].double()
    y = x.double().clone()
    for i, axis in enumerate(s["pair_axes"]):
        a, b = (i, i + r) if s["case"]["style"] == "half" else (2 * i, 2 * i + 1)
        co, si = tab[s["positions"][axis], i, None], tab[s["positions"][axis], r + i, None]
        y[..., a], y[..., b] = x[..., a] * co - x[..., b] * si, x[..., b] * co + x[..., a] * si
    return y


def _exact_slots(s):
    c = s["case"]
    live = (s["slots"] >= 0).nonzero()[:, 0]
    q = s["q_out"].double()
    q[live] = _turn64(s["q"], s)[live]
    out = {"q": q}
    for name, x in (("k", _turn64(s["k"], s)), ("v", s["v"].double())):
        pool, scale = s[name + "_pool"], s[name + "_scale"]
        flat = (pool if c["pool"] == "bf16" else _f8(pool, c["pool"])).double().transpose(1, 2).flatten(0, 1).clone()
        y = x[live]
        if c["pool"] != "bf16":
            y = y / scale.double()[:, None]
            y = _grid64(y, 3, -6, E4M3_MAX) if c["pool"] == "e4m3" else _grid64(y, 2, -14, E5M2_MAX)
        flat[s["slots"][live]] = y
        out[name + "_pool"] = flat.unflatten(0, (-1, BLOCK)).transpose(1, 2).contiguous()
    return out


def _scale64(most):
    m, e = torch.frexp(most / E4M3_MAX)            # m = 1/2: a power of two itself
    return torch.exp2(torch.where(most > 0, torch.where(m > 0.5, e, e - 1), -126).clamp(min=-126).double())


def _exact_append(s):
    new, ctx = _lens(s["case"])
    out = {"q": _turn64(s["q"], s)}
    at = [sum(new[:i]) for i in range(len(new))]
    for name, x in (("k", _turn64(s["k"], s)), ("v", s["v"].double())):
        pool, scale = _f8(s[name + "_pool"]).double(), s[name + "_scale"].double()
        for n, t, a, row in zip(new, ctx, at, s["table"].tolist()):
            # the sequence's touched pages as [pages][heads][16][D]: kept tokens first, then the new ones
            p0, p1 = (t - n) // BLOCK, (t + BLOCK - 1) // BLOCK
            ids = torch.tensor(row[p0:p1], device="cuda")
            kept = (t - n) % BLOCK
            y = torch.zeros(((p1 - p0) * BLOCK,) + x.shape[1:], dtype=torch.float64, device="cuda")
            y[kept:kept + n] = x[a:a + n]
            y = y.unflatten(0, (-1, BLOCK)).transpose(1, 2)
            sc = _scale64(y.abs().amax((2, 3)))
            if kept:
                sc[0] = torch.maximum(sc[0], scale[ids[0]])
                y[0, :, :kept] = pool[ids[0], :, :kept] * scale[ids[0]][:, None, None]
            y = _grid64(y / sc[:, :, None, None], 3, -6, E4M3_MAX)
            end = kept + n - (p1 - p0 - 1) * BLOCK
            y[-1, :, end:] = pool[ids[-1], :, end:]
            pool[ids], scale[ids] = y, sc
        out[name + "_pool"], out[name + "_scale"] = pool, scale
    return out


def _keys64(s, name, row, t, g):
    ids = torch.tensor(row[:(t + BLOCK - 1) // BLOCK], device="cuda")
    return (_f8(s[name + "_pool"])[ids, g].double() * s[name + "_scale"][ids, g].double()[:, None, None]).flatten(0, 1)[:t]


def _exact_shared(s):
    """Every sequence by itself over its own table's keys."""
    c = s["case"]
    hq, h, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (t, row) in enumerate(zip(s["lens"], s["table"].tolist())):
        for g in range(h if t else 0):
            lo = max(0, t - c["window"]) if c["window"] else 0
            k, v = _keys64(s, "k", row, t, g)[lo:], _keys64(s, "v", row, t, g)[lo:]
            heads = slice(g * (hq // h), (g + 1) * (hq // h))
            out[b, heads] = torch.softmax(s["q"][b, heads].double() @ k.T / d ** 0.5, 1) @ v
    return out


def _exact_weights(s):
    c = s["case"]
    hq, h, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    out, a = s["weights"].double(), 0
    for b, (n, t, row) in enumerate(zip(_lens(c)[0], s["lens"], s["table"].tolist())):
        pos = torch.arange(t - n, t, device="cuda")[:, None]
        hidden = torch.arange(t, device="cuda") > pos
        for g in range(h):
            k = _keys64(s, "k", row, t, g)
            w = torch.zeros(t, dtype=torch.float64, device="cuda")
            for i in range(g * (hq // h), (g + 1) * (hq // h)):
                w += torch.softmax((s["q"][a:a + n, i].double() @ k.T / d ** 0.5).masked_fill(hidden, -math.inf), 1).sum(0)
            w[:t - n] += c["decay"] * out[b, g, :t - n]
            out[b, g, :t] = w
        a += n
    return out


def _exact_evict(s):
    c = s["case"]
    kept, lens = s["kept"].double() * 0 - 1, s["new_lens"].double()
    moved = s["new_weights"].double()
    pools = {name: (_f8(s[name + "_pool"]).double(), s[name + "_scale"].double()) for name in ("k", "v")}
    out = {name: (p.clone(), sc.clone()) for name, (p, sc) in pools.items()}
    for b, t in enumerate(s["lens"]):
        n = min(t, c["budget"])
        lens[b] = n
        src, dst = s["table"][b].long(), s["new_table"][b].long()
        for g in range(c["kv_heads"]):
            w = s["weights"][b, g, :t].double()
            sure = torch.zeros(t, dtype=torch.bool, device="cuda")
            sure[:c["sink"]] = True
            sure[max(0, t - c["recent"]):] = True
            # a token stays if fewer than n come before it: those that always stay, more weight, or the same and a lower index
            place = torch.empty(t, dtype=torch.int64, device="cuda")
            by = torch.argsort(torch.where(sure, -math.inf, -w), stable=True)
            place[by] = torch.arange(t, device="cuda")
            ids = (place < n).nonzero()[:, 0]
            kept[b, g, :n] = ids.double()
            moved[b, g, :n] = w[ids]
            to = dst[torch.arange(n, device="cuda") // BLOCK]
            for name, (pool, scale) in pools.items():
                x = pool[src[ids // BLOCK], g, ids % BLOCK] * scale[src[ids // BLOCK], g][:, None]
                new = out[name]
                most = torch.zeros(new[1].shape[0], dtype=torch.float64, device="cuda").index_reduce_(0, to, x.abs().amax(1), "amax")
                blocks = torch.unique(to)
                new[1][blocks, g] = _scale64(most[blocks])
                new[0][to, g, torch.arange(n, device="cuda") % BLOCK] = _grid64(x / new[1][to, g][:, None], 3, -6, E4M3_MAX)
    return {"kept": None, "new_lens": None, "new_weights": moved, "k_pool": out["k"][0], "v_pool": out["v"][0],
            "k_scale": out["k"][1], "v_scale": out["v"][1]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "axes":
        return _exact_slots(s) if case["form"] == "slots" else _exact_append(s)
    return {"shared": _exact_shared, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)
