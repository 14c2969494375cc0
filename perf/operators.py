"""Cases and plain forms of the rotary cache writes and of the block-scaled FP8 cache.

Four operators of a serving step's attention:

  rope    ``kv_rope_cache``: the rotary position embedding of the new tokens' queries and
          keys, and the write of K and V into a paged pool with per-tensor or per-head
          scales (e4m3, e5m2) or a bf16 pool, by slot.
  append  ``kv_block_cache``: the same into a block-scaled e4m3 pool, whose every block of
          16 tokens has a power-of-two scale per KV head for K and one for V, chosen from
          the block's own tokens; tokens already in a block that continues are brought to
          its new scale.
  decode  ``fp8_block_decode_attn``: one query per sequence over a block-scaled pool.
  prefill ``fp8_block_prefill_attn``: chunks of queries, causal (with or without a sliding
          window) or not, over a block-scaled pool.

``run`` computes a case's operator either in its plain form (elementary torch operations,
float32) or, with ``own`` true, through the library's binding.
"""
import math

import torch

own = False

BLOCK = 16                 # tokens of a pool block
E4M3_MAX, E5M2_MAX = 448.0, 57344.0
MAX_POSITIONS = 131072     # rows of the rotary table
WORKSPACE = 32 << 20       # bytes of decode workspace a program keeps


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # ---- rope
        # one decode step of a Llama-3.1-8B-shaped layer, 8 sequences: latency
        dict(name="rope step", op="rope", tokens=8, pad=0, q_heads=32, kv_heads=8, head_dim=128, rot_dim=128,
             style="half", pool="e4m3"),
        # a ragged mixed batch, padded at its end, of a layer kept in bf16 by the skip-layer
        # mask (gpt-oss-20b-shaped heads)
        dict(name="rope mixed batch bf16", op="rope", tokens=4133, pad=27, q_heads=64, kv_heads=8, head_dim=64,
             rot_dim=64, style="half", pool="bf16"),
        # filling the cache with long prompts (131,072 tokens in the largest workload; half here)
        dict(name="rope fill", op="rope", tokens=65536, pad=0, q_heads=32, kv_heads=8, head_dim=128, rot_dim=128,
             style="half", pool="e4m3"),
        # ---- append
        # one decode step, 8 sequences of 16k to 24k tokens: latency, blocks that continue
        dict(name="append step", op="append", batch=8, new_lo=1, new_hi=1, ctx_lo=16384, ctx_hi=24576, q_heads=32,
             kv_heads=8, head_dim=128, rot_dim=128, style="half"),
        # chunks of odd lengths that begin and end inside blocks, partial rotation in pairs
        dict(name="append odd chunks", op="append", batch=5, new_lo=1, new_hi=1501, ctx_lo=1600, ctx_hi=9001,
             q_heads=8, kv_heads=2, head_dim=256, rot_dim=64, style="pairs"),
        # filling the cache with four long prompts
        dict(name="append fill", op="append", batch=4, new_lo=16384, new_hi=16384, ctx_lo=16384, ctx_hi=16384,
             q_heads=32, kv_heads=8, head_dim=128, rot_dim=128, style="half"),
        # ---- decode
        # a single sequence of 4,096 tokens: latency
        dict(name="decode 4k", op="decode", batch=1, ctx_lo=4096, ctx_hi=4096, q_heads=32, kv_heads=8, head_dim=128,
             window=0),
        # the Llama-3.1-8B-shaped decode under load, one layer
        dict(name="decode 8 x 16k-24k", op="decode", batch=8, ctx_lo=16384, ctx_hi=24576, q_heads=32, kv_heads=8,
             head_dim=128, window=0),
        # the gpt-oss-20b-shaped decode, a full-attention layer
        dict(name="decode d64 8 x 8k-32k", op="decode", batch=8, ctx_lo=8192, ctx_hi=32768, q_heads=64, kv_heads=8,
             head_dim=64, window=0),
        # ---- prefill
        # a few drafted tokens of three sequences verified at once: latency, ragged
        dict(name="prefill drafts", op="prefill", batch=3, new_lo=3, new_hi=9, ctx_lo=611, ctx_hi=2050, q_heads=32,
             kv_heads=8, head_dim=128, window=0, causal=True),
        # a chunk of a long prompt
        dict(name="prefill chunk", op="prefill", batch=1, new_lo=2048, new_hi=2048, ctx_lo=32768, ctx_hi=32768,
             q_heads=32, kv_heads=8, head_dim=128, window=0, causal=True),
        # whole prompts at head_dim 256
        dict(name="prefill prompts d256", op="prefill", batch=4, new_lo=8192, new_hi=8192, ctx_lo=8192, ctx_hi=8192,
             q_heads=8, kv_heads=1, head_dim=256, window=0, causal=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("rope", "append", "decode", "prefill"))
    head_dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 4, 8, 16) if head_dim <= 128 else (1, 2, 4, 8))
    if group * kv_heads > 64:
        kv_heads = 64 // group
    heads = dict(q_heads=group * kv_heads, kv_heads=kv_heads, head_dim=head_dim)
    rot = dict(rot_dim=rng.choice([r for r in (32, 64, 96, 128, 256) if r <= head_dim]),
               style=rng.choice(("half", "pairs")))
    row = (group + 2) * kv_heads * head_dim                      # elements of a token
    if op == "rope":
        tokens = _log(rng, 1, min(65536, 65536 * 6144 // row))
        return dict(op=op, tokens=tokens, pad=rng.choice((0, 0, tokens // 7)), pool=rng.choice(("e4m3", "bf16", "e5m2")),
                    **heads, **rot)
    if op == "append":
        batch = _log(rng, 1, 32)
        new_hi = _log(rng, 1, min(16384, 65536 * 6144 // row // batch))
        before = _log(rng, 1, 16384) - 1
        return dict(op=op, batch=batch, new_lo=rng.choice((1, (new_hi + 1) // 2, new_hi)), new_hi=new_hi,
                    ctx_lo=new_hi + before // 2, ctx_hi=new_hi + before, **heads, **rot)
    if op == "decode":
        batch = _log(rng, 1, 32)
        ctx_hi = _log(rng, 1, min(131072, (400 << 20) // (2 * batch * kv_heads * head_dim)))
        return dict(op=op, batch=batch, ctx_lo=rng.choice((0, ctx_hi // 3, ctx_hi)), ctx_hi=ctx_hi,
                    window=rng.choice((0, 0, _log(rng, 1, 4096))), **heads)
    while True:
        batch = _log(rng, 1, 6)
        new_hi = _log(rng, 1, 8192)
        ctx_hi = new_hi + _log(rng, 1, 32768) - 1
        if batch * heads["q_heads"] * new_hi * ctx_hi <= 1 << 30:
            break
    causal = rng.random() < 0.8
    return dict(op=op, batch=batch, new_lo=rng.choice((1, (new_hi + 1) // 2, new_hi)), new_hi=new_hi,
                ctx_lo=(new_hi + ctx_hi) // 2, ctx_hi=ctx_hi, causal=causal,
                window=rng.choice((0, _log(rng, 1, 4096))) if causal else 0, **heads)


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], the last of them hi, in an order without a pattern."""
    return [lo + int((hi - lo) * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(n - 1)] + [hi]


def _lens(c):
    """(new tokens, context lengths with the new tokens) of an append or prefill case's sequences."""
    return _spread(c["new_lo"], c["new_hi"], c["batch"]), _spread(c["ctx_lo"], c["ctx_hi"], c["batch"])


# --------------------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _codes(g, shape):
    """Bytes left in a pool by earlier use: any e4m3 code."""
    return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)


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


def _int(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


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


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    hq, h, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    if c["op"] == "rope":
        n = c["tokens"]
        s["q"], s["k"], s["v"] = _fused(g, n, c)
        s["positions"] = torch.randint(0, MAX_POSITIONS, (n,), generator=g, device="cuda")
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
        s["q_out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
        s["cos_sin"] = _table(c["rot_dim"])
        return s
    if c["op"] == "append":
        new, s["lens"] = _lens(c)
        s["q"], s["k"], s["v"] = _fused(g, sum(new), c)
        s["cos_sin"] = _table(c["rot_dim"])
        s["q_out"] = torch.zeros(sum(new), hq, d, dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "decode":
        new, s["lens"] = None, _spread(c["ctx_lo"], c["ctx_hi"], c["batch"])
        s["q"] = _randn(g, c["batch"], hq, d).to(torch.bfloat16)
        s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")
    else:
        new, s["lens"] = _lens(c)
        s["q"] = _randn(g, sum(new), hq, d).to(torch.bfloat16)
    s["table"], nb = _pages(g, s["lens"])
    s["ctx"] = _int(s["lens"])
    if new is not None:
        s["cu"], s["max_new"] = _int([sum(new[:i]) for i in range(len(new) + 1)]), max(new)
    s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _block_pool(g, nb, c)
    if c["op"] != "append":
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


def _rope_plain(s):
    c = s["case"]
    cs = s["cos_sin"][s["positions"]]
    keep = s["slots"] >= 0
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


def _places(s):
    """Position of each new token and the pool block and slot that hold it."""
    n = s["k"].shape[0] if "k" in s else s["q"].shape[0]
    at = torch.arange(n, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], at, right=True) - 1
    pos = (s["ctx"][seq] - s["cu"][seq + 1] + at).long()
    return pos, s["table"][seq, pos // BLOCK].long(), pos % BLOCK


def _append_plain(s):
    c = s["case"]
    pos, block, off = _places(s)
    cs = s["cos_sin"][pos]
    s["q_out"].copy_(_rotate(s["q"].float(), cs, c["style"]))
    for x, pool, scale in ((_rotate(s["k"].float(), cs, c["style"]), s["k_pool"], s["k_scale"]),
                           (s["v"].float(), s["v_pool"], s["v_scale"])):
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


def _gathered(s, pool, scale, dtype):
    """[batch][KV head][key][head_dim] values of the sequences' blocks, zero behind each sequence."""
    tab = s["table"].clamp(min=0).long()
    x = _f8(pool[tab]).to(dtype) * scale[tab].to(dtype)[..., None, None]     # [B][pages][H][16][D]
    x = x.transpose(1, 2).flatten(2, 3)
    live = torch.arange(x.shape[2], device="cuda") < s["ctx"][:, None]
    return x.masked_fill_(~live[:, None, :, None], 0)


def _attend(q, k, v, seen, d):
    """q [B][H][rows][D], k / v [B][H][keys][D], seen [B][1][rows][keys]; a row that sees nothing gives 0."""
    p = (q @ k.mT).mul_(1 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    return (p @ v) / p.sum(-1, keepdim=True).clamp_(min=1e-30)


def _decode_plain(s, dtype):
    c = s["case"]
    b, hq, d = s["q"].shape
    h = c["kv_heads"]
    k, v = _gathered(s, s["k_pool"], s["k_scale"], dtype), _gathered(s, s["v_pool"], s["v_scale"], dtype)
    key, t = torch.arange(k.shape[2], device="cuda"), s["ctx"][:, None]
    seen = (key < t) & (key >= (t - c["window"] if c["window"] else 0))
    return _attend(s["q"].to(dtype).view(b, h, hq // h, d), k, v, seen[:, None, None], d).view(b, hq, d)


def _prefill_plain(s, dtype):
    c = s["case"]
    n, hq, d = s["q"].shape
    h, b, m = c["kv_heads"], c["batch"], s["max_new"]
    k, v = _gathered(s, s["k_pool"], s["k_scale"], dtype), _gathered(s, s["v_pool"], s["v_scale"], dtype)
    # the ragged queries padded to the longest chunk
    row = s["cu"][:-1, None] + torch.arange(m, device="cuda")
    real = row < s["cu"][1:, None]
    q = s["q"].to(dtype)[row.clamp(max=n - 1).long()]                        # [B][m][Hq][D]
    q = q.view(b, m, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, hq // h * m, d)
    pos = (s["ctx"][:, None] - s["cu"][1:, None] + row)[:, :, None]          # [B][m][1]
    key, t = torch.arange(k.shape[2], device="cuda"), s["ctx"][:, None, None]
    seen = key < t
    if c["causal"]:
        seen = seen & (key <= pos)
        if c["window"]:
            seen = seen & (key > pos - c["window"])
    seen = seen.expand(b, m, -1)[:, None, None].expand(b, 1, hq // h, m, -1).flatten(2, 3)
    o = _attend(q, k, v, seen, d)
    return o.view(b, h, hq // h, m, d).permute(0, 3, 1, 2, 4).reshape(b, m, hq, d)[real]


# --------------------------------------------------------------------------- a pass

def _run_own(s):
    import fp8_kv_cache_quant_gb300 as f
    c = s["case"]
    if c["op"] == "rope":
        rope = f.Rope(s["cos_sin"], interleaved=c["style"] == "pairs")
        skip = [1] if c["pool"] == "bf16" else None
        cache = f.LayerCache(s["k_pool"], s["v_pool"], f.KV_E5M2 if c["pool"] == "e5m2" else f.KV_E4M3)
        f.kv_rope_cache(s["q"], s["k"], s["v"], s["positions"], s["slots"], rope, cache, s["k_scale"], s["v_scale"],
                        gran=f.SCALE_PER_HEAD, skip_layer_mask=skip, q_out=s["q_out"])
        return s["q_out"]
    cache = f.BlockCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
    if c["op"] == "append":
        rope = f.Rope(s["cos_sin"], interleaved=c["style"] == "pairs")
        f.kv_block_cache(s["k"], s["v"], s["cu"], s["max_new"], cache, s["table"], s["ctx"], rope=rope, q=s["q"],
                         q_out=s["q_out"])
        return s["q_out"]
    if c["op"] == "decode":
        return f.fp8_block_decode_attn(s["q"], cache, s["table"], s["ctx"], window=c["window"],
                                       workspace=s["workspace"])
    return f.fp8_block_prefill_attn(s["q"], s["cu"], s["max_new"], cache, s["table"], s["ctx"], causal=c["causal"],
                                    window=c["window"])


def run(state):
    s, c = state, state["case"]
    if own:
        out = _run_own(s)
    elif c["op"] == "rope":
        _rope_plain(s)
        out = s["q_out"]
    elif c["op"] == "append":
        _append_plain(s)
        out = s["q_out"]
    elif c["op"] == "decode":
        out = _decode_plain(s, torch.float32).to(torch.bfloat16)
    else:
        out = _prefill_plain(s, torch.float32).to(torch.bfloat16)
    if c["op"] in ("decode", "prefill"):
        return out
    if c["op"] == "rope":
        pools = (s["k_pool"], s["v_pool"]) if c["pool"] == "bf16" else (_f8(s["k_pool"], c["pool"]), _f8(s["v_pool"], c["pool"]))
        return {"q": out, "k_pool": pools[0], "v_pool": pools[1]}
    return {"q": out, "k_pool": _f8(s["k_pool"]), "v_pool": _f8(s["v_pool"]), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


# --------------------------------------------------------------------------- work

def _pairs(c):
    """Visible (query, key) pairs of one query head, and the keys some query sees."""
    new, ctx = _lens(c)
    pairs = keys = 0
    for n, t in zip(new, ctx):
        if not c["causal"]:
            pairs, keys = pairs + n * t, keys + t
            continue
        w = c["window"] or t
        full = min(n, max(0, t - w + 1))             # rows that see a whole window: positions >= w - 1
        part = n - full
        first = t - n + 1                            # keys the first row sees, if no window cuts them
        pairs += full * w + part * (2 * first + part - 1) // 2
        keys += min(t, n + w - 1)
    return pairs, keys


def work(case):
    c = case
    hq, h, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    if c["op"] in ("rope", "append"):
        n = c["tokens"] - c["pad"] if c["op"] == "rope" else sum(_lens(c)[0])
        out = 2 if c.get("pool") == "bf16" else 1
        by = n * (2 * (2 * hq + 2 * h) * d + out * 2 * h * d + 4 * min(c["rot_dim"], d))
        if c["op"] == "rope":
            by += 16 * n
        else:
            new, ctx = _lens(c)
            kept = sum((t - m) % BLOCK for m, t in zip(new, ctx))
            pages = sum((t + BLOCK - 1) // BLOCK - (t - m) // BLOCK for m, t in zip(new, ctx))
            by += 2 * h * (kept * d + 4 * pages)
        return {"bytes": by, "flops": n * (3 * c["rot_dim"] * (hq + h) + 2 * h * d)}
    if c["op"] == "decode":
        ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["batch"])
        keys = sum(min(t, c["window"] or t) for t in ctx)
        rows, pairs = c["batch"], keys
    else:
        pairs, keys = _pairs(c)
        rows = sum(_lens(c)[0])
    return {"bytes": 2 * h * keys * (d + 4 / BLOCK) + 4 * rows * hq * d, "flops": 4 * pairs * hq * d}


# --------------------------------------------------------------------------- 64 bits

def _grid64(x, bits, low, top):
    """x rounded to the nearest value (ties to even) of a float format with `bits` fraction bits, least
    normal exponent `low` and largest value `top`, saturating; float64."""
    e = (torch.frexp(x)[1] - 1).clamp(min=low)
    step = torch.exp2((e - bits).double())
    return (torch.round(x / step) * step).clamp(-top, top)


def _turn64(x, positions, case):
    """The rotation by angles evaluated in float64 from the table's own float32 entries."""
    r = case["rot_dim"]
    x = x.double()
    y = x.clone()
    half = r // 2
    i = torch.arange(half, device="cuda")
    a, b = (i, i + half) if case["style"] == "half" else (2 * i, 2 * i + 1)
    co, si = positions[:, None, :half].double(), positions[:, None, half:].double()
    y[..., a] = x[..., a] * co - x[..., b] * si
    y[..., b] = x[..., b] * co + x[..., a] * si
    return y


def _exact_rope(s):
    c = s["case"]
    rows = s["cos_sin"][s["positions"]]
    live = (s["slots"] >= 0).nonzero()[:, 0]
    q = s["q_out"].double()
    q[live] = _turn64(s["q"], rows, c)[live]
    pools = []
    for x, pool, scale in ((_turn64(s["k"], rows, c), s["k_pool"], s["k_scale"]), (s["v"].double(), s["v_pool"], s["v_scale"])):
        flat = (pool if c["pool"] == "bf16" else _f8(pool, c["pool"])).double().transpose(1, 2).flatten(0, 1).clone()
        y = x[live]
        if c["pool"] != "bf16":
            y = y / scale.double()[:, None]
            y = _grid64(y, 3, -6, E4M3_MAX) if c["pool"] == "e4m3" else _grid64(y, 2, -14, E5M2_MAX)
        flat[s["slots"][live]] = y
        pools.append(flat.unflatten(0, (-1, BLOCK)).transpose(1, 2).contiguous())
    return {"q": q, "k_pool": pools[0], "v_pool": pools[1]}


def _exact_append(s):
    c = s["case"]
    new, ctx = _lens(c)
    pos = torch.cat([torch.arange(t - n, t) for n, t in zip(new, ctx)]).cuda()
    rows = s["cos_sin"][pos]
    out = {"q": _turn64(s["q"], rows, c)}
    at = [sum(new[:i]) for i in range(len(new))]
    for name, x in (("k", _turn64(s["k"], rows, c)), ("v", s["v"].double())):
        pool, scale = _f8(s[name + "_pool"]).double(), s[name + "_scale"].double()
        for n, t, a, row in zip(new, ctx, at, s["table"].tolist()):
            # the sequence's touched pages as [pages][heads][16][D]: kept tokens first, then the new ones
            p0, p1 = (t - n) // BLOCK, (t + BLOCK - 1) // BLOCK
            ids = torch.tensor(row[p0:p1], device="cuda")
            kept = (t - n) % BLOCK
            y = torch.zeros(((p1 - p0) * BLOCK,) + x.shape[1:], dtype=torch.float64, device="cuda")
            y[kept:kept + n] = x[a:a + n]
            y = y.unflatten(0, (-1, BLOCK)).transpose(1, 2)
            most = y.abs().amax((2, 3))
            sc = torch.exp2(torch.ceil(torch.log2(most / E4M3_MAX)).clamp(min=-126))
            if kept:
                sc[0] = torch.maximum(sc[0], scale[ids[0]])
                y[0, :, :kept] = pool[ids[0], :, :kept] * scale[ids[0]][:, None, None]
            y = _grid64(y / sc[:, :, None, None], 3, -6, E4M3_MAX)
            end = kept + n - (p1 - p0 - 1) * BLOCK
            y[-1, :, end:] = pool[ids[-1], :, end:]
            pool[ids], scale[ids] = y, sc
        out[name + "_pool"], out[name + "_scale"] = pool, scale
    return out


def _exact_attend(s, c):
    """Sequence by sequence and head by head, in float64."""
    hq, h, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    new = [1] * c["batch"] if c["op"] == "decode" else _lens(c)[0]
    out, a = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for n, t, row in zip(new, s["lens"], s["table"].tolist()):
        if t:
            ids = torch.tensor(row[:(t + BLOCK - 1) // BLOCK], device="cuda")
            pos = torch.arange(t - n, t, device="cuda")[:, None]
            key = torch.arange(t, device="cuda")
            hidden = key > pos if c["op"] == "decode" or c["causal"] else torch.zeros(n, t, dtype=torch.bool, device="cuda")
            if c["window"]:
                hidden = hidden | (key <= pos - c["window"])
            for g in range(h):
                k = (_f8(s["k_pool"])[ids, g].double() * s["k_scale"][ids, g].double()[:, None, None]).flatten(0, 1)[:t]
                v = (_f8(s["v_pool"])[ids, g].double() * s["v_scale"][ids, g].double()[:, None, None]).flatten(0, 1)[:t]
                for i in range(g * (hq // h), (g + 1) * (hq // h)):
                    w = s["q"][a:a + n, i].double() @ k.T / d ** 0.5
                    out[a:a + n, i] = torch.softmax(w.masked_fill(hidden, -math.inf), 1) @ v
        a += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_attend(s, case)
