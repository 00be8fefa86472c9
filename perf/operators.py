"""Measured cases of the packed attention and the 8-bit cache operators.

kinds: "forward" (packed attention), "train" (packed attention with its gradients), "decode"
(attention over the 8-bit cache), "append" (writing new tokens into it), "extend" (block tables and
slot maps for a step).  A case names sizes only; the lengths of its sequences follow from
(batch, lo, hi, lengths_seed)."""
import math
import random

import torch

own = False


def _lengths(batch, lo, hi, seed):
    """`batch` lengths in [lo, hi], spread over their logarithm; the first is hi, so the range is used."""
    r = random.Random(seed)
    some = [min(hi, max(lo, int(round(math.exp(r.uniform(math.log(lo), math.log(hi + 0.5))))))) for _ in range(batch - 1)]
    return [hi] + some


def _case_lengths(c):
    """(query lengths, key lengths) of a case's sequences."""
    keys = _lengths(c["batch"], c["lo"], c["hi"], c["lengths_seed"])
    if c["kind"] == "decode":
        qs = _lengths(c["batch"], 1, c["q_hi"], c["lengths_seed"] + 1)
        return [min(a, b) for a, b in zip(qs, keys)], keys
    if c["kind"] in ("forward", "train") and c["q_hi"]:
        return _lengths(c["batch"], c["q_lo"], c["q_hi"], c["lengths_seed"] + 1), keys
    return keys, keys


def listed():
    packed = dict(q_lo=0, q_hi=0, causal=True, head_dim=128, heads=24, kv_heads=8)
    cache = dict(block_tokens=64, heads=24, kv_heads=8, head_dim=128)
    return [
        # a batch of short prompts through a text model: latency counts
        dict(packed, name="forward_short", kind="forward", batch=16, lo=1, hi=77, lengths_seed=1),
        # one long document, prefilled whole
        dict(packed, name="forward_long", kind="forward", batch=1, lo=16384, hi=16384, lengths_seed=2),
        # video tokens of two 18x24x24 latents attend to their text keys: not causal, every head its own keys
        dict(packed, name="forward_text_keys", kind="forward", batch=2, lo=77, hi=226, q_lo=10368, q_hi=10368,
             causal=False, kv_heads=24, lengths_seed=3),
        # a training step's packed row of odd lengths, head size 64, eight query heads to a key head
        dict(packed, name="train_ragged", kind="train", batch=6, lo=301, hi=2047, heads=16, kv_heads=2, head_dim=64,
             lengths_seed=4),
        # a training step on one long sequence
        dict(packed, name="train_long", kind="train", batch=1, lo=8192, hi=8192, lengths_seed=5),
        # one user, one token
        dict(cache, name="decode_one", kind="decode", batch=1, lo=1000, hi=1000, q_hi=1, lengths_seed=6),
        # a serving batch of ragged lengths
        dict(cache, name="decode_batch", kind="decode", batch=64, lo=501, hi=8000, q_hi=1, lengths_seed=7),
        # a few drafted tokens for each request, small blocks, long caches
        dict(cache, name="decode_drafts", kind="decode", batch=7, lo=3001, hi=30011, q_hi=6, block_tokens=16, heads=16,
             kv_heads=2, head_dim=64, lengths_seed=8),
        # the tokens of one serving step
        dict(cache, name="append_step", kind="append", batch=64, lo=501, hi=8000, new_lo=1, new_hi=1, lengths_seed=9),
        # prompts entering the cache
        dict(cache, name="append_prompts", kind="append", batch=6, lo=1, hi=97, new_lo=513, new_hi=8000, lengths_seed=10),
        # tables for one serving step
        dict(name="extend_step", kind="extend", batch=64, lo=501, hi=8000, new_lo=1, new_hi=1, block_tokens=64, ended=3,
             lengths_seed=11),
        # tables for a large step with prompts in it
        dict(name="extend_prompts", kind="extend", batch=500, lo=1, hi=4000, new_lo=1, new_hi=2000, block_tokens=16,
             ended=37, lengths_seed=12),
    ]


def _between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["forward", "forward", "train", "train", "decode", "decode", "append", "extend"])
    c = dict(kind=kind, lengths_seed=rng.randrange(1 << 30))
    heads, kv = rng.choice([(24, 8), (24, 24), (24, 4), (16, 2), (8, 1), (12, 12), (2, 2), (10, 2)])
    d = rng.choice([64, 128, 128])
    if kind in ("forward", "train"):
        hi = _between(rng, 24, 8192)
        batch = max(1, min(_between(rng, 1, 24), int(3.2e9 / (24.0 * hi * hi)) or 1, 16384 // hi))
        cross = kind == "forward" and rng.random() < 0.35
        if cross:  # queries of other lengths than the keys
            q_hi = _between(rng, 24, 4096)
            c.update(q_lo=max(1, q_hi // _between(rng, 1, 9)), q_hi=q_hi, causal=rng.random() < 0.4)
            batch = max(1, min(batch, 16384 // q_hi))
        else:
            c.update(q_lo=0, q_hi=0, causal=rng.random() < 0.85)
        c.update(batch=batch, hi=hi, lo=max(1, hi // _between(rng, 1, 30)), heads=heads, kv_heads=kv, head_dim=d)
    else:
        bt = rng.choice([16, 32, 64, 128])
        hi = _between(rng, 20, 30000)
        batch = max(1, min(_between(rng, 1, 96), 200000 // hi))
        c.update(batch=batch, hi=hi, lo=max(1, hi // _between(rng, 1, 30)), block_tokens=bt)
        if kind != "extend":
            c.update(heads=heads, kv_heads=min(kv, 8) if heads % min(kv, 8) == 0 else 1, head_dim=d)
        if kind == "decode":
            c.update(q_hi=rng.choice([1, 1, 1, 2, 3, 5, 8]))
        else:
            new_hi = rng.choice([1, _between(rng, 1, 4000)])
            c.update(new_lo=max(1, new_hi // _between(rng, 1, 20)), new_hi=new_hi)
            c["batch"] = max(1, min(batch, 24000 // new_hi))
        if kind == "extend":
            c.update(batch=_between(rng, 1, 500), hi=min(hi, 4000), ended=0)
            c["lo"] = min(c["lo"], c["hi"])
            c["new_hi"] = min(c["new_hi"], 2000)
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
            c["ended"] = rng.randrange(0, max(1, c["batch"] // 4))
    return c


def _cu(lengths, device):
    total, out = 0, [0]
    for n in lengths:
        total += n
        out.append(total)
    return torch.tensor(out, dtype=torch.int32, device=device)


def _pow2_scale(amax):
    """The smallest power of two 2^e, -60 <= e <= 120, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax / 448.0)  # amax / 448 = m * 2^e, 0.5 <= m < 1
    e = torch.where(m > 0.5, e, e - 1)
    e = torch.where(amax > 0, e, torch.full_like(e, -60)).clamp(-60, 120)
    return torch.ldexp(torch.ones_like(amax), e)


def _pages(lengths, block_tokens, spare, g, device):
    """Block tables over a shuffled pool with `spare` free blocks: (tables, free stack, free count, pool size)."""
    held = [-(-n // block_tokens) for n in lengths]
    pool = sum(held) + spare
    width = max(held) + -(-spare // max(1, len(lengths))) + 1
    order = torch.randperm(pool, generator=g, device=device).to(torch.int32)
    tables = torch.full((len(lengths), width), -1, dtype=torch.int32, device=device)
    at = 0
    for b, n in enumerate(held):
        tables[b, :n] = order[at:at + n]
        at += n
    free = torch.full((pool,), -1, dtype=torch.int32, device=device)
    free[:spare] = order[at:]
    return tables, free, spare, pool


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case)
    if c["kind"] in ("forward", "train"):
        nq, nk = _case_lengths(c)
        H, K, d = c["heads"], c["kv_heads"], c["head_dim"]
        s.update(cu_q=_cu(nq, dev), cu_k=_cu(nk, dev), max_q=max(nq), max_k=max(nk), scale=1.0 / math.sqrt(d))
        if c["q_hi"]:
            s["q"] = randn(sum(nq), H, d).bfloat16()
            kv = randn(sum(nk), 2 * K, d).bfloat16()
            s["k"], s["v"] = kv[:, :K], kv[:, K:]
        else:  # one projection gives q, k and v side by side
            qkv = randn(sum(nq), H + 2 * K, d).bfloat16()
            s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        if c["kind"] == "train":
            s["dout"] = randn(sum(nq), H, d).bfloat16()
        return s
    bt = c["block_tokens"]
    nk = _lengths(c["batch"], c["lo"], c["hi"], c["lengths_seed"])
    s["lengths"] = torch.tensor(nk, dtype=torch.int32, device=dev)
    if c["kind"] == "extend":
        new = _lengths(c["batch"], c["new_lo"], c["new_hi"], c["lengths_seed"] + 1)
        max_slots = sum(new)  # room for every token, whichever requests have ended
        spare = sum(-(-n // bt) + 1 for n in new)
        random.Random(seed).shuffle(new)
        for b in random.Random(seed + 1).sample(range(c["batch"]), c["ended"]):
            new[b] = -1
        tables, free, count, _ = _pages(nk, bt, spare, g, dev)
        held = -(-max(nk) // bt) + -(-c["new_hi"] // bt) + 1
        if tables.shape[1] < held:
            wide = torch.full((len(nk), held), -1, dtype=torch.int32, device=dev)
            wide[:, :tables.shape[1]] = tables
            tables = wide
        s.update(new=torch.tensor(new, dtype=torch.int32, device=dev), tables=tables, free=free,
                 count=torch.tensor([count], dtype=torch.int32, device=dev),
                 max_slots=max_slots)
        return s
    H, K, d = c["heads"], c["kv_heads"], c["head_dim"]
    new = [0] * c["batch"] if c["kind"] == "decode" else _lengths(c["batch"], c["new_lo"], c["new_hi"], c["lengths_seed"] + 1)
    tables, _, _, pool = _pages([a + b for a, b in zip(nk, new)], bt, 3, g, dev)
    for name in ("k", "v"):
        x = randn(pool, K, bt, d)
        x *= torch.exp(0.5 * randn(pool, K, 1, 1)) if name == "v" else 1.0 + (torch.arange(d, device=dev) % 32 == 5) * 3.0
        scale = _pow2_scale(x.abs().amax((2, 3)))
        s[name + "_cache"] = (x / scale[:, :, None, None]).to(torch.float8_e4m3fn)
        s[name + "_scales"] = scale
        del x
    s["tables"] = tables
    if c["kind"] == "decode":
        nq, _ = _case_lengths(c)
        s.update(cu_q=_cu(nq, dev), max_q=max(nq), max_k=max(nk), scale=1.0 / math.sqrt(d))
        s["q"] = randn(sum(nq), H, d).bfloat16()
    else:
        slots = []
        for b, n in enumerate(new):
            pos = torch.arange(nk[b], nk[b] + n, device=dev)
            slots.append(tables[b].long()[pos // bt] * bt + pos % bt)
        s["slots"] = torch.cat(slots)
        kv = randn(sum(new), 2 * K, d).bfloat16()
        s["k"], s["v"] = kv[:, :K], kv[:, K:]
    return s


def work(case):
    c = case
    if c["kind"] == "extend":
        new = _lengths(c["batch"], c["new_lo"], c["new_hi"], c["lengths_seed"] + 1)
        blocks = sum(-(-n // c["block_tokens"]) for n in new)
        return {"bytes": 4.0 * (4 * c["batch"] + 2 * blocks) + 8.0 * sum(new), "flops": 2.0 * sum(new)}
    H, K, d = c["heads"], c["kv_heads"], c["head_dim"]
    if c["kind"] == "append":
        new = sum(_lengths(c["batch"], c["new_lo"], c["new_hi"], c["lengths_seed"] + 1))
        return {"bytes": new * (K * d * 2 * (2.0 + 1.0) + 8.0), "flops": new * K * d * 2 * 2.0}
    nq, nk = _case_lengths(c)
    causal = c["kind"] == "decode" or c["causal"]
    pairs = 0
    for a, b in zip(nq, nk):
        first = b - a  # query i sees first + i + 1 keys
        skip = max(0, -first)
        pairs += (a - skip) * (first + skip + 1 + b) // 2 if causal else a * b
    tq, tk = sum(nq), sum(nk)
    if c["kind"] == "decode":
        held = sum(-(-b // c["block_tokens"]) for b in nk)
        return {"bytes": 2.0 * tk * K * d + 8.0 * held * K + tq * H * (4.0 * d + 4), "flops": 4.0 * d * H * pairs}
    io = 2.0 * d * (2 * tq * H + 2 * tk * K) + 4.0 * tq * H
    if c["kind"] == "forward":
        return {"bytes": io, "flops": 4.0 * d * H * pairs}
    return {"bytes": io + 2.0 * d * (2 * tq * H + 2 * tk * K), "flops": 14.0 * d * H * pairs}


# ---------------------------------------------------------------- plain forms
def _padded(x, cu, length):
    """Packed [T, heads, d] -> fp32 [B, heads, length, d], zeros behind each sequence."""
    at = torch.arange(length, device=x.device)
    valid = at[None, :] < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None].long() + at).clamp(max=x.shape[0] - 1)
    return (x[rows].float() * valid[:, :, None, None]).transpose(1, 2)


def _packed(x, cu, total):
    """[B, heads, length, ...] -> packed [total, heads, ...]."""
    t = torch.arange(total, device=x.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    return x.transpose(1, 2)[b, t - cu.long()[b]]


def _visible(nq, nk, length_q, length_k, causal):
    """[B, length_q, length_k]: does query i of sequence b see key j?"""
    i = torch.arange(length_q, device=nq.device)[None, :, None]
    j = torch.arange(length_k, device=nq.device)[None, None, :]
    seen = (i < nq[:, None, None]) & (j < nk[:, None, None])
    return seen & (j <= nk[:, None, None] - nq[:, None, None] + i) if causal else seen


def _softmax_attention(q, k, v, seen, scale):
    """q [B, H, Lq, d], k and v [B, K, Lk, d], fp32: (probabilities [B, K, G, Lq, Lk], o, lse)."""
    B, H, Lq, d = q.shape
    K, Lk = k.shape[1], k.shape[2]
    s = torch.matmul(q.reshape(B, K, H // K * Lq, d), k.transpose(2, 3)).view(B, K, H // K, Lq, Lk)
    s *= scale
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s -= m
    p = s.exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).view(B, H, Lq)
    p /= torch.where(l > 0, l, torch.ones_like(l))
    o = torch.matmul(p.view(B, K, H // K * Lq, Lk), v).view(B, H, Lq, d)
    return p, o, lse


def _plain_packed(s):
    T = s["q"].shape[0]
    nq, nk = s["cu_q"][1:] - s["cu_q"][:-1], s["cu_k"][1:] - s["cu_k"][:-1]
    q, k, v = (_padded(s[n], s["cu_" + w], s["max_" + w]) for n, w in (("q", "q"), ("k", "k"), ("v", "k")))
    seen = _visible(nq, nk, s["max_q"], s["max_k"], s["causal"])
    p, o, lse = _softmax_attention(q, k, v, seen, s["scale"])
    out = {"o": _packed(o, s["cu_q"], T).bfloat16(), "lse": _packed(lse, s["cu_q"], T).t().contiguous()}
    if s["kind"] == "forward":
        return out
    B, H, Lq, d = q.shape
    K, Lk = k.shape[1], k.shape[2]
    do = _padded(s["dout"], s["cu_q"], s["max_q"])
    rows = do.reshape(B, K, H // K * Lq, d)
    dv = torch.matmul(p.view(B, K, -1, Lk).transpose(2, 3), rows)
    dp = torch.matmul(rows, v.transpose(2, 3)).view(p.shape)
    dp -= (do * o).sum(-1).view(B, K, H // K, Lq, 1)
    ds = dp.mul_(p).mul_(s["scale"]).view(B, K, -1, Lk)
    dq = torch.matmul(ds, k).view(B, H, Lq, d)
    dk = torch.matmul(ds.transpose(2, 3), q.reshape(B, K, H // K * Lq, d))
    Tk = s["k"].shape[0]
    return {"o": out["o"], "dq": _packed(dq, s["cu_q"], T).bfloat16(), "dk": _packed(dk, s["cu_k"], Tk).bfloat16(),
            "dv": _packed(dv, s["cu_k"], Tk).bfloat16()}


def _from_cache(codes, scales, tables, length):
    """[B, K, length, d] fp32: the values of each sequence's first `length` tokens."""
    bt = codes.shape[2]
    page = tables[:, :-(-length // bt)].long().clamp(min=0)
    x = codes.view(torch.uint8)[page].view(torch.float8_e4m3fn).float() * scales[page][..., None, None]
    B, W, K, _, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, K, W * bt, d)[:, :, :length]


def _plain_decode(s):
    nq, nk = s["cu_q"][1:] - s["cu_q"][:-1], s["lengths"]
    k = _from_cache(s["k_cache"], s["k_scales"], s["tables"], s["max_k"])
    v = _from_cache(s["v_cache"], s["v_scales"], s["tables"], s["max_k"])
    seen = _visible(nq, nk, s["max_q"], s["max_k"], True)
    _, o, lse = _softmax_attention(_padded(s["q"], s["cu_q"], s["max_q"]), k, v, seen, s["scale"])
    T = s["q"].shape[0]
    return {"o": _packed(o, s["cu_q"], T).bfloat16(), "lse": _packed(lse, s["cu_q"], T).t().contiguous()}


def _plain_append_one(x, codes, scales, slots):
    """Writes x [T, K, d] at `slots`; a block's scale grows to hold them and its codes follow."""
    P, K, bt, d = codes.shape
    page, at = slots // bt, slots % bt
    x = x.float()
    amax = torch.zeros(P, K, device=x.device)
    amax.scatter_reduce_(0, page[:, None].expand(-1, K), x.abs().amax(2), "amax")
    first = torch.full((P,), bt, dtype=torch.long, device=x.device).scatter_reduce_(0, page, at, "amin")
    touched = first < bt
    fresh = first == 0  # nothing held yet: the old scale does not count
    scale = _pow2_scale(amax)
    scale = torch.where(fresh[:, None], scale, torch.maximum(scale, scales))
    scale = torch.where(touched[:, None], scale, scales)
    raw = codes.view(torch.uint8)
    some = page if len(page) < P else torch.arange(P, device=x.device)  # the blocks whose codes may change, at least
    held = raw[some].view(torch.float8_e4m3fn).float()
    held = (held * (scales[some] / scale[some])[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    raw[some] = torch.where(fresh[some][:, None, None, None], raw[some], held)
    raw[page, :, at] = (x / scale[page][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scales.copy_(scale)


def _plain_append(s):
    for name in ("k", "v"):
        _plain_append_one(s[name], s[name + "_cache"], s[name + "_scales"], s["slots"])
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales")}


def _plain_extend(s):
    bt, length, new, tables, free = s["block_tokens"], s["lengths"].long(), s["new"].long(), s["tables"], s["free"]
    B, W = tables.shape
    count = s["count"].long()
    ended, add = new < 0, new.clamp(min=0)
    held = (length + bt - 1) // bt
    back = torch.where(ended, held, 0)
    need = torch.where(ended, 0, (length + add + bt - 1) // bt - held)
    there = count + back.sum()
    lack = (need.sum() - there).clamp(min=0)
    wide = ((length + add) > W * bt).any()
    short = torch.where(wide, -1, lack)
    fine = short == 0
    j = torch.arange(W, device=tables.device)[None]
    to = count + (back.cumsum(0) - back)[:, None] + j
    pool = torch.cat([free, free.new_zeros(1)])
    pool[torch.where(fine & (j < back[:, None]), to, free.numel())] = tables
    i = j - held[:, None]
    take = (there - 1 - (need.cumsum(0) - need)[:, None] - i).clamp(0, free.numel() - 1)
    tables.copy_(torch.where(fine & (i >= 0) & (i < need[:, None]), pool[take], tables))
    free.copy_(pool[:-1])
    add = torch.where(fine, add, 0)
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)])
    t = torch.arange(s["max_slots"], device=tables.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    pos = length[b] + t - cu[b]
    slots = tables[b, (pos // bt).clamp(max=W - 1)].long() * bt + pos % bt
    return {"tables": tables, "free": free, "slots": torch.where(t < cu[-1], slots, -1), "cu": cu.int(),
            "lengths": torch.where(fine, torch.where(ended, 0, length + add), length).int(),
            "count": torch.where(fine, there - need.sum(), count).int(), "short": short.int().view(1)}


def run(state):
    s = state
    if not own:
        with torch.no_grad():
            return {"forward": _plain_packed, "train": _plain_packed, "decode": _plain_decode, "append": _plain_append,
                    "extend": _plain_extend}[s["kind"]](s)
    import sparse_attention_video_sta_b200 as sta

    if s["kind"] in ("forward", "train"):
        o, lse = sta.sta_packed_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["causal"],
                                          softmax_scale=s["scale"])
        if s["kind"] == "forward":
            return {"o": o, "lse": lse}
        dq, dk, dv = sta.sta_packed_attention_backward(s["q"], s["k"], s["v"], o, lse, s["dout"], s["cu_q"], s["cu_k"],
                                                       causal=s["causal"], softmax_scale=s["scale"])
        return {"o": o, "dq": dq, "dk": dk, "dv": dv}
    if s["kind"] == "decode":
        o, lse = sta.sta_cache_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["tables"],
                                         s["lengths"], cu_q=s["cu_q"], softmax_scale=s["scale"])
        return {"o": o, "lse": lse}
    if s["kind"] == "append":
        sta.sta_cache_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales")}
    r = sta.sta_cache_extend(s["new"], s["lengths"], s["tables"], s["free"], s["count"], s["block_tokens"], s["max_slots"])
    return {"tables": s["tables"], "free": s["free"], "slots": r.slots, "cu": r.cu_new, "lengths": r.lengths,
            "count": r.free_count, "short": r.short}


# ---------------------------------------------------------------- 64 bits
def _exact_row_block(q, k, v, first, scale, do=None):
    """One sequence and key head in 64 bits: q [G, n, d]; query i sees keys up to first + i (all if first is None)."""
    q, k, v = q.double(), k.double(), v.double()
    x = torch.einsum("gnd,md->gnm", q, k) * scale
    if first is not None:
        i, j = torch.arange(q.shape[1], device=q.device), torch.arange(k.shape[0], device=q.device)
        x = torch.where(j[None, :] > i[:, None] + first, float("-inf"), x)
    lse = torch.logsumexp(x, -1)
    x -= torch.where(lse.isinf(), 0.0, lse)[..., None]
    p = x.exp_()
    o = torch.einsum("gnm,md->gnd", p, v)
    if do is None:
        return o, lse
    do = do.double()
    dv = torch.einsum("gnm,gnd->md", p, do)
    t = torch.einsum("gnd,md->gnm", do, v)
    t -= torch.einsum("gnm,gnm->gn", p, t)[..., None]
    t *= p
    return o, lse, scale * torch.einsum("gnm,md->gnd", t, k), scale * torch.einsum("gnm,gnd->md", t, q), dv


def _exact_packed(s, key, value, keys_of):
    """key(b, h), value(b, h): [n, d] of sequence b and key head h."""
    H, d = s["q"].shape[1:]
    G = H // s["kv_heads"]
    cq = s["cu_q"].tolist()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((H, s["q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    train = s["kind"] == "train"
    dq = torch.zeros_like(o)
    dk, dv = (torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") if train else None for _ in range(2))
    for b in range(len(cq) - 1):
        n, rows = cq[b + 1] - cq[b], slice(cq[b], cq[b + 1])
        first = keys_of[b] - n if s["kind"] == "decode" or s["causal"] else None
        for h in range(s["kv_heads"]):
            hs = slice(h * G, (h + 1) * G)
            args = (s["q"][rows, hs].transpose(0, 1), key(b, h), value(b, h), first, s["scale"])
            if train:
                ck = s["cu_k"].tolist()
                r = _exact_row_block(*args, s["dout"][rows, hs].transpose(0, 1))
                dq[rows, hs] = r[2].transpose(0, 1)
                dk[ck[b]:ck[b + 1], h], dv[ck[b]:ck[b + 1], h] = r[3], r[4]
            else:
                r = _exact_row_block(*args)
            o[rows, hs], lse[hs, rows] = r[0].transpose(0, 1), r[1]
    return {"o": o, "dq": dq, "dk": dk, "dv": dv} if train else {"o": o, "lse": lse}


def _exact_code(x):
    """Nearest e4m3 value, ties to even, in 64 bits; |x| <= 448."""
    e = torch.frexp(x)[1].sub(1).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(x), e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("forward", "train"):
        ck = s["cu_k"].tolist()
        return _exact_packed(s, lambda b, h: s["k"][ck[b]:ck[b + 1], h], lambda b, h: s["v"][ck[b]:ck[b + 1], h],
                             [y - x for x, y in zip(ck, ck[1:])])
    bt = case["block_tokens"]
    if case["kind"] == "decode":
        n = s["lengths"].tolist()

        def of(name):
            def get(b, h):
                page = s["tables"][b, :-(-n[b] // bt)].long()
                x = s[name + "_cache"].view(torch.uint8)[page, h].view(torch.float8_e4m3fn).double()
                return (x * s[name + "_scales"].double()[page, h, None, None]).flatten(0, 1)[:n[b]]
            return get
        return _exact_packed(s, of("k"), of("v"), n)
    if case["kind"] == "append":
        out = {}
        slots = s["slots"]
        for name in ("k", "v"):
            codes, scales = s[name + "_cache"].double(), s[name + "_scales"].double()
            x = s[name].double()
            page, start = torch.unique(slots // bt, return_inverse=True)
            top = torch.zeros(len(page), x.shape[1], dtype=torch.float64, device="cuda")
            top.index_reduce_(0, start, x.abs().amax(2), "amax")
            low = torch.full((len(page),), bt, dtype=torch.int64, device="cuda").index_reduce_(0, start, slots % bt, "amin")
            want = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-30) / 448.0)).clamp(-60, 120))
            old = scales[page]
            want = torch.where((low == 0)[:, None], want, torch.maximum(want, old))
            again = _exact_code(codes[page] * (old / want)[:, :, None, None])
            codes[page] = torch.where((low == 0)[:, None, None, None], codes[page], again)
            scales[page] = want
            codes[slots // bt, :, slots % bt] = _exact_code(x / scales[slots // bt][:, :, None])
            out[name + "_cache"], out[name + "_scales"] = codes, scales
        return out
    return None
