"""The 8-bit cache: append (bit for bit), block tables and slots (equal), attention over it (64-bit reference)."""
import math
import random

import pytest
import torch

import prompt_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sta():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    import sparse_attention_video_sta_b200 as s
    return s


def empty_cache(blocks, K, bt, d, fill=0):
    codes = [torch.full((blocks, K, bt, d), fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for _ in range(2)]
    scales = [torch.full((blocks, K), 2.0 ** -60, device="cuda") for _ in range(2)]
    return codes + scales


def values(codes, scales):
    return codes.float().double() * scales.double()[..., None, None]


def tables_for(lengths, bt, blocks, width=None, seed=0):
    held = [-(-n // bt) for n in lengths]
    ids = list(range(blocks))
    random.Random(seed).shuffle(ids)
    t = torch.full((len(lengths), width or max(held + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        t[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    return t.cuda()


def slots_for(table, first, n, bt):
    pos = torch.arange(first, first + n, device="cuda")
    return table.long()[pos // bt] * bt + pos % bt


# ---------------------------------------------------------------- append
def append_reference(x, slots, codes, scales, bt):
    """What append leaves: lists of 64-bit values and scales, token by token of each block's run."""
    codes, scales = codes.float().double().cpu(), scales.double().cpu().clone()
    x, slots = x.double().cpu(), slots.cpu().tolist()
    runs, i = [], 0
    while i < len(slots):
        if slots[i] < 0:
            i += 1
            continue
        j = i
        while j < len(slots) and slots[j] >= 0 and slots[j] // bt == slots[i] // bt:
            j += 1
        runs.append((i, j))
        i = j
    for i, j in runs:
        blk, off = slots[i] // bt, slots[i] % bt
        for h in range(x.shape[1]):
            top = x[i:j, h].abs()
            want = ref.scale_of(float(torch.where(top.isnan(), 0.0, top).max()))
            if off:
                old = float(scales[blk, h])
                if want > old:
                    codes[blk, h] = ref.e4m3(codes[blk, h] * (old / want))
                want = max(want, old)
            scales[blk, h] = want
            for t in range(i, j):
                codes[blk, h, slots[t] % bt] = ref.e4m3(x[t, h] / want)
    return codes, scales


@pytest.mark.parametrize("K,d", [(1, 64), (3, 128), (2, 64)])
@pytest.mark.parametrize("bt", [16, 32, 64, 128])
@pytest.mark.parametrize("lengths", [[1], [5, 0, 130], [300], [16, 64, 128, 1, 1]])
def test_append_prompts_then_tokens(sta, lengths, bt, K, d):
    """Prompts written whole, then single tokens of growing and falling size, each step bit for bit."""
    g = torch.Generator("cuda").manual_seed(bt + K)
    steps = 4
    table = tables_for([n + steps for n in lengths], bt, 40)
    kc, vc, ks, vs = empty_cache(40, K, bt, d, fill=0x7f)  # NaN codes: a block begun anew forgets them
    held = [0] * len(lengths)
    for step in range(steps + 1):
        new = lengths if step == 0 else [1] * len(lengths)
        if not sum(new):
            continue
        slots = torch.cat([slots_for(table[b], held[b], n, bt) for b, n in enumerate(new)])
        kv = torch.randn(sum(new), 2 * K, d, generator=g, device="cuda") * (1.0, 7.0, 0.01, 300.0, 1e-4)[step]
        kv = kv.bfloat16()
        k, v = kv[:, :K], kv[:, K:]
        want = [append_reference(x, slots, c, s, bt) for x, c, s in ((k, kc, ks), (v, vc, vs))]
        sta.sta_cache_append(k, v, slots, kc, vc, ks, vs)
        assert sta.sta_operator_status() == 0
        for (codes, scales), c, s in zip(want, (kc, vc), (ks, vs)):
            assert torch.equal(s.double().cpu(), scales)
            got = c.float().double().cpu()
            assert bool(((got == codes) | (got.isnan() & codes.isnan())).all())
        held = [a + b for a, b in zip(held, new)]


def test_append_skips_and_special_values(sta):
    bt, K, d = 16, 2, 64
    kc, vc, ks, vs = empty_cache(4, K, bt, d)
    x = torch.ones(6, K, d, dtype=torch.bfloat16, device="cuda")
    x[1, 0, 3] = float("nan")
    x[4, 1, 5] = float("inf")
    x[5] = 0.0
    x[5, 0, 0], x[5, 0, 1] = 2.0 ** -67, -(2.0 ** -72)  # representable, and under half of the smallest step
    slots = torch.tensor([0, 1, -1, 17, 33, 48], dtype=torch.int64, device="cuda")
    sta.sta_cache_append(x, -x, slots, kc, vc, ks, vs)
    k, v = values(kc, ks), values(vc, vs)
    assert sta.sta_operator_status() == 0
    assert bool(k[0, 0, 1, 3].isnan()) and int(k.isnan().sum()) == 1
    assert bool((k[0, :, 0] == 1.0).all()) and bool((v[0, :, 0] == -1.0).all())
    assert bool((k[1, :, 1] == 1.0).all()) and not bool(k[1, :, 0].any())
    assert float(ks[2, 1]) == 2.0 ** 120 and float(k[2, 1, 1, 5]) == 448.0 * 2.0 ** 120 and float(k[2, 0, 1, 5]) == 1.0
    assert float(ks[3, 0]) == 2.0 ** -60 and float(k[3, 0, 0, 0]) == 2.0 ** -67 and float(k[3, 0, 0, 1]) == 0.0


def test_append_slots_out_of_the_pool_are_reported(sta):
    bt, K, d = 16, 1, 64
    kc, vc, ks, vs = empty_cache(2, K, bt, d)
    x = torch.ones(3, K, d, dtype=torch.bfloat16, device="cuda")
    sta.sta_cache_append(x, x, torch.tensor([32, 5, 1 << 40], device="cuda"), kc, vc, ks, vs)
    assert sta.sta_operator_status() == sta.STA_ERR_BOUNDS
    assert sta.sta_operator_status() == 0
    assert int(values(kc, ks).count_nonzero()) == d


def test_append_same_slot_in_a_row_keeps_the_last(sta):
    kc, vc, ks, vs = empty_cache(1, 1, 16, 64)
    x = torch.arange(1, 4, device="cuda").bfloat16()[:, None, None].expand(3, 1, 64).contiguous()
    sta.sta_cache_append(x, x, torch.tensor([4, 4, 4], device="cuda"), kc, vc, ks, vs)
    assert bool((values(kc, ks)[0, 0, 4] == 3.0).all())


# ---------------------------------------------------------------- extend
def extend_reference(new, lengths, tables, free, count, bt, max_slots):
    new, lengths, free = list(new), list(lengths), list(free)
    t2, out_len, pool, width = [list(r) for r in tables], list(lengths), len(free), len(tables[0])
    nothing = (tables, free, [-1] * max_slots, [0] * (len(new) + 1), lengths, count)
    if any(n < 0 or n + max(a, 0) > width * bt for n, a in zip(lengths, new)) or not 0 <= count <= pool or \
            sum(max(a, 0) for a in new) > max_slots:
        return nothing + (-1,)
    c = count
    for b, a in enumerate(new):
        if a < 0:
            for j in range(-(-lengths[b] // bt)):
                if c >= pool:
                    return nothing + (-1,)
                free[c] = tables[b][j]
                c += 1
            out_len[b] = 0
    slots, cu = [], [0]
    for b, a in enumerate(new):
        if a >= 0:
            for j in range(-(-lengths[b] // bt), -(-(lengths[b] + a) // bt)):
                c -= 1
                if c >= 0:
                    t2[b][j] = free[c]
            slots += [t2[b][p // bt] * bt + p % bt for p in range(lengths[b], lengths[b] + a)]
            out_len[b] += a
        cu.append(len(slots))
    if c < 0:
        return nothing + (-c,)
    return t2, free, slots + [-1] * (max_slots - len(slots)), cu, out_len, c, 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,hi,new_hi,bt,short", [(1, 0, 1, 16, 0), (3, 40, 20, 16, 0), (64, 500, 1, 64, 0),
                                                      (700, 90, 300, 128, 0), (5, 100, 60, 32, 2), (1500, 3, 2, 16, 0),
                                                      (8192, 20, 3, 16, 0), (200, 600, 1, 16, 50)])
def test_extend(sta, batch, hi, new_hi, bt, short, in_place):
    r = random.Random(batch * 31 + hi)
    lengths = [r.randint(0, hi) for _ in range(batch)]
    new = [r.choice([-1, 0, r.randint(0, new_hi), r.randint(1, new_hi)]) if batch > 1 else new_hi for _ in range(batch)]
    held = [-(-n // bt) for n in lengths]
    need = sum(-(-(n + a) // bt) - h for n, a, h in zip(lengths, new, held) if a >= 0)
    back = sum(h for a, h in zip(new, held) if a < 0)
    count = max(0, need - back + (3 if not short else -short))
    pool = sum(held) + count + 2
    ids = list(range(pool))
    r.shuffle(ids)
    width = -(-(hi + new_hi) // bt) + 1
    tables, at = [], 0
    for h in held:
        tables.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    free = ids[at:at + count] + [-7] * (pool - count)
    max_slots = sum(max(a, 0) for a in new) + 5
    want = extend_reference(new, lengths, tables, free, count, bt, max_slots)

    def dev(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    t, f, n, c = dev(tables), dev(free), dev(lengths), dev([count])
    s = sta.sta_cache_extend(dev(new), n, t, f, c, bt, max_slots, in_place=in_place)
    torch.cuda.synchronize()
    got = (t.tolist(), f.tolist(), s.slots.tolist(), s.cu_new.tolist(), s.lengths.tolist(), int(s.free_count), int(s.short))
    for name, a, b in zip(("tables", "free", "slots", "cu", "lengths", "count", "short"), got, want):
        assert a == b, name
    assert (s.lengths is n) == in_place and (n.tolist() == lengths) == (not in_place or want[4] == lengths)


def test_extend_refuses_on_the_device(sta):
    """Lengths, counts and totals out of range change nothing and say -1."""
    def dev(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    for new, lengths, count, max_slots in (([1, 2], [5, -1], 3, 9), ([1, 2], [5, 65], 3, 9), ([1, 60], [5, 5], 3, 99),
                                           ([1, 2], [5, 5], -1, 9), ([1, 2], [5, 5], 5, 9), ([1, 9], [5, 5], 2, 9),
                                           ([2 ** 31 - 1, 2 ** 31 - 1], [5, 5], 3, 9), ([-1, 2], [17, 5], 3, 9)):
        t, f = dev([[0, 1, 2, 3], [0, 1, 2, 3]]), dev([9, 8, 7, 6])
        s = sta.sta_cache_extend(dev(new), dev(lengths), t, f, dev([count]), 16, max_slots)
        assert int(s.short) == -1 and s.lengths.tolist() == lengths and int(s.free_count) == count
        assert s.cu_new.tolist() == [0, 0, 0] and set(s.slots.tolist()) <= {-1}
        assert t.tolist() == [[0, 1, 2, 3]] * 2 and f.tolist() == [9, 8, 7, 6]


# ---------------------------------------------------------------- attention
def filled_cache(lengths, K, bt, d, seed, spread=1.0, blocks=None):
    """A cache of random codes and power-of-two scales (every code of the pool drawn, tails included)."""
    g = torch.Generator("cuda").manual_seed(seed)
    need = sum(-(-n // bt) for n in lengths)
    blocks = blocks or need + 3
    out = []
    for _ in range(2):
        x = torch.randn(blocks, K, bt, d, generator=g, device="cuda")
        out.append((x * 100).clamp(-448, 448).to(torch.float8_e4m3fn))  # past 448 a cast gives NaN
    scales = [torch.exp2(torch.round(torch.randn(blocks, K, generator=g, device="cuda") * spread - 7)) for _ in range(2)]
    return out[0], out[1], scales[0], scales[1], tables_for(lengths, bt, blocks, seed=seed)


def attention_reference(q, kc, vc, ks, vs, table, lengths, lens_q, scale, bt):
    """One 64-bit reference for each sequence and key head, packed like the call's outputs."""
    T, H, d = q.shape
    K = kc.shape[1]
    G = H // K
    out = {n: torch.zeros(T, H, d, dtype=torch.float64, device="cuda") for n in ("o", "o_tol")}
    out["lse"] = torch.full((H, T), -math.inf, dtype=torch.float64, device="cuda")
    out["lse_tol"] = torch.zeros_like(out["lse"])
    a = 0
    for b, (n, m) in enumerate(zip(lens_q, lengths)):
        page = table[b, :-(-m // bt)].long()
        raw = lambda c: c.view(torch.uint8)[page].view(torch.float8_e4m3fn).float()  # noqa: E731
        k, v = raw(kc) * ks[page][..., None, None], raw(vc) * vs[page][..., None, None]
        for h in range(K):
            hs = slice(h * G, h * G + G)
            unit = vs[page, h].repeat_interleave(bt)[:m]
            r = ref.one_sequence(q[a:a + n, hs].transpose(0, 1), k[:, h].reshape(-1, d)[:m], v[:, h].reshape(-1, d)[:m],
                                 True, scale, p_step=ref.H16, v_unit=unit)
            for name in ("o", "o_tol"):
                out[name][a:a + n, hs] = r[name].transpose(0, 1)
            for name in ("lse", "lse_tol"):
                out[name][hs, a:a + n] = r[name]
        a += n
    return out


@pytest.mark.parametrize("bt", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,K,d", [(2, 2, 64), (24, 8, 128), (8, 1, 64), (10, 2, 128), (20, 1, 128)])
@pytest.mark.parametrize("lengths,lens_q", [([1], None), ([16, 17, 31, 300], None), ([1000], [5]), ([2500, 3, 64], [1, 3, 2]),
                                            ([40, 0, 129], [0, 0, 7]), ([4, 700], [9, 33])])
def test_attention(sta, lengths, lens_q, heads, K, d, bt):
    lens_q = lens_q or [1] * len(lengths)
    kc, vc, ks, vs, table = filled_cache(lengths, K, bt, d, seed=bt + heads)
    q = torch.randn(sum(lens_q), heads, d, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    scale = 1 / math.sqrt(d)
    want = attention_reference(q, kc, vc, ks, vs, table, lengths, lens_q, scale, bt)
    o, lse = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, cu_q=ref.cu_of(lens_q))
    assert sta.sta_operator_status() == 0
    ref.check(o, want, "o")
    ref.check(lse, want, "lse")
    if lens_q == [1] * len(lengths):
        o1, lse1 = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n)
        assert torch.equal(o1, o) and torch.equal(lse1, lse)


@pytest.mark.parametrize("batch,hi", [(1, 20000), (70, 900), (3, 9000)])
def test_attention_split_over_long_caches(sta, batch, hi):
    r = random.Random(batch)
    lengths = [hi] + [r.randint(1, hi) for _ in range(batch - 1)]
    kc, vc, ks, vs, table = filled_cache(lengths, 2, 64, 128, seed=batch)
    q = torch.randn(batch, 6, 128, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want = attention_reference(q, kc, vc, ks, vs, table, lengths, [1] * batch, 0.1, 64)
    o, lse = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, softmax_scale=0.1)
    ref.check(o, want, "o")
    ref.check(lse, want, "lse")
    again = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, softmax_scale=0.1)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("gain", [1e-30, 1.0, 30.0, 1e20])
def test_attention_scales_far_apart(sta, gain):
    """Blocks whose scales differ by 2^30 and queries far outside fp16: the block that matters is not lost."""
    lengths, K, bt, d = [400], 2, 16, 64
    kc, vc, ks, vs, table = filled_cache(lengths, K, bt, d, seed=7, spread=0.0)
    vs *= torch.exp2(torch.round(torch.linspace(-30, 0, vs.shape[0], device="cuda")))[:, None]
    q = (torch.randn(1, 4, d, generator=torch.Generator("cuda").manual_seed(2), device="cuda") * gain).bfloat16()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    scale = 0.1 / gain if gain != 30.0 else 0.1
    want = attention_reference(q, kc, vc, ks, vs, table, lengths, [1], scale, bt)
    o, lse = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, softmax_scale=scale)
    ref.check(o, want, "o")
    ref.check(lse, want, "lse")


def test_attention_never_reads_behind_the_last_token(sta):
    """NaN codes and scales wherever no token is held change nothing."""
    lengths, K, bt, d = [70, 5], 2, 64, 128
    kc, vc, ks, vs, table = filled_cache(lengths, K, bt, d, seed=3)
    q = torch.randn(2, 4, d, device="cuda").bfloat16()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n)
    held = torch.zeros(kc.shape[0], bt, dtype=torch.bool, device="cuda")
    for b, m in enumerate(lengths):
        for j in range(-(-m // bt)):
            held[int(table[b, j]), :min(bt, m - j * bt)] = True
    for c in (kc, vc):
        c.view(torch.uint8)[~held[:, None, :].expand(-1, K, -1)] = 0x7f
    for s in (ks, vs):
        s[~held.any(1)] = float("nan")
    got = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("heads,K,d", [(4, 4, 64), (8, 2, 128), (24, 1, 128)])
@pytest.mark.parametrize("held,drafts", [(9, 9), (40, 6), (2000, 17)])
def test_attention_drafts_that_a_query_does_not_see_do_not_count(sta, held, drafts, heads, K, d):
    """NaN in a drafted token's keys or values: the queries before it keep their bits; those that see it have NaN, from
    its values in that column alone."""
    lengths, bt = [held, 33], 16
    kc, vc, ks, vs, table = filled_cache(lengths, K, bt, d, seed=held)
    lens_q = [drafts, 1]
    q = torch.randn(drafts + 1, heads, d, generator=torch.Generator("cuda").manual_seed(3), device="cuda").bfloat16()
    n, cu = torch.tensor(lengths, dtype=torch.int32, device="cuda"), ref.cu_of(lens_q)
    want, want_lse = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, cu)
    hk, c = K - 1, d - 5
    mine = torch.arange(hk * (heads // K), (hk + 1) * (heads // K), device="cuda")
    rest = [x for x in range(d) if x != c]
    for i in {0, drafts // 2, drafts - 1}:
        pos = held - drafts + i
        at = (int(table[0, pos // bt]), hk, pos % bt)
        for code in (0x7f, 0xff):
            bad = vc.clone()
            bad.view(torch.uint8)[at + (c,)] = code
            o, lse = sta.sta_cache_attention(q, kc, bad, ks, vs, table, n, cu)
            assert torch.equal(lse, want_lse)
            sees = torch.zeros_like(o, dtype=torch.bool)
            sees[i:drafts, mine, c] = True
            assert torch.equal(torch.where(sees, 0, o), torch.where(sees, 0, want)) and bool(o[sees].isnan().all())
            bad = kc.clone()
            bad.view(torch.uint8)[at + (c,)] = code
            o, lse = sta.sta_cache_attention(q, bad, vc, ks, vs, table, n, cu)
            sees[i:drafts, mine] = True
            assert torch.equal(torch.where(sees, 0, o), torch.where(sees, 0, want)) and bool(o[sees].isnan().all())


def test_attention_blocks_out_of_the_pool_are_not_seen(sta):
    lengths, K, bt, d = [100, 64], 1, 16, 64
    kc, vc, ks, vs, table = filled_cache(lengths, K, bt, d, seed=5)
    q = torch.randn(2, 2, d, device="cuda").bfloat16()
    # a bad id in the last block: as if the sequence ended before it
    short = torch.tensor([96, 64], dtype=torch.int32, device="cuda")
    want = sta.sta_cache_attention(q, kc, vc, ks, vs, table, short)
    for bad in (-1, kc.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 6] = bad
        got = sta.sta_cache_attention(q, kc, vc, ks, vs, t, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
        assert sta.sta_operator_status() == sta.STA_ERR_BOUNDS
        tol = 2 * ref.U * want[0].double().abs() + 2.0 ** -9
        assert bool(((got[0].double() - want[0].double()).abs() <= tol).all())
    # lengths past the table: its tokens count, no more
    n = torch.tensor([7 * bt + 5, 64], dtype=torch.int32, device="cuda")
    got = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n)
    assert sta.sta_operator_status() == sta.STA_ERR_BOUNDS and bool(got[0].isfinite().all())


def test_rows_behind_the_last_query_stay(sta):
    lengths, bt, d = [50, 20], 16, 64
    kc, vc, ks, vs, table = filled_cache(lengths, 1, bt, d, seed=6)
    q = torch.randn(9, 2, d, device="cuda").bfloat16()
    n, cu = torch.tensor(lengths, dtype=torch.int32, device="cuda"), ref.cu_of([2, 3])
    o, lse = torch.full_like(q, 7.0), torch.full((2, 9), 7.0, device="cuda")
    sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, cu_q=cu, o=o, lse=lse)
    assert bool((o[5:] == 7).all()) and bool((lse[:, 5:] == 7).all()) and not bool((o[:5] == 7).all(2).any())
    o2, lse2 = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, cu_q=cu)
    assert torch.equal(o2[:5], o[:5]) and not bool(o2[5:].any()) and bool((lse2[:, 5:] == -math.inf).all())


def test_pool_past_32_bits(sta):
    """A pool whose codes pass 2^32 bytes: append and attention in its last blocks."""
    bt, K, d, blocks = 128, 4, 128, (1 << 32) // (128 * 4 * 128) + 9
    kc, vc = (torch.empty(blocks, K, bt, d, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(blocks, K, device="cuda") for _ in range(2))
    n = 300
    ids = torch.tensor([[blocks - 1, blocks - 4, blocks - 2]], dtype=torch.int32, device="cuda")
    low = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    kv = torch.randn(n, 2 * K, d, generator=torch.Generator("cuda").manual_seed(4), device="cuda").bfloat16()
    q = torch.randn(1, 8, d, device="cuda").bfloat16()
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = []
    for table in (ids, low):
        sta.sta_cache_append(kv[:, :K], kv[:, K:], slots_for(table[0], 0, n, bt), kc, vc, ks, vs)
        out.append(sta.sta_cache_attention(q, kc, vc, ks, vs, table, lengths))
    assert sta.sta_operator_status() == 0
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1]) and bool(out[0][0].any())


def test_empty_calls(sta):
    kc, vc, ks, vs = empty_cache(4, 2, 16, 64)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    free, count = torch.arange(4, dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda")
    s = sta.sta_cache_extend(e, e, torch.empty(0, 5, dtype=torch.int32, device="cuda"), free, count, 16, 3)
    assert s.slots.tolist() == [-1] * 3 and s.cu_new.tolist() == [0] and int(s.free_count) == 3 and int(s.short) == 0
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    sta.sta_cache_append(x, x, torch.empty(0, dtype=torch.int64, device="cuda"), kc, vc, ks, vs)
    o, lse = sta.sta_cache_attention(torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), kc, vc, ks, vs,
                                     torch.empty(0, 5, dtype=torch.int32, device="cuda"), e)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    # queries behind no sequence at all
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = sta.sta_cache_attention(q, kc, vc, ks, vs, torch.empty(0, 5, dtype=torch.int32, device="cuda"), e,
                                     cu_q=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert not bool(o.any()) and bool((lse == -math.inf).all())


def test_many_requests(sta):
    """More requests than one pass of the lengths takes, with and without queries of their own."""
    r = random.Random(2)
    lengths = [r.randint(0, 90) for _ in range(700)]
    lens_q = [min(n, r.choice([0, 1, 1, 2])) for n in lengths]
    kc, vc, ks, vs, table = filled_cache(lengths, 1, 16, 64, seed=9)
    q = torch.randn(sum(lens_q), 4, 64, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want = attention_reference(q, kc, vc, ks, vs, table, lengths, lens_q, 0.125, 16)
    o, lse = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, cu_q=ref.cu_of(lens_q))
    ref.check(o, want, "o")
    ref.check(lse, want, "lse")


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_clean(sta):
    lengths, K, bt, d = [3000, 5, 800], 2, 64, 128
    kc, vc, ks, vs, table = filled_cache(lengths, K, bt, d, seed=3)
    q = torch.randn(3, 6, d, device="cuda").bfloat16()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n)
    sta.sta_debug_inject_operator_timeout(1, 20)
    try:
        sta.sta_cache_attention(q, kc, vc, ks, vs, table, n)
        assert sta.sta_operator_status() == sta.STA_ERR_TIMEOUT
    finally:
        sta.sta_debug_inject_operator_timeout(0)
    got = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n)
    assert sta.sta_operator_status() == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("H,K,d,bt", [(6, 2, 128, 16), (8, 1, 64, 64)])
def test_serving_prompts_and_tokens(sta, H, K, d, bt):
    """Prompts through packed attention and into the cache, then a captured step (tables, append, attention)
    replayed token by token; requests end and others take their blocks.  Each step's attention is checked
    against the cache's own values."""
    pool, width, B = 40, 12, 3
    kc, vc, ks, vs = empty_cache(pool, K, bt, d, fill=0x7f)
    tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pool, device="cuda", generator=torch.Generator("cuda").manual_seed(0)).int()
    count = torch.tensor([pool], dtype=torch.int32, device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    prompt = [37, 1, 64]
    qkv = torch.randn(sum(prompt), H + 2 * K, d, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    step = sta.sta_cache_extend(torch.tensor(prompt, dtype=torch.int32, device="cuda"), lengths, tables, free, count, bt,
                                sum(prompt), in_place=True)
    assert int(step.short) == 0
    o, lse = sta.sta_packed_attention(q, k, v, step.cu_new)
    want = ref.packed(q, k, v, prompt, prompt, True, 1 / math.sqrt(d))
    ref.check(o, want, "o")
    ref.check(lse, want, "lse")
    sta.sta_cache_append(k, v, step.slots, kc, vc, ks, vs)
    # the whole prompt again, over the cache: the keys' rounding aside it is the same attention
    o8, _ = sta.sta_cache_attention(q, kc, vc, ks, vs, tables, lengths, cu_q=step.cu_new)
    ref.check(o8, attention_reference(q, kc, vc, ks, vs, tables, prompt, prompt, 1 / math.sqrt(d), bt), "o")
    assert float((o8.double() - want["o"]).norm() / want["o"].norm()) < 0.2
    new = torch.ones(B, dtype=torch.int32, device="cuda")
    x = torch.zeros(B, H + 2 * K, d, dtype=torch.bfloat16, device="cuda")

    def one():
        s = sta.sta_cache_extend(new, lengths, tables, free, count, bt, B, in_place=True)
        sta.sta_cache_append(x[:, H:H + K], x[:, H + K:], s.slots, kc, vc, ks, vs)
        return s, sta.sta_cache_attention(x[:, :H], kc, vc, ks, vs, tables, lengths, cu_q=s.cu_new)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s, (o, lse) = one()
    held = list(prompt)
    for i in range(40):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        if i == 11:
            new[0] = -1
        elif i == 12:
            new[0] = 0
        elif i == 20:
            new[0] = 1
        graph.replay()
        torch.cuda.synchronize()
        now = new.tolist()
        held = [0 if a < 0 else n + a for n, a in zip(held, now)]
        assert int(s.short) == 0 and lengths.tolist() == held
        blocks = sum(-(-n // bt) for n in held)
        assert int(count) == pool - blocks
        used = [int(tables[b, j]) for b in range(B) for j in range(-(-held[b] // bt))] + free[:int(count)].tolist()
        assert sorted(used) == list(range(pool))
        rows = [max(a, 0) for a in now]
        if i % 7 == 0 or i in (11, 12, 20, 39):
            want = attention_reference(x[:sum(rows), :H], kc, vc, ks, vs, tables, held, rows, 1 / math.sqrt(d), bt)
            ref.check(o[:sum(rows)], want, "o")
            ref.check(lse[:, :sum(rows)], want, "lse")
    assert sta.sta_operator_status() == 0
    del graph


def test_extend_the_largest_tables(sta):
    """The most requests a step may have, with slots enough for every CTA, against a plain loop."""
    B, bt, width = 8192, 16, 4
    r = random.Random(5)
    lengths = [r.randint(0, 40) for _ in range(B)]
    new = [r.choice((-1, 0, 1, 1, 3, 20)) for _ in range(B)]
    pool = sum(-(-n // bt) for n in lengths) + 8192
    ids = list(range(pool))
    r.shuffle(ids)
    table = [[-1] * width for _ in range(B)]
    for b, n in enumerate(lengths):
        for j in range(-(-n // bt)):
            table[b][j] = ids.pop()
    free = ids + [-1] * (pool - len(ids))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    t, f = i32(table), i32(free)
    step = sta.sta_cache_extend(i32(new), i32(lengths), t, f, i32([len(ids)]), bt, sum(max(n, 0) for n in new) + 500)
    for b, n in enumerate(new):
        if n < 0:
            ids += table[b][:-(-lengths[b] // bt)]
    slots, held = [], []
    for b, n in enumerate(new):
        for pos in range(lengths[b], lengths[b] + max(n, 0)):
            if pos % bt == 0:
                table[b][pos // bt] = ids.pop()
            slots.append(table[b][pos // bt] * bt + pos % bt)
        held.append(0 if n < 0 else lengths[b] + n)
    assert int(step.short) == 0 and int(step.free_count) == len(ids) and step.lengths.tolist() == held
    assert step.slots.tolist() == slots + [-1] * 500 and f[:len(ids)].tolist() == ids
    assert step.cu_new.tolist() == [0] + [sum(max(n, 0) for n in new[:i + 1]) for i in range(B)]
    got = t.tolist()
    for b, n in enumerate(held):
        assert got[b][:-(-n // bt)] == table[b][:-(-n // bt)]


def test_extend_over_a_cluster_first_called_inside_a_capture():
    """A fresh process captures a step of many slots (a cluster of CTAs) before any other call."""
    code = """
import torch
import sparse_attention_video_sta_b200 as sta
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
new, n, free, count = i32([9000, 3, -1]), i32([5, 0, 40]), torch.arange(700, dtype=torch.int32, device="cuda"), i32([600])
table = torch.arange(100, 100 + 3 * 600, dtype=torch.int32, device="cuda").view(3, 600) % 700
torch.cuda.synchronize()
def run():
    t, f = table.clone(), free.clone()
    return (t, f) + tuple(sta.sta_cache_extend(new, n, t, f, count, 16, 20000))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
want = run()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and int(want[-1]) == 0 and int((want[2] >= 0).sum()) == 9003
del graph
print("fine")
"""
    import os
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-3000:]


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("given", [(), ("o",), ("lse",), ("o", "lse")], ids=lambda g: "-".join(g) or "none")
@pytest.mark.parametrize("lens_q", [[2, 3], [0, 0], []])
def test_rows_of_no_sequence_in_given_and_new_outputs(sta, lens_q, given, side):
    """Given tensors keep the rows behind the last query, new ones have zeros and -inf there, in every mixture and
    without any sequence."""
    B = len(lens_q)
    kc, vc, ks, vs, table = filled_cache([50, 20], 1, 16, 64, seed=6)
    q = torch.randn(9, 2, 64, device="cuda").bfloat16()
    n, cu = torch.tensor([50, 20][:B], dtype=torch.int32, device="cuda"), ref.cu_of(lens_q)
    args, used = (q, kc, vc, ks, vs, table[:B], n), sum(lens_q)
    want = sta.sta_cache_attention(*args, cu_q=cu)
    # memory that is handed out again holds something else than zeros and -inf
    for t in [torch.full_like(q, 3.0), torch.full((2, 9), 3.0, device="cuda")]:
        del t
    kw = {"o": torch.full_like(q, 7.0), "lse": torch.full((2, 9), 7.0, device="cuda")}
    kw = {name: t for name, t in kw.items() if name in given}
    torch.cuda.synchronize()
    s = torch.cuda.Stream() if side else None
    if side:
        with torch.cuda.stream(s):
            torch.full_like(q, 3.0), torch.full((2, 9), 3.0, device="cuda")
    o, lse = sta.sta_cache_attention(*args, cu_q=cu, stream=s, **kw)
    torch.cuda.synchronize()
    assert sta.sta_operator_status() == 0
    assert torch.equal(o[:used], want[0][:used]) and torch.equal(lse[:, :used], want[1][:, :used])
    assert bool((o[used:] == (7.0 if "o" in given else 0.0)).all())
    assert bool((lse[:, used:] == (7.0 if "lse" in given else -math.inf)).all())
    assert all(t is kw[name] for name, t in (("o", o), ("lse", lse)) if name in kw)


@pytest.mark.parametrize("heads,K,d", [(4, 2, 64), (24, 8, 128), (16, 1, 64)])
@pytest.mark.parametrize("batch", [1, 2, 3, 64, 256, 257, 700, 1500])
def test_attention_bounds_that_fall_are_cut_and_reported(sta, batch, heads, K, d):
    """Bounds of the queries that fall or leave the tensors: the call is the one with the bounds made rising, and says
    BOUNDS; no row is written by two sequences."""
    r = random.Random(batch + heads)
    T = 2 * batch + 5
    lengths = [r.randint(0, 60) for _ in range(batch - 1)] + [2500]
    kc, vc, ks, vs, table = filled_cache(lengths, K, 16, d, seed=9)
    q = torch.randn(T, heads, d, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    steady = [min(T, 2 * i) for i in range(batch + 1)]
    for trial in range(4):
        bad = list(steady)
        for i in ([batch] if trial == 0 else [r.randint(1, batch) for _ in range(1 + batch // 5)]):
            bad[i] = r.choice([-7, 0, 1, T, T + 9, 2 ** 31 - 1, -2 ** 31, r.randint(0, T), max(0, bad[i - 1] - 1)])
        if trial == 1:
            bad[1:] = bad[:0:-1]
        cut, top = [], 0
        for c in bad:
            top = max(top, min(c, T))
            cut.append(top)
        cu, want_cu = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (bad, cut))
        for given in (False, True):
            kw = [dict(o=torch.full_like(q, 7.0), lse=torch.full((heads, T), 7.0, device="cuda")) if given else {} for _ in range(2)]
            want = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, cu_q=want_cu, **kw[0])
            assert sta.sta_operator_status() == 0
            got = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, cu_q=cu, **kw[1])
            assert sta.sta_operator_status() == (sta.STA_ERR_BOUNDS if bad != cut else 0)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("batch", [1, 2, 300])
@pytest.mark.parametrize("given", [False, True])
def test_queries_before_the_first_sequence_are_no_ones(sta, batch, given):
    """A first bound above 0 is reported; the rows before it are zeros in new tensors, left alone in given ones."""
    lengths, lens_q = [5 + i % 40 for i in range(batch)], [1 + i % 3 for i in range(batch)]
    kc, vc, ks, vs, table = filled_cache(lengths, 2, 16, 64, seed=6)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    first, tail = 4, 3
    q = torch.randn(first + sum(lens_q) + tail, 8, 64, device="cuda").bfloat16()
    cu = ref.cu_of(lens_q)
    rows = slice(first, first + sum(lens_q))
    want = attention_reference(q[rows], kc, vc, ks, vs, table, lengths, lens_q, 0.125, 16)
    kw = dict(o=torch.full_like(q, 7.0), lse=torch.full((8, q.shape[0]), 7.0, device="cuda")) if given else {}
    for t in [torch.full_like(q, 3.0), torch.full((8, q.shape[0]), 3.0, device="cuda")]:
        del t
    o, lse = sta.sta_cache_attention(q, kc, vc, ks, vs, table, n, cu_q=cu + first, **kw)
    assert sta.sta_operator_status() == sta.STA_ERR_BOUNDS
    ref.check(o[rows], want, "o")
    ref.check(lse[:, rows], want, "lse")
    others = [i for i in range(q.shape[0]) if not rows.start <= i < rows.stop]
    assert bool((o[others] == (7.0 if given else 0.0)).all())
    assert bool((lse[:, others] == (7.0 if given else -math.inf)).all())


def test_extend_from_several_threads_at_once(sta):
    """Steps of different sizes (shared memory from a few bytes to the most) called at the same time, each on its
    own stream: none changes what another's launch needs."""
    from concurrent.futures import ThreadPoolExecutor
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    free, count = torch.arange(8192, dtype=torch.int32, device="cuda"), i32([8192])

    def steps(batch):
        lengths, new = i32([5] * batch), i32([12] * batch)  # 17 tokens: one block more of 16
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(150):
                t, f = torch.zeros(batch, 2, dtype=torch.int32, device="cuda"), free.clone()
                s = sta.sta_cache_extend(new, lengths, t, f, count, 16, 12 * batch)
            torch.cuda.current_stream().synchronize()
        return int(s.short), int(s.free_count), s.slots[-1].item()
    torch.cuda.synchronize()
    sizes = [8192, 3100, 4000, 8192, 6000, 100, 3500, 5000]
    with ThreadPoolExecutor(len(sizes)) as pool:
        got = list(pool.map(steps, sizes))
    for batch, (short, left, slot) in zip(sizes, got):
        # the last request's last token is the first of its new block, the batch-th from the top
        assert short == 0 and left == 8192 - batch and slot == (8192 - batch) * 16


@pytest.mark.parametrize("before", [0, 1, 15, 40])
@pytest.mark.parametrize("bt,d", [(16, 64), (32, 128), (128, 128)])
def test_append_slots_named_twice(sta, bt, d, before):
    """Slots of a block named again keep the later token, wherever in the run; a run longer than a block is cut at
    one block's worth and reported."""
    K, blocks = 2, 60
    for extra in (0, 1, 2 * bt):  # tokens past a block's worth
        names = [3, 3] + list(range(4, bt)) + [3, 7]
        names = (names + [5] * (bt + extra))[:bt + extra]
        slots = [(10 + i) * bt for i in range(before)] + names + [5 * bt, 5 * bt + 1]
        # many tokens of other blocks behind, so that more than one range is taken
        slots += [6 * bt + i for i in range(bt)] + [-1] * 9
        g = torch.Generator("cuda").manual_seed(bt + before)
        x = torch.randn(len(slots), K, d, generator=g, device="cuda").bfloat16()
        kc, vc, ks, vs = empty_cache(blocks, K, bt, d)
        sta.sta_cache_append(x, -x, torch.tensor(slots, dtype=torch.int64, device="cuda"), kc, vc, ks, vs)
        assert sta.sta_operator_status() == (sta.STA_ERR_BOUNDS if extra else 0)
        taken = {s: i for i, s in list(enumerate(slots))[before:before + bt]}
        taken.update({s: i for i, s in enumerate(slots) if s >= bt})
        for codes, scales, sign in ((kc, ks, 1), (vc, vs, -1)):
            got = values(codes, scales).transpose(1, 2).reshape(blocks * bt, K, d)
            for b in sorted({s // bt for s in taken}):
                mine = [s for s in taken if s // bt == b]
                used = range(before, before + bt) if b == 0 else [taken[s] for s in mine]
                for h in range(K):
                    scale = ref.scale_of(max(float(x[i, h].abs().max()) for i in used))
                    assert float(scales[b, h]) == scale
                    for s in mine:
                        assert torch.equal(got[s, h], ref.e4m3(sign * x[taken[s], h].double() / scale) * scale)
            rest = sorted(set(range(blocks * bt)) - set(taken))
            assert not bool(got[rest].any())
