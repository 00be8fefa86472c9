"""Packed attention (forward, backward, autograd) against a 64-bit reference with bounds derived from the
roundings that the kernels make (prompt_ref.py)."""
import math

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


def make(lens_q, lens_k, heads, kv_heads, d, seed=0, tail=0, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(t, h):
        return (gain * torch.randn(t + tail, h, d, generator=g, device="cuda")).bfloat16()
    q, k, v = randn(sum(lens_q), heads), randn(sum(lens_k), kv_heads), randn(sum(lens_k), kv_heads)
    return q, k, v, randn(sum(lens_q), heads)


# (query lengths, key lengths or None for the same)
LENGTHS = [
    ([1], None), ([2], None), ([127, 128, 129], None), ([0, 5, 0, 300, 1], None), ([64], [513]),
    ([1, 1, 1], [7, 200, 1025]), ([50, 200, 10], [20, 60, 0]), ([0, 3], [9, 0]), ([700], None), ([33, 1, 385, 77], None),
    ([3, 260], [400, 129]),
]
HEADS = [(2, 2, 64), (6, 2, 128), (8, 1, 64), (10, 2, 128), (3, 3, 128)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,kv_heads,d", HEADS)
@pytest.mark.parametrize("lens_q,lens_k", LENGTHS)
def test_forward_and_backward(sta, lens_q, lens_k, heads, kv_heads, d, causal):
    lens_k = lens_k or lens_q
    q, k, v, do = make(lens_q, lens_k, heads, kv_heads, d, seed=len(lens_q) + heads)
    cq, ck, scale = ref.cu_of(lens_q), ref.cu_of(lens_k), 1.0 / math.sqrt(d)
    want = ref.packed(q, k, v, lens_q, lens_k, causal, scale, do)
    o, lse = sta.sta_packed_attention(q, k, v, cq, ck, causal=causal)
    dq, dk, dv = sta.sta_packed_attention_backward(q, k, v, o, lse, do, cq, ck, causal=causal)
    assert sta.sta_operator_status() == 0
    for name, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(t, want, name)


@pytest.mark.parametrize("heads,kv_heads,d,n", [(128, 1, 64, 70), (100, 1, 128, 33), (40, 2, 64, 150), (14, 2, 128, 400),
                                                 (24, 8, 128, 2100)])
def test_many_heads_to_a_key_head(sta, heads, kv_heads, d, n):
    q, k, v, do = make([n, 3], [n, 3], heads, kv_heads, d, seed=5)
    cu = ref.cu_of([n, 3])
    want = ref.packed(q, k, v, [n, 3], [n, 3], True, 0.1, do)
    o, lse = sta.sta_packed_attention(q, k, v, cu, softmax_scale=0.1)
    grads = sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu, softmax_scale=0.1)
    for name, t in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads):
        ref.check(t, want, name)


def test_many_sequences(sta):
    """More sequences than one pass of the bounds' scan takes, most of them tiny."""
    lens = [(i * 7) % 5 for i in range(2500)] + [260]
    q, k, v, do = make(lens, lens, 2, 1, 64, seed=8)
    cu = ref.cu_of(lens)
    o, lse = sta.sta_packed_attention(q, k, v, cu)
    dq, dk, dv = sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu)
    assert sta.sta_operator_status() == 0
    want = ref.packed(q, k, v, lens, lens, True, 0.125, do)
    for name, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(t, want, name)


@pytest.mark.parametrize("gain,scale", [(6.0, 0.4), (0.01, 1.0), (3.0, 0.02)])
def test_large_and_small_scores(sta, gain, scale):
    """Scores of hundreds (rows dominated by one key, maxima that keep rising) and of nearly nothing."""
    lens = [400, 129]
    q, k, v, do = make(lens, lens, 4, 2, 64, seed=11, gain=gain)
    k[::7] *= 3
    cu = ref.cu_of(lens)
    o, lse = sta.sta_packed_attention(q, k, v, cu, softmax_scale=scale)
    grads = sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu, softmax_scale=scale)
    want = ref.packed(q, k, v, lens, lens, True, scale, do)
    for name, t in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads):
        ref.check(t, want, name)


def test_rising_scores_rescale(sta):
    """Every key's score above all before it, far past the first chunk's maximum."""
    n, d = 600, 64
    q, k, v, do = make([n], [n], 2, 1, d, seed=12)
    q[:] = 1.0
    k[:] = (torch.arange(n, device="cuda") * 0.05)[:, None, None].bfloat16()
    cu = ref.cu_of([n])
    want = ref.packed(q, k, v, [n], [n], False, 0.5, do)
    o, lse = sta.sta_packed_attention(q, k, v, cu, causal=False, softmax_scale=0.5)
    grads = sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu, causal=False, softmax_scale=0.5)
    for name, t in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads):
        ref.check(t, want, name)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nothing_of_other_sequences_or_the_tail_is_mixed_in(sta, bad):
    """Non-finite values in another sequence and behind the last one reach no row of the others."""
    lens = [100, 60, 171]
    q, k, v, do = make(lens, lens, 6, 2, 128, seed=3, tail=40)
    want = ref.packed(q, k, v, lens, lens, True, 0.1, do)
    for t in (q, k, v, do):
        t[100:160] = bad
        t[331:] = bad
    cu = ref.cu_of(lens)
    o, lse = sta.sta_packed_attention(q, k, v, cu, softmax_scale=0.1)
    dq, dk, dv = sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu, softmax_scale=0.1)
    assert sta.sta_operator_status() == 0
    for name, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        for rows in (slice(0, 100), slice(160, None)):
            assert bool(((t[rows].double() - want[name][rows]).abs() <= want[name + "_tol"][rows]).all()), name
    for rows in (slice(0, 100), slice(160, None)):
        ref.check(lse, want, "lse", rows)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_masked_scores_never_count(sta, bad):
    """A non-finite key is masked for the queries before it: those rows are as if it were not there."""
    n = 300
    q, k, v, do = make([n], [n], 2, 1, 64, seed=4)
    want = ref.packed(q, k, v, [n], [n], True, 0.125)
    k[200] = bad
    o, lse = sta.sta_packed_attention(q, k, v, ref.cu_of([n]))
    assert bool(((o[:200].double() - want["o"][:200]).abs() <= want["o_tol"][:200]).all())
    ref.check(lse, want, "lse", slice(0, 200))


def test_rows_behind_the_last_sequence_stay(sta):
    lens_q, lens_k = [40, 90], [77, 130]
    q, k, v, do = make(lens_q, lens_k, 4, 2, 64, seed=6, tail=29)
    cq, ck = ref.cu_of(lens_q), ref.cu_of(lens_k)
    o, dq, dk, dv = (torch.full_like(t, 7.0) for t in (q, q, k, v))
    lse = torch.full((4, q.shape[0]), 7.0, device="cuda")
    sta.sta_packed_forward(q, k, v, o, lse, cq, ck)
    sta.sta_packed_backward(q, k, v, o, lse, do, dq, dk, dv, cq, ck)
    for t, n in ((o, 130), (dq, 130), (dk, 207), (dv, 207)):
        assert bool((t[n:] == 7.0).all()) and not bool((t[:n] == 7.0).all(2).any())
    assert bool((lse[:, 130:] == 7.0).all())
    o2, lse2 = sta.sta_packed_attention(q, k, v, cq, ck)
    grads = sta.sta_packed_attention_backward(q, k, v, o2, lse2, do, cq, ck)
    assert torch.equal(o2[:130], o[:130]) and not bool(o2[130:].any()) and bool((lse2[:, 130:] == -math.inf).all())
    for t, u, n in zip(grads, (dq, dk, dv), (130, 207, 207)):
        assert torch.equal(t[:n], u[:n]) and not bool(t[n:].any())


def test_strides(sta):
    """Parts of a fused projection, head-major storage, and strided outputs give the bits of contiguous tensors."""
    lens, H, K, d = [65, 200, 7], 6, 2, 64
    T, cu = sum(lens), ref.cu_of([65, 200, 7])
    qkv = torch.randn(T, H + 2 * K, d, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    do = torch.randn(H, T, d, device="cuda").bfloat16().transpose(0, 1)
    o0, lse0 = sta.sta_packed_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    g0 = sta.sta_packed_attention_backward(q.contiguous(), k.contiguous(), v.contiguous(), o0, lse0, do.contiguous(), cu)
    o = torch.zeros(H, T + 3, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[:T]
    dqkv = torch.zeros(T, H + 2 * K, d + 8, dtype=torch.bfloat16, device="cuda")[..., :d]
    lse = torch.empty_like(lse0)
    sta.sta_packed_forward(q, k, v, o, lse, cu)
    sta.sta_packed_backward(q, k, v, o, lse, do, dqkv[:, :H], dqkv[:, H:H + K], dqkv[:, H + K:], cu)
    assert torch.equal(o, o0) and torch.equal(lse, lse0)
    for a, b in zip(g0, (dqkv[:, :H], dqkv[:, H:H + K], dqkv[:, H + K:])):
        assert torch.equal(a, b)


def test_same_bits_again_and_on_another_stream(sta):
    lens = [1000, 13, 400]
    q, k, v, do = make(lens, lens, 12, 4, 128, seed=9)
    cu = ref.cu_of(lens)

    def both(stream=None):
        o, lse = sta.sta_packed_attention(q, k, v, cu, stream=stream)
        return (o, lse) + sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu, stream=stream)
    first = both()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = [both(s) for s in streams * 3]
    torch.cuda.synchronize()
    for r in runs + [both()]:
        assert all(torch.equal(a, b) for a, b in zip(first, r))


def test_graphs_follow_new_bounds(sta):
    """One capture of forward and backward; replayed with other lengths in the same bounds array.  Two graphs
    replayed at the same time do not disturb each other."""
    T, H, K, d = 700, 4, 2, 64
    q, k, v, do = make([T], [T], H, K, d, seed=10)
    cus = [torch.tensor(c, dtype=torch.int32, device="cuda") for c in ([0, 700, 700, 700], [0, 0, 300, 700], [0, 129, 130, 700])]
    want = []
    for cu in cus:
        o, lse = sta.sta_packed_attention(q, k, v, cu)
        want.append((o, lse) + sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu))
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        cu = cus[0].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = sta.sta_packed_attention(q, k, v, cu)
            out = (o, lse) + sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu)
        graphs.append((g, cu, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, j in ((0, 1), (1, 2), (2, 0)):
        for n, s, (g, cu, _) in zip((i, j), streams, graphs):
            cu.copy_(cus[n])
        torch.cuda.synchronize()
        for s, (g, _, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for n, (_, _, out) in zip((i, j), graphs):
            assert all(torch.equal(a, b) for a, b in zip(out, want[n]))
    del graphs


def test_autograd_against_the_formula_and_differences(sta):
    """StaPackedAttention on broadcast and transposed inputs: gradients summed into the leaves, and the
    directional derivative of the 64-bit forward."""
    lens, H, K, d = [37, 140], 4, 2, 64
    T, cu = 177, ref.cu_of(lens)
    g = torch.Generator("cuda").manual_seed(2)
    q = torch.randn(H, T, d, generator=g, device="cuda").bfloat16().requires_grad_()
    kv = torch.randn(T, 1, 2 * d, generator=g, device="cuda").bfloat16().requires_grad_()  # one head for both key heads
    do = torch.randn(T, H, d, generator=g, device="cuda").bfloat16()
    o = sta.StaPackedAttention.apply(q.transpose(0, 1), kv[..., :d].expand(T, K, d), kv[..., d:].expand(T, K, d), cu)
    o.backward(do)
    kx, vx = kv.detach()[..., :d].expand(T, K, d), kv.detach()[..., d:].expand(T, K, d)
    r = ref.packed(q.detach().transpose(0, 1), kx, vx, lens, lens, True, 1 / math.sqrt(d), do)
    assert bool(((q.grad.transpose(0, 1).double() - r["dq"]).abs() <= r["dq_tol"]).all())
    for part, name in ((kv.grad[..., :d], "dk"), (kv.grad[..., d:], "dv")):
        want, tol = r[name].sum(1, keepdim=True), r[name + "_tol"].sum(1, keepdim=True)
        # the two heads' gradients are summed in bf16 by autograd: one more rounding
        assert bool(((part.double() - want).abs() <= tol + 2 * ref.U * (want.abs() + tol)).all())
    # central differences of the 64-bit loss along a random direction
    step = 1e-4
    u = [torch.randn(t.shape, generator=g, device="cuda").double() for t in (r["dq"], r["dk"], r["dv"])]

    def loss(s):
        x = [a.double() + s * b for a, b in zip((q.detach().transpose(0, 1), kx, vx), u)]
        return float((ref.packed(*x, lens, lens, True, 1 / math.sqrt(d))["o"] * do.double()).sum())
    slope = (loss(step) - loss(-step)) / (2 * step)
    o1, lse1 = sta.sta_packed_attention(q.detach().transpose(0, 1), kx.contiguous(), vx.contiguous(), cu)
    grads = sta.sta_packed_attention_backward(q.detach().transpose(0, 1), kx.contiguous(), vx.contiguous(), o1, lse1, do, cu)
    got = sum(float((a.double() * b).sum()) for a, b in zip(grads, u))
    bound = sum(float((r[n + "_tol"] * b.abs()).sum()) for n, b in zip(("dq", "dk", "dv"), u))
    assert abs(got - slope) <= bound + 1e-4 * (1 + abs(slope))


def test_backward_captured_while_an_eager_graph_lives(sta):
    """Autograd forward and backward captured into a CUDA graph on their own stream, on leaves of their own that
    share the storage of an eager graph still alive: the replay gives the eager gradients."""
    lens = [60, 200]
    q, k, v, do = make(lens, lens, 4, 2, 64, seed=13)
    cu = ref.cu_of(lens)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    eager = sta.StaPackedAttention.apply(*leaves, cu)
    want = torch.autograd.grad(eager, leaves, do, retain_graph=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fresh = [t.detach().requires_grad_() for t in leaves]
        torch.autograd.grad(sta.StaPackedAttention.apply(*fresh, cu), fresh, do)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = torch.autograd.grad(sta.StaPackedAttention.apply(*fresh, cu), fresh, do)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    again = torch.autograd.grad(eager, leaves, do)
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    del g


def test_empty_problems(sta):
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = sta.sta_packed_attention(q, k, k, cu)
    assert o.shape == q.shape and lse.shape == (4, 0)
    sta.sta_packed_attention_backward(q, k, k, o, lse, q, cu)
    # keys but no queries: zero gradients; queries but no keys: zeros and -inf
    k9 = torch.ones(9, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu0, cu9 = ref.cu_of([0, 0]), ref.cu_of([4, 5])
    _, dk, dv = sta.sta_packed_attention_backward(q, k9, k9, q, lse, q, cu0, cu9)
    assert not bool(dk.any()) and not bool(dv.any())
    q9 = torch.ones(9, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = sta.sta_packed_attention(q9, k, k, cu9, cu0, causal=False)
    assert not bool(o.any()) and bool((lse == -math.inf).all())
    dq, _, _ = sta.sta_packed_attention_backward(q9, k, k, o, lse, q9, cu9, cu0, causal=False)
    assert not bool(dq.any())
    assert sta.sta_operator_status() == 0


@pytest.mark.parametrize("cu_q,cu_k", [([0, 90, 40, 130], [0, 90, 40, 130]), ([0, 60, 500], [0, 60, 500]),
                                       ([-5, 60, 130], [-5, 60, 130]), ([0, 130], [0, 2 ** 31 - 1]),
                                       ([0, 60, 60, -1], [0, -7, 20, 130])])
def test_bounds_that_do_not_fit_are_cut_and_reported(sta, cu_q, cu_k):
    """Bounds that decrease or leave the tensors: the call is the one with the cut bounds, and says BOUNDS."""
    T, H, K, d = 130, 4, 2, 64
    q, k, v, do = make([T], [T], H, K, d, seed=14)

    def cut(c):
        out, top = [], 0
        for x in c:
            top = max(top, min(x, T))
            out.append(top)
        return torch.tensor(out, dtype=torch.int32, device="cuda")

    def both(a, b):
        o, lse = sta.sta_packed_attention(q, k, v, a, b)
        return (o, lse) + sta.sta_packed_attention_backward(q, k, v, o, lse, do, a, b)
    want = both(cut(cu_q), cut(cu_k))
    assert sta.sta_operator_status() == 0
    got = both(*(torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_k)))
    assert sta.sta_operator_status() == sta.STA_ERR_BOUNDS
    assert sta.sta_operator_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_sequences_clear_every_row(sta):
    q, k, v, do = make([5], [7], 4, 2, 64)
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = sta.sta_packed_attention(q, k, v, cu)
    assert not bool(o.any()) and bool((lse == -math.inf).all())
    for t in sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu):
        assert not bool(t.any())
    assert sta.sta_operator_status() == 0


@pytest.mark.parametrize("lens_q,lens_k,heads,kv_heads,d,causal", [
    ([5], [9000], 2, 1, 64, True), ([40, 1], [4100, 6000], 6, 2, 128, True), ([3000], [130], 4, 1, 128, False),
    ([2300], [2300], 8, 1, 64, True), ([1500, 60], [3000, 2900], 3, 1, 128, False)])
def test_long_walks_are_split_and_joined(sta, lens_q, lens_k, heads, kv_heads, d, causal):
    """Few blocks with long walks, over keys (forward, dQ) and over queries (dK, dV): split into parts."""
    q, k, v, do = make(lens_q, lens_k, heads, kv_heads, d, seed=21)
    k[::5] *= 2
    cq, ck, scale = ref.cu_of(lens_q), ref.cu_of(lens_k), 0.15
    want = ref.packed(q, k, v, lens_q, lens_k, causal, scale, do)
    o, lse = sta.sta_packed_attention(q, k, v, cq, ck, causal=causal, softmax_scale=scale)
    grads = sta.sta_packed_attention_backward(q, k, v, o, lse, do, cq, ck, causal=causal, softmax_scale=scale)
    assert sta.sta_operator_status() == 0
    for name, t in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads):
        ref.check(t, want, name)


def test_offsets_past_32_bits(sta):
    """Rows 2^27 elements apart: byte and element offsets past 2^32 and 2^31, in every tensor."""
    n, H, d, apart = 40, 2, 64, 1 << 27
    big = torch.empty((n - 1) * apart + 8 * H * d, dtype=torch.bfloat16, device="cuda")

    def rows(i):
        return big[i * H * d:].as_strided((n, H, d), (apart, d, 1))
    small = make([n], [n], H, H, d, seed=15)
    q, k, v, do, o, dq, dk, dv = (rows(i) for i in range(8))
    for a, b in zip((q, k, v, do), small):
        a.copy_(b)
    cu = ref.cu_of([n])
    want_o, want_lse = sta.sta_packed_attention(*small[:3], cu)
    want = sta.sta_packed_attention_backward(*small[:3], want_o, want_lse, small[3], cu)
    lse = torch.empty_like(want_lse)
    sta.sta_packed_forward(q, k, v, o, lse, cu)
    sta.sta_packed_backward(q, k, v, o, lse, do, dq, dk, dv, cu)
    assert torch.equal(o, want_o) and torch.equal(lse, want_lse)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), want))


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing of the calls' first-time set-up breaks a capture: a fresh process captures before it has
    made any call, and the replay gives the eager bits."""
    code = """
import torch, sys
sys.path.insert(0, "tests")
import sparse_attention_video_sta_b200 as sta
import prompt_ref as ref
torch.manual_seed(0)
lens = [300, 77] * 20
q, k, v, do = (torch.randn(sum(lens), h, 64, device="cuda").bfloat16() for h in (4, 2, 2, 4))
cu = ref.cu_of(lens)
table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
codes = [torch.zeros(40, 2, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
scales = [torch.ones(40, 2, device="cuda") for _ in range(2)]
n = torch.tensor([9, 300], dtype=torch.int32, device="cuda")
one = torch.ones(2, dtype=torch.int32, device="cuda")
free, count = torch.arange(8, dtype=torch.int32, device="cuda"), torch.tensor([8], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
def run():
    o, lse = sta.sta_packed_attention(q, k, v, cu)
    g = sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu)
    s = sta.sta_cache_extend(one, n, table.clone(), free.clone(), count, 16, 2)
    sta.sta_cache_append(k[:2], v[:2], s.slots, *codes, *scales)
    return (o, lse) + g + sta.sta_cache_attention(q[:2], *codes, *scales, table, n)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
want = run()
assert all(torch.equal(a, b) for a, b in zip(got, want)), [torch.equal(a, b) for a, b in zip(got, want)]
assert sta.sta_operator_status() == 0
del graph
print("fine")
"""
    import os
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-3000:]


@pytest.mark.parametrize("lens,d", [([700, 300], 128), ([60] * 40, 64), ([30, 5], 64), ([4000], 64)])
def test_a_wait_that_runs_out_is_reported_and_the_next_calls_are_clean(sta, lens, d):
    """Each kernel's load thread waits on a barrier that nothing arrives at, with a short limit: the kernels end,
    the status says so, and the same calls give their results again."""
    q, k, v, do = make(lens, lens, 4, 2, d, seed=16)
    cu = ref.cu_of(lens)

    def both():
        o, lse = sta.sta_packed_attention(q, k, v, cu)
        return (o, lse) + sta.sta_packed_attention_backward(q, k, v, want[0] if want else o, want[1] if want else lse, do, cu)
    want = None
    want = both()
    assert sta.sta_operator_status() == 0
    sta.sta_debug_inject_operator_timeout(1, 20)
    try:
        for call in (lambda: sta.sta_packed_attention(q, k, v, cu),
                     lambda: sta.sta_packed_attention_backward(q, k, v, want[0], want[1], do, cu)):
            call()
            assert sta.sta_operator_status() == sta.STA_ERR_TIMEOUT
    finally:
        sta.sta_debug_inject_operator_timeout(0)
    assert all(torch.equal(a, b) for a, b in zip(both(), want))
    assert sta.sta_operator_status() == 0


HIDDEN = [  # query lengths, key lengths, heads, key heads, d
    ([300, 77], [300, 77], 4, 4, 128), ([300, 77], [300, 77], 12, 4, 128), ([260, 9], [260, 9], 16, 2, 64),
    ([1500], [1500], 6, 2, 128), ([1000, 1000], [1000, 1000], 24, 8, 128), ([4000], [4000], 4, 4, 64),
    ([50, 200], [333, 120], 8, 2, 128), ([30], [30], 32, 1, 64),
]


def poison(t, head, row, elements):
    t = t.clone()
    for c, x in elements:
        t[row, head, c] = x
    return t


@pytest.mark.parametrize("nq,nk,H,K,d", HIDDEN, ids=lambda x: str(x).replace(" ", ""))
def test_what_a_causal_mask_hides_does_not_count(sta, nq, nk, H, K, d):
    """Infinities and NaN in tokens that a query does not see leave its results as they were, bit for bit, and so
    do those of a query for the keys that it does not see; whoever sees them gets them, in their column."""
    q, k, v, do = make(nq, nk, H, K, d, seed=31)
    cq, ck = ref.cu_of(nq), ref.cu_of(nk)
    G = H // K
    run = lambda q, k, v, do: (lambda o, l: (o, l) + sta.sta_packed_attention_backward(q, k, v, o, l, do, cq, ck))(
        *sta.sta_packed_attention(q, k, v, cq, ck))
    o0, l0, dq0, dk0, dv0 = run(q, k, v, do)
    odd = [(3, math.inf), (d - 1, math.nan), (17, -math.inf)]
    cols = [c for c, _ in odd]
    rest = [c for c in range(d) if c not in cols]
    hk = K - 1
    heads = list(range(hk * G, hk * G + G))
    others = [h for h in range(H) if h not in heads]
    a, ka = 0, 0
    for n, m in zip(nq, nk):
        first = max(0, m - n)  # the first query's own key
        for t in sorted({0, m // 2, m - 1, max(0, m - 2), min(m - 1, 129)}):
            sees = max(0, min(n, t - (m - n)))  # queries from this one on see key t
            rows, before = slice(a + sees, a + n), slice(a, a + sees)
            o, l, dq, dk, dv = run(q, k, poison(v, hk, ka + t, odd), do)
            assert torch.equal(l, l0) and torch.equal(o[:, others], o0[:, others])
            assert torch.equal(o[before], o0[before]) and torch.equal(dq[before], dq0[before])
            assert torch.equal(o[rows][:, heads][..., rest], o0[rows][:, heads][..., rest])
            assert not o[rows][:, heads][..., cols].isfinite().any()
            o, l, dq, dk, dv = run(q, poison(k, hk, ka + t, odd), v, do)
            assert torch.equal(o[before], o0[before]) and torch.equal(dq[before], dq0[before])
            assert torch.equal(dq[:, others], dq0[:, others]) and torch.equal(l[:, before], l0[:, before])
            assert not dq[rows][:, heads].isfinite().any()
        for i in sorted({0, n // 2, n - 1, min(n - 1, 43)}):
            seen = max(0, min(m, i + m - n + 1))
            h = heads[-1]
            behind, upto = slice(ka + seen, ka + m), slice(ka, ka + seen)
            _, _, _, dk, dv = run(q, k, v, poison(do, h, a + i, odd))
            assert torch.equal(dk[behind], dk0[behind]) and torch.equal(dv[behind], dv0[behind])
            assert torch.equal(dv[upto, hk][:, rest], dv0[upto, hk][:, rest])
            assert not dv[upto, hk][:, cols].isfinite().any() and not dk[upto, hk].isfinite().any()
            keep = [x for x in range(K) if x != hk]
            assert torch.equal(dk[:, keep], dk0[:, keep]) and torch.equal(dv[:, keep], dv0[:, keep])
            _, _, _, dk, dv = run(poison(q, h, a + i, [(3, math.nan), (8, math.inf)]), k, v, do)
            assert torch.equal(dk[behind], dk0[behind]) and torch.equal(dv[behind], dv0[behind])
            assert not dv[upto, hk].isfinite().any() and not dk[upto, hk].isfinite().any()
        a, ka = a + n, ka + m


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,K,d", [(8, 8, 128), (8, 4, 64)])
def test_many_keys_that_no_query_sees(sta, H, K, d, causal):
    """A sequence of keys without queries, more than five of its key blocks to an SM, beside one with both: its dK and
    dV are zeros, written to rows far apart, the other's are its own, and no wait runs out."""
    lens_q, lens_k = [300, 0], [300, 24000 * 8 // K]
    q, k, v, do = make(lens_q, lens_k, H, K, d, seed=41)
    cq, ck, scale = ref.cu_of(lens_q), ref.cu_of(lens_k), 0.1
    want = ref.packed(q, k[:300], v[:300], [300], [300], causal, scale, do)
    o, lse = sta.sta_packed_attention(q, k, v, cq, ck, causal=causal, softmax_scale=scale)
    for _ in range(3):
        out = torch.full((2, k.shape[0], 4 * K, d), math.nan, dtype=torch.bfloat16, device="cuda")
        dk, dv, dq = out[0, :, :K], out[1, :, K:2 * K], torch.empty_like(q)
        sta.sta_packed_backward(q, k, v, o, lse, do, dq, dk, dv, cq, ck, causal=causal, softmax_scale=scale)
        assert sta.sta_operator_status() == 0
        for name, t in (("dq", dq), ("dk", dk[:300]), ("dv", dv[:300])):
            ref.check(t, want, name)
        for t in (dk, dv):
            assert not bool(t[300:].any())


@pytest.mark.parametrize("lens_q,lens_k,H,K,d", [
    ([30, 5], [30, 5], 4, 2, 64), ([300, 100], [300, 100], 4, 2, 128), ([60] * 40, [60] * 40, 4, 2, 64),
    ([3500], [3500], 12, 12, 64), ([40, 70], [0, 0], 4, 2, 64), ([0, 0], [90, 30], 4, 2, 128), ([20], [500], 6, 2, 128)])
@pytest.mark.parametrize("first_q,first_k", [(3, 3), (50, 0), (0, 17)])
def test_rows_before_the_first_sequence_are_no_ones(sta, lens_q, lens_k, H, K, d, first_q, first_k):
    """A first bound above 0 is reported; the rows before it are zeros in new tensors and left alone in given ones,
    the sequences' own are those of the same bounds with one more sequence in front."""
    first_q, first_k = (first_q if sum(lens_q) else 0), (first_k if sum(lens_k) else 0)
    if not first_q and not first_k:
        first_q = first_k = 2
    q, k, v, do = make([first_q] + lens_q, [first_k] + lens_k, H, K, d, seed=51)
    cq, ck = ref.cu_of([first_q] + lens_q), ref.cu_of([first_k] + lens_k)

    def both(a, b, clear):
        o, dq, dk, dv = (torch.full_like(t, 7.0) for t in (q, q, k, v))
        lse = torch.full((H, q.shape[0]), 7.0, device="cuda")
        if clear:
            o, lse = sta.sta_packed_attention(q, k, v, a, b)
            return (o, lse) + sta.sta_packed_attention_backward(q, k, v, o, lse, do, a, b)
        sta.sta_packed_forward(q, k, v, o, lse, a, b)
        sta.sta_packed_backward(q, k, v, o, lse, do, dq, dk, dv, a, b)
        return o, lse, dq, dk, dv
    for clear in (True, False):
        want = both(cq, ck, clear)
        assert sta.sta_operator_status() == 0
        for t in [torch.full_like(x, 3.0) for x in want]:  # memory that is handed out again holds something
            del t
        got = both(cq[1:].contiguous(), ck[1:].contiguous(), clear)
        assert sta.sta_operator_status() == sta.STA_ERR_BOUNDS
        for name, a, b, n in zip(("o", "lse", "dq", "dk", "dv"), got, want, (first_q, first_q, first_q, first_k, first_k)):
            if name == "lse":
                a, b = a.t(), b.t()
            assert torch.equal(a[n:], b[n:]), name
            assert bool((a[:n] == (7.0 if not clear else -math.inf if name == "lse" else 0.0)).all()), name


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,K,d,n", [(24, 8, 128, 300), (10, 2, 64, 300), (100, 1, 64, 9), (2, 2, 128, 300)])
def test_keys_of_no_weight_have_no_gradient(sta, H, K, d, n, causal, what):
    """Keys whose scores are -inf (and then their values, zeros or not) leave dK and dV of their own rows zero, also where
    128 is no multiple of the query heads to a key head."""
    q, k, v, do = make([n], [n], H, K, d, seed=71)
    q[..., 0], k[..., 0] = 1.0, 0.0
    keys = [1, n // 2, n - 1]
    k[keys, :, 0] = -math.inf
    if what == "v":
        v[keys] = 0.0
    cu = ref.cu_of([n])
    o, lse = sta.sta_packed_attention(q, k, v, cu, causal=causal, softmax_scale=0.1)
    _, dk, dv = sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu, causal=causal, softmax_scale=0.1)
    assert bool(o.isfinite().all()) and not bool(dk[keys].any()) and not bool(dv[keys].any())
    if not causal:
        rest = [i for i in range(n) if i not in keys]
        want = ref.packed(q, k[rest], v[rest], [n], [n - 3], False, 0.1, do)
        for name, t in (("o", o), ("lse", lse), ("dk", dk[rest]), ("dv", dv[rest])):
            ref.check(t, want, name)


@pytest.mark.parametrize("hidden", [128, 300])
@pytest.mark.parametrize("n,m,H,K,d,causal", [
    (400, 400, 4, 2, 64, True), (400, 500, 4, 4, 128, False), (1100, 1100, 24, 8, 128, True), (3500, 3500, 12, 12, 64, True),
    (5, 9000, 2, 1, 64, True), (40, 9000, 4, 1, 128, False)])
def test_first_keys_whose_scores_are_minus_infinity(sta, n, m, H, K, d, causal, hidden):
    """The first chunks' scores are all -inf, the others far below zero: the results are those over the others alone,
    in both forward kernels and in split walks."""
    q, k, v, do = make([n], [m], H, K, d, seed=61)
    q[..., 0] = 1.0
    q[..., 1], k[..., 1] = 40.0, -100.0  # scores of -400, 2^-577
    k[..., 0] = 0.0
    k[:hidden, :, 0] = -math.inf
    scale, cq, ck = 0.1, ref.cu_of([n]), ref.cu_of([m])
    want = ref.packed(q, k[hidden:], v[hidden:], [n], [m - hidden], causal, scale, do)
    o, lse = sta.sta_packed_attention(q, k, v, cq, ck, causal=causal, softmax_scale=scale)
    ref.check(o, want, "o")
    ref.check(lse, want, "lse")
    _, dk, dv = sta.sta_packed_attention_backward(q, k, v, o, lse, do, cq, ck, causal=causal, softmax_scale=scale)
    ref.check(dk[hidden:], want, "dk")
    ref.check(dv[hidden:], want, "dv")
    assert not bool(dk[:hidden].any()) and not bool(dv[:hidden].any())
    assert sta.sta_operator_status() == 0
