"""The prompt side's compiled binding: what it refuses, the streams it takes, who owns new tensors."""
import math

import pytest
import torch

import prompt_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def sta():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    import sparse_attention_video_sta_b200 as s
    return s


def packed_args():
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    return dict(q=r(9, 4, 64), k=r(9, 2, 64), v=r(9, 2, 64), o=r(9, 4, 64), lse=torch.zeros(4, 9, device="cuda"),
                cu_q=ref.cu_of([5, 4]))


PACKED = [
    ("q", lambda t: t.cpu(), "CUDA"), ("q", lambda t: t.float(), "bf16"), ("q", lambda t: t[0], "tokens, heads, d"),
    ("k", lambda t: t.half(), "bf16"), ("k", lambda t: t.cpu(), "bf16"), ("v", lambda t: t[:, :, :32], "shape"),
    ("v", lambda t: t[:-1], "shape"), ("k", lambda t: torch.zeros(9, 2, 128, device="cuda", dtype=BF)[..., ::2], "contiguous"),
    ("k", lambda t: torch.zeros(9, 2, 68, device="cuda", dtype=BF)[..., :64], "multiples of 8"),
    ("k", lambda t: torch.zeros(9, 2, 72, device="cuda", dtype=BF)[..., 4:68], "aligned"),
    ("v", lambda t: t[:1].expand(9, -1, -1), "positive"), ("o", lambda t: t[:, :2], "shape"),
    ("lse", lambda t: t.double(), "fp32"), ("lse", lambda t: t.t().contiguous(), "shape"),
    ("cu_q", lambda t: t.long(), "Int"), ("cu_q", lambda t: t.cpu(), "cuda"), ("cu_q", lambda t: t[None], "sequences"),
    ("cu_q", lambda t: t[:0], "sequences"), ("cu_q", lambda t: t.repeat(2)[::2], "contiguous"),
    ("cu_k", lambda t: ref.cu_of([9]), "shape"),
    ("workspace", lambda t: torch.empty(1 << 20, device="cuda"), "uint8"),
    ("workspace", lambda t: torch.empty(1 << 20, dtype=torch.uint8), "uint8"),
]


@pytest.mark.parametrize("name,change,word", PACKED, ids=[f"{n}-{i}" for i, (n, _, _) in enumerate(PACKED)])
def test_packed_refusals(sta, name, change, word):
    a = packed_args()
    a[name] = change(a.get(name))
    with pytest.raises(ValueError, match=word):
        sta.sta_packed_forward(**a)
    if name != "o" and name != "lse" and name != "workspace":
        b = {n: a[n] for n in a if n not in ("o", "lse")}
        with pytest.raises(ValueError, match=word):
            sta.sta_packed_attention(**b)
    d = packed_args()
    d[name] = a[name]
    with pytest.raises(ValueError, match=word):
        sta.sta_packed_backward(d.pop("q"), d.pop("k"), d.pop("v"), d.pop("o"), d.pop("lse"), torch.zeros(9, 4, 64, device="cuda", dtype=BF),
                                torch.zeros(9, 4, 64, device="cuda", dtype=BF), torch.zeros(9, 2, 64, device="cuda", dtype=BF),
                                torch.zeros(9, 2, 64, device="cuda", dtype=BF), d.pop("cu_q"), **d)


def test_library_errors_come_through(sta):
    a = packed_args()
    a["k"], a["v"] = (torch.zeros(9, 3, 64, device="cuda", dtype=BF) for _ in range(2))  # 4 heads, 3 key heads
    with pytest.raises(sta.StaError, match="sta_packed_workspace"):
        sta.sta_packed_forward(**a)
    a = packed_args()
    with pytest.raises(ValueError, match="workspace"):
        sta.sta_packed_backward(a["q"], a["k"], a["v"], a["o"], a["lse"], a["o"], a["o"].clone(), a["k"].clone(),
                                a["v"].clone(), a["cu_q"], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sta.StaError):
        sta.sta_packed_forward(**packed_args(), softmax_scale=math.nan)
    with pytest.raises(TypeError):
        sta.sta_packed_forward(None, *list(packed_args().values())[1:])


def cache_args(K=2, d=64, bt=32, blocks=4):
    codes = [torch.zeros(blocks, K, bt, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.full((blocks, K), 2.0 ** -60, device="cuda") for _ in range(2)]
    return codes + scales


CACHE = [
    (0, lambda t: t.cpu(), "CUDA"), (0, lambda t: t[0], "CUDA"), (0, lambda t: t.view(torch.int8), "e4m3"),
    (1, lambda t: t[:-1], "shape"), (1, lambda t: t.transpose(1, 2), "shape"), (2, lambda t: t.double(), "fp32"),
    (3, lambda t: t[:, :1], "shape"), (3, lambda t: t.t().contiguous().t(), "contiguous"),
]


@pytest.mark.parametrize("which,change,word", CACHE, ids=[f"{n}-{i}" for i, (n, _, _) in enumerate(CACHE)])
def test_cache_refusals(sta, which, change, word):
    c = cache_args()
    c[which] = change(c[which])
    x = torch.zeros(3, 2, 64, device="cuda", dtype=BF)
    with pytest.raises(ValueError, match=word):
        sta.sta_cache_append(x, x, torch.arange(3, device="cuda"), *c)
    with pytest.raises(ValueError, match=word):
        sta.sta_cache_attention(x, *c, torch.zeros(3, 1, dtype=torch.int32, device="cuda"),
                                torch.ones(3, dtype=torch.int32, device="cuda"))


def test_cache_argument_refusals(sta):
    c = cache_args()
    x = torch.zeros(3, 2, 64, device="cuda", dtype=BF)
    t, n = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    slots = torch.arange(3, device="cuda")
    for k, s in ((x, slots.int()), (x[:2], slots), (x, slots.cpu()), (x.float(), slots), (x, slots[None])):
        with pytest.raises(ValueError):
            sta.sta_cache_append(k, x, s, *c)
    for q, tt, nn, kw in ((x[:2], t, n, {}), (x, t.long(), n, {}), (x, t[:2], n, {}), (x, t[:, :0], n, {}), (x, t[:, 0], n, {}),
                          (x, t.t().contiguous().t(), n, {}), (x, t, n.long(), {}), (x, t, n[None], {}),
                          (x, t, n, dict(cu_q=n)), (x, t, n, dict(o=x.float())), (x, t, n, dict(lse=n.float())),
                          (x, t[:1].expand(3, 2), n, {}), (x.expand(3, 2, 64)[:, :, ::2], t, n, {})):
        with pytest.raises((ValueError, sta.StaError)):
            sta.sta_cache_attention(q, *c, tt, nn, **kw)
    free, count = torch.arange(4, dtype=torch.int32, device="cuda"), torch.tensor([4], dtype=torch.int32, device="cuda")
    for kw in (dict(new_tokens=n[:2]), dict(lengths=n.cpu()), dict(block_tables=t.long()), dict(free_blocks=free.long()),
               dict(free_count=free), dict(block_tokens=33), dict(block_tokens=-32), dict(max_slots=-1)):
        a = dict(new_tokens=n, lengths=n, block_tables=t, free_blocks=free, free_count=count, block_tokens=32, max_slots=3)
        a.update(kw)
        with pytest.raises((ValueError, sta.StaError)):
            sta.sta_cache_extend(**a)


def test_streams(sta):
    """A stream object, its raw handle and the current stream give the same; memory that a call on a side stream
    used is not handed out before that stream is done with it."""
    a = packed_args()
    args = (a["q"], a["k"], a["v"], a["cu_q"])
    want = sta.sta_packed_attention(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        got = sta.sta_packed_attention(*args, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    with torch.cuda.stream(side):
        got = sta.sta_packed_attention(*args)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # outputs dropped while the side stream is still busy: their memory must not be given to the current stream
    big = torch.zeros(1 << 27, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big.add_(1.0)
    o, lse = sta.sta_packed_attention(*args, stream=side)
    p = o.data_ptr()
    del o
    assert all(torch.empty_like(a["q"]).data_ptr() != p for _ in range(3)) or side.query()
    torch.cuda.synchronize()


def test_no_grad_history_and_contiguous_outputs(sta):
    a = packed_args()
    q = a["q"].transpose(0, 1).contiguous().transpose(0, 1).requires_grad_()
    o, lse = sta.sta_packed_attention(q, a["k"], a["v"], a["cu_q"])
    assert o.is_contiguous() and lse.is_contiguous() and not o.requires_grad and o.grad_fn is None
    c = cache_args()
    step = sta.sta_cache_extend(torch.ones(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
                                torch.full((2, 1), -1, dtype=torch.int32, device="cuda"),
                                torch.arange(4, dtype=torch.int32, device="cuda"),
                                torch.tensor([4], dtype=torch.int32, device="cuda"), 32, 2)
    assert isinstance(step, sta.CacheStep) and step.slots.dtype is torch.int64 and int(step.short) == 0
    x = torch.zeros(2, 2, 64, device="cuda", dtype=BF)
    sta.sta_cache_append(x, x, step.slots, *c)
    for cu in (None, torch.zeros(1, dtype=torch.int32, device="cuda")):  # no queries, no sequences
        o, lse = sta.sta_cache_attention(x[:0], *c, torch.zeros(0, 1, dtype=torch.int32, device="cuda"),
                                         torch.zeros(0, dtype=torch.int32, device="cuda"), cu)
        assert o.shape == (0, 2, 64) and lse.shape == (2, 0)


def test_captured_between_other_work_and_over_two_streams(sta):
    """Kernels that start while the one before ends, in a graph: after another library's kernels and copies, after
    events, and on two streams that meet again; replayed with new inputs, against eager calls."""
    a = packed_args()
    c = cache_args(blocks=8)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    new, lengths, free, count = i32([5, 4]), i32([0, 0]), torch.arange(8, dtype=torch.int32, device="cuda"), i32([8])
    src = torch.randn(9, 4, 64, device="cuda")
    q, k = torch.empty(9, 4, 64, device="cuda", dtype=BF), torch.empty(9, 2, 64, device="cuda", dtype=BF)

    def step(side):
        q.copy_(src)
        k.copy_(src[:, :2] * 0.5)
        o, lse = sta.sta_packed_attention(q, k, k, a["cu_q"])
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            table = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
            f = free.clone()
            s = sta.sta_cache_extend(new, lengths, table, f, count, 32, 9)
            sta.sta_cache_append(k, k, s.slots, *c)
        grads = sta.sta_packed_attention_backward(q, k, k, o, lse, o * 2, a["cu_q"])
        here.wait_stream(side)
        got = sta.sta_cache_attention(q, *c, table, s.lengths, a["cu_q"])
        return (o, lse, *grads, *got, got[0] + 1)
    side = torch.cuda.Stream()
    want = []
    inputs = [torch.randn(9, 4, 64, device="cuda") for _ in range(3)]
    for x in inputs:
        src.copy_(x)
        want.append([t.clone() for t in step(side)])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(side)
    for x, w in list(zip(inputs, want)) * 3:
        src.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, r) for p, r in zip(out, w))
    assert sta.sta_operator_status() == 0
    del g


def calls_with_new_memory(sta):
    """Each call that allocates outputs or scratch, as f(stream) -> tensors."""
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    lens = [100, 37] * 20  # more than the forward plans without scratch
    q, k, v, do, cu = r(sum(lens), 4, 64), r(sum(lens), 2, 64), r(sum(lens), 2, 64), r(sum(lens), 4, 64), ref.cu_of(lens)
    o, lse = sta.sta_packed_attention(q, k, v, cu)
    o2, lse2, dq, dk, dv = (torch.empty_like(t) for t in (o, lse, q, k, v))
    c = cache_args(blocks=200)
    c[0].view(torch.uint8).copy_((torch.rand(c[0].shape, generator=g, device="cuda") * 100).byte())
    c[1].copy_(c[0])
    c[2].fill_(0.01), c[3].fill_(0.01)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = torch.arange(200, dtype=torch.int32, device="cuda").view(2, 100)
    n, free, count = i32([3000, 777]), torch.arange(90, dtype=torch.int32, device="cuda"), i32([90])
    new, held, wide = i32([5] * 40), i32([0] * 40), torch.zeros(40, 2, dtype=torch.int32, device="cuda")
    stock = [(wide.clone(), free.clone()) for _ in range(9)]  # (a call changes them)

    def extend(stream):
        t, f = stock.pop()
        return tuple(sta.sta_cache_extend(new, held, t, f, count, 32, 300, stream=stream))
    return [
        lambda s: sta.sta_packed_attention(q, k, v, cu, stream=s),
        lambda s: sta.sta_packed_forward(q, k, v, o2, lse2, cu, stream=s),
        lambda s: sta.sta_packed_attention_backward(q, k, v, o, lse, do, cu, stream=s),
        lambda s: sta.sta_packed_backward(q, k, v, o, lse, do, dq, dk, dv, cu, stream=s),
        lambda s: sta.sta_cache_attention(q[:2], *c, table, n, stream=s),
        extend,
    ]


@pytest.mark.parametrize("which", range(6))
def test_new_memory_of_a_call_on_another_stream(sta, which):
    """Blocks that the current stream has given back while work on them is queued there are not what a call on
    another stream computes in; and its new tensors, dropped on the current stream, outlast what that has queued."""
    call = calls_with_new_memory(sta)[which]
    side, raw = torch.cuda.Stream(), torch.cuda.current_stream()
    want = [t.clone() for t in call(None)]
    call(side)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        spots = [torch.empty(n, dtype=torch.uint8, device="cuda")
                 for n in [t.numel() * t.element_size() for t in want] + [1 << i for i in range(9, 25)]]
        used = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in spots]
        torch.cuda._sleep(400_000_000)
        for t in spots:
            t.fill_(0x7f)
        del spots, t
        got = call(stream)
        side.synchronize()
        assert not raw.query()
        if which in (0, 2, 4, 5):
            for t in got:
                a = t.data_ptr()
                assert not any(a < hi and lo < a + t.numel() * t.element_size() for lo, hi in used)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    if which in (0, 2, 4, 5):
        torch.cuda._sleep(400_000_000)
        kept, p = got[0].clone(), got[0].data_ptr()
        del got, t
        with torch.cuda.stream(side):
            assert all(torch.empty_like(want[0]).data_ptr() != p for _ in range(3)) or raw.query()
            torch.empty_like(want[0]).fill_(7.0)
        torch.cuda.synchronize()
        assert torch.equal(kept, want[0])


def test_the_default_stream_from_another_one(sta):
    """stream=0 while another stream is the current one, and the current stream is what it was afterwards."""
    a = packed_args()
    args = (a["q"], a["k"], a["v"], a["cu_q"])
    want = sta.sta_packed_attention(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = sta.sta_packed_attention(*args, stream=0)
        assert torch.cuda.current_stream() == side
        with pytest.raises(ValueError):
            sta.sta_packed_attention(a["q"], a["k"][:-1], a["v"], a["cu_q"], stream=0)
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_captured_calls_on_a_stream_that_joined_the_capture(sta):
    """A call with `stream=` inside a capture, on a stream forked from the captured one: its memory is the graph's,
    and replays beside eager work on the same streams give the eager results."""
    calls = calls_with_new_memory(sta)
    want = [[t.clone() for t in calls[i](None)] for i in (0, 2, 4)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = [calls[i](side) for i in (0, 2, 4)]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        g.replay()
        other = [calls[i](side) for i in (0, 2, 4)]
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, other):
            assert all(torch.equal(x, y) and torch.equal(z, y) for x, y, z in zip(a, b, c))
    assert sta.sta_operator_status() == 0
    del g


def test_a_timeout_and_a_cut_bound_are_both_reported(sta):
    """Both are pending, of one call or of two: the timeout first, whose outputs are lost, then the bound."""
    a = packed_args()
    bad = torch.tensor([0, 7, 4, 9], dtype=torch.int32, device="cuda")
    a["cu_q"] = bad
    assert sta.sta_operator_status() == 0
    for one_call in (True, False):
        sta.sta_debug_inject_operator_timeout(1, 20)
        try:
            sta.sta_packed_attention(a["q"], a["k"], a["v"], bad if one_call else ref.cu_of([5, 4]))
            torch.cuda.synchronize()
        finally:
            sta.sta_debug_inject_operator_timeout(0)
        if not one_call:
            sta.sta_packed_attention(a["q"], a["k"], a["v"], bad)
        assert sta.sta_operator_status() == sta.STA_ERR_TIMEOUT
        assert sta.sta_operator_status(stream=torch.cuda.Stream()) == sta.STA_ERR_BOUNDS
        assert sta.sta_operator_status() == 0
    # each alone, asked from several threads at once: said once
    from concurrent.futures import ThreadPoolExecutor
    for _ in range(20):
        sta.sta_packed_attention(a["q"], a["k"], a["v"], bad)
        torch.cuda.synchronize()
        with ThreadPoolExecutor(4) as pool:
            got = list(pool.map(lambda i: sta.sta_operator_status(device=0, stream=torch.cuda.Stream(device=0)), range(4)))
        assert sorted(got) == [0, 0, 0, sta.STA_ERR_BOUNDS]
