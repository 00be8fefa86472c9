"""Refusals of the packed attention and the 8-bit cache calls, before any launch (no GPU), and their workspaces."""
import ctypes

import pytest

import sparse_attention_video_sta_b200 as sta
from sparse_attention_video_sta_b200._prompt import _Cache, _Packed, _Rows

INV, UNS, OK = sta.STA_ERR_INVALID_ARG, sta.STA_ERR_UNSUPPORTED, 0
P = 1 << 20  # a pointer that is never read


def packed(**kw):
    a = dict(batch=2, heads=8, kv_heads=2, head_dim=64, tokens_q=100, tokens_k=120, cu_q=P, cu_k=P, causal=1,
             clear_tail=0, softmax_scale=0.125)
    a.update(kw)
    return _Packed(*a.values())


def rows(data=P, token=512, head=64):
    return _Rows(data, token, head)


def cache(**kw):
    a = dict(blocks=4, block_tokens=16, kv_heads=2, head_dim=64, k_codes=P, v_codes=P, k_scales=P, v_scales=P)
    a.update(kw)
    return _Cache(*a.values())


BAD_PROBLEMS = [
    (dict(batch=-1), INV), (dict(heads=0), INV), (dict(kv_heads=0), INV), (dict(heads=7), INV), (dict(tokens_q=-1), INV),
    (dict(tokens_k=-5), INV), (dict(causal=2), INV), (dict(clear_tail=-1), INV), (dict(softmax_scale=0.0), INV),
    (dict(softmax_scale=-1.0), INV), (dict(softmax_scale=float("nan")), INV), (dict(softmax_scale=float("inf")), INV),
    (dict(head_dim=96), UNS), (dict(head_dim=0), UNS), (dict(heads=258, kv_heads=2), UNS), (dict(tokens_q=1 << 29), UNS),
    (dict(tokens_k=1 << 31), UNS), (dict(tokens_q=1 << 62), UNS),
]


@pytest.mark.parametrize("kw,status", BAD_PROBLEMS)
def test_problem_is_refused(kw, status):
    n = ctypes.c_int64(0)
    L = sta._lib
    for backward in (0, 1):
        assert L.sta_packed_workspace(packed(**kw), backward, ctypes.byref(n)) == status
    r = rows()
    assert L.sta_packed_forward(packed(**kw), r, r, r, r, P, P, 1 << 40, None) == status
    assert L.sta_packed_backward(packed(**kw), r, r, r, r, r, P, r, r, r, P, 1 << 40, None) == status


def test_packed_buffers_are_refused():
    L, p, n = sta._lib, packed(batch=40), ctypes.c_int64(0)  # (a forward of few sequences needs no workspace)
    assert L.sta_packed_workspace(p, 2, ctypes.byref(n)) == INV
    assert L.sta_packed_workspace(p, 0, None) == INV
    assert L.sta_packed_workspace(None, 0, ctypes.byref(n)) == INV
    sizes = []
    for backward in (0, 1):
        assert L.sta_packed_workspace(p, backward, ctypes.byref(n)) == OK and n.value > 0
        sizes.append(n.value)

    def fwd(q=rows(), k=rows(), v=rows(), o=rows(), lse=P, ws=P, size=sizes[0], p=p):
        return L.sta_packed_forward(p, q, k, v, o, lse, ws, size, None)

    def bwd(size=sizes[1], ws=P, lse=P, p=p, **kw):
        r = {m: rows() for m in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")}
        r.update(kw)
        return L.sta_packed_backward(p, r["q"], r["k"], r["v"], r["o"], r["dout"], lse, r["dq"], r["dk"], r["dv"], ws,
                                     size, None)
    for bad in (rows(data=None), rows(data=P + 8), rows(token=0), rows(token=-512), rows(token=516), rows(head=0),
                rows(head=4), rows(head=-64), None):
        for name in ("q", "k", "v", "o"):
            assert fwd(**{name: bad}) == INV, name
        for name in ("q", "k", "v", "o", "dout", "dq", "dk", "dv"):
            assert bwd(**{name: bad}) == INV, name
    for f, size in ((fwd, sizes[0]), (bwd, sizes[1])):
        assert f(lse=None) == INV and f(lse=P + 2) == INV
        assert f(ws=None) == INV and f(ws=P + 128) == INV and f(size=size - 1) == INV
        for kw in (dict(cu_q=None), dict(cu_k=None), dict(cu_q=P + 2), dict(cu_k=P + 1)):
            assert f(p=packed(batch=40, **kw)) == INV
    assert L.sta_packed_workspace(packed(), 0, ctypes.byref(n)) == OK and n.value == 0
    assert L.sta_packed_workspace(packed(), 1, ctypes.byref(n)) == OK and n.value > 0
    # nothing to do: pointers are not read
    none = rows(data=None)
    assert fwd(q=none, o=none, lse=None, p=packed(tokens_q=0)) == OK
    assert bwd(p=packed(tokens_q=0, tokens_k=0), lse=None, **{m: none for m in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")}) == OK


def test_cache_calls_are_refused():
    L = sta._lib
    n = ctypes.c_int64(0)
    bad = [(dict(blocks=0), INV), (dict(kv_heads=0), INV), (dict(k_codes=None), INV), (dict(v_codes=P + 8), INV),
           (dict(k_scales=None), INV), (dict(v_scales=P + 2), INV), (dict(block_tokens=8), UNS),
           (dict(block_tokens=48), UNS), (dict(head_dim=80), UNS)]
    r, q1 = rows(), packed(cu_q=None, tokens_q=2)
    assert L.sta_cache_workspace(cache(), q1, ctypes.byref(n)) == OK
    size = n.value

    def att(c=cache(), p=q1, lengths=P, tables=P, width=4, stride=4, q=r, o=r, lse=P, ws=P, size=size):
        return L.sta_cache_attention(c, p, lengths, tables, width, stride, q, o, lse, ws, size, None)
    for kw, status in bad:
        assert L.sta_cache_append(cache(**kw), r, r, 3, P, None) == status
        assert L.sta_cache_workspace(cache(**kw), q1, ctypes.byref(n)) == status
        assert att(c=cache(**kw)) == status
    c = cache()
    assert L.sta_cache_append(None, r, r, 3, P, None) == INV
    assert L.sta_cache_append(c, r, r, -1, P, None) == INV
    assert L.sta_cache_append(c, r, r, 3, None, None) == INV
    assert L.sta_cache_append(c, r, r, 3, P + 4, None) == INV
    assert L.sta_cache_append(c, rows(head=4), r, 3, P, None) == INV
    assert L.sta_cache_append(c, r, None, 3, P, None) == INV
    assert L.sta_cache_append(c, rows(data=None), rows(data=None), 0, None, None) == OK
    for kw, status in BAD_PROBLEMS:
        if "tokens_k" not in kw and "causal" not in kw:
            assert att(p=packed(**{"cu_q": P, **kw})) == status, kw
    assert att(p=packed(cu_q=None, tokens_q=3)) == INV  # one query for each of two sequences
    assert att(p=packed(kv_heads=4, cu_q=P)) == INV and att(p=packed(head_dim=128, cu_q=P)) == INV
    for kw in (dict(lengths=None), dict(tables=None), dict(tables=P + 2), dict(width=0), dict(stride=3), dict(q=None),
               dict(o=rows(token=4)), dict(lse=None), dict(ws=None), dict(ws=P + 16), dict(size=size - 1)):
        assert att(**kw) == INV, kw
    assert att(width=1 << 28, stride=1 << 28) == UNS
    assert att(p=packed(batch=0, tokens_q=0, cu_q=P)) == OK


def test_extend_is_refused():
    def ext(batch=2, bt=16, new=P, ln=P, lo=P, t=P, w=4, st=4, f=P, pool=8, c=P, co=P, s=P, ms=5, cu=P, sh=P):
        return sta._lib.sta_cache_extend(batch, bt, new, ln, lo, t, w, st, f, pool, c, co, s, ms, cu, sh, None)
    for kw in (dict(batch=-1), dict(bt=0), dict(w=0), dict(st=3), dict(pool=0), dict(ms=-1), dict(s=None), dict(s=P + 4),
               dict(new=None), dict(ln=None), dict(lo=None), dict(t=None), dict(f=None), dict(c=None), dict(co=None),
               dict(cu=None), dict(sh=None), dict(ln=P + 2)):
        assert ext(**kw) == INV, kw
    assert ext(batch=8193) == UNS and ext(bt=48) == UNS


def test_timeout_injection_arguments():
    f = sta._lib.sta_debug_inject_operator_timeout
    assert f(2, 50) == INV and f(-1, 50) == INV and f(1, 0) == INV and f(1, 10001) == INV and f(0, 50) == OK


def test_cache_attention_without_sequences():
    """Nothing to clear: no pointer is read.  Rows to clear: the outputs are checked, lengths and tables are not."""
    r, L = rows(), sta._lib
    att = lambda clear, q=r, o=r, lse=P, ws=P: L.sta_cache_attention(  # noqa: E731
        cache(), packed(batch=0, tokens_q=5, cu_q=P, clear_tail=clear), None, None, 4, 4, q, o, lse, ws, 1 << 40, None)
    assert att(0) == OK and att(0, q=None, o=None, lse=None, ws=None) == OK
    for kw in (dict(q=None), dict(o=rows(data=P + 8)), dict(lse=None), dict(lse=P + 2), dict(ws=None), dict(ws=P + 16)):
        assert att(1, **kw) == INV, kw


def run(code):
    import os
    import subprocess
    import sys
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                          cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


MISSING = {
    "not there": 'sys.modules["sparse_attention_video_sta_b200._sta_torch"] = None',
    "of another torch": """
import types
m = types.ModuleType("sparse_attention_video_sta_b200._sta_torch")
m.built_for, m.bind = "torch 1.0, cpython-30", None
sys.modules[m.__name__] = m""",
    "of an older package": """
import types
m = types.ModuleType("sparse_attention_video_sta_b200._sta_torch")
sys.modules[m.__name__] = m""",
}


@pytest.mark.parametrize("how", MISSING)
def test_without_the_compiled_binding_the_other_calls_work(how):
    """The package loads and plans; a call that needs _sta_torch.so says that it is missing and how to build it."""
    r = run(f"""
import sys
{MISSING[how]}
import torch
import sparse_attention_video_sta_b200 as sta
with sta.sta_plan_host((12, 16, 16), (6, 8, 8), 1, 2, [(6, 8, 8)] * 2) as plan:
    assert plan.query(0, 0) == [0]
assert sta._lib.sta_packed_workspace(None, 0, None) == sta.STA_ERR_INVALID_ARG
t = torch.zeros(1, 1, 64)
for call in (lambda: sta.sta_packed_attention(t, t, t, t), lambda: sta.sta_cache_append(t, t, t, t, t, t, t),
             lambda: sta.StaPackedAttention.apply(t, t, t, t)):
    try:
        call()
    except ImportError as e:
        assert "_build.py" in str(e) and "_sta_torch" in str(e), e
    else:
        raise SystemExit("no error")
print("fine")
""")
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-3000:]


def test_the_compiled_binding_is_built_again_for_another_torch_or_python(tmp_path, monkeypatch):
    from sparse_attention_video_sta_b200 import _build, _sta_torch
    key = _build.torch_key()
    assert _sta_torch.built_for == key
    monkeypatch.setattr(_build.os.path, "getmtime", lambda f: 1.0)  # sources and library of the same age
    monkeypatch.setattr(_build, "TORCH_STAMP", str(tmp_path / "stamp"))
    assert not _build._torch_up_to_date()
    (tmp_path / "stamp").write_text(key)
    assert _build._torch_up_to_date()
    monkeypatch.setattr(_build, "torch_key", lambda: "torch 99.0, cpython-399")
    assert not _build._torch_up_to_date()
    assert any("torch 99.0" in a for a in _build._torch_command("x.so"))
