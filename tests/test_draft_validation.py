"""Refusals of the calls for drafted tokens, on the host (nothing is launched), and worked values of the fp64
forms their GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import entropy_bounded_denoising_gb300 as dg
from test_serving_validation import BAD_CACHES, _kv

import draft_ref as dref


def test_append_norm_refusals():
    lib = dg.load()

    def call(k=16, ldk=128, v=16, ldv=128, q=16, ldq=256, qo=32, cu=16, n=1, total=4, Hq=2, Hkv=1, D=128, qn=16, kn=16,
             eps=1e-6, pos=16, w=16, rot=128, kv=None):
        c = _kv() if kv is None else kv
        return lib.dg_kv_append_norm(k, ldk, v, ldv, q, ldq, qo, cu, n, total, Hq, Hkv, D, qn, kn, eps, pos, w, rot, 0,
                                     ctypes.byref(c), None)

    for kw in (dict(k=None), dict(v=None), dict(cu=None), dict(qo=None), dict(n=-1), dict(n=65536), dict(total=-1),
               dict(Hq=0), dict(Hkv=0), dict(rot=24), dict(w=None), dict(ldk=120), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=math.inf), dict(eps=math.nan), dict(eps=1e-39), dict(q=None, qo=None)):
        assert call(**kw) == dg.DG_ERR_INVALID_ARG, kw
    assert call(D=96) == dg.DG_ERR_UNSUPPORTED
    for kw in (dict(k=24), dict(qn=18), dict(kn=17), dict(pos=18), dict(ldk=132)):
        assert call(**kw) == dg.DG_ERR_ALIGNMENT, kw
    for kw, rc in BAD_CACHES:
        assert call(kv=_kv(**kw)) == rc, kw
    assert call(n=0, k=None) == dg.DG_OK and call(total=0, k=None) == dg.DG_OK


def test_attention_refusals():
    lib = dg.load()
    need = dg.dg_tree_attention_workspace_bytes(1, 40, 2, 1, 128)
    assert 0 < need < 1 << 30
    assert dg.dg_tree_attention_workspace_bytes(0, 4, 2, 1, 128) == 0
    assert dg.dg_tree_attention_workspace_bytes(1, 4, 3, 2, 128) == 0
    assert dg.dg_tree_attention_workspace_bytes(1, 4, 2, 1, 96) == 0

    def tree(q=16, kv=None, o=16, lse=16, cu=16, mask=16, words=2, pos=16, n=1, mq=40, total=44, Hq=2, Hkv=1, D=128,
             window=5, sinks=0, scale=1.0, ws=256, size=need):
        c = _kv() if kv is None else kv
        return lib.dg_tree_attention(q, ctypes.byref(c), o, lse, cu, mask, words, pos, n, mq, total, Hq, Hkv, D, window,
                                     sinks, scale, ws, size, None)

    def sink(q=16, kv=None, o=16, lse=16, cu=16, n=1, mq=40, total=44, Hq=2, Hkv=1, D=128, window=5, sinks=0, scale=1.0,
             ws=256, size=need):
        c = _kv() if kv is None else kv
        return lib.dg_sink_attention(q, ctypes.byref(c), o, lse, cu, n, mq, total, Hq, Hkv, D, window, sinks, scale, ws,
                                     size, None)

    for call in (tree, sink):
        for kw in (dict(q=None), dict(o=None), dict(cu=None), dict(n=-1), dict(n=65536), dict(mq=0), dict(total=-1),
                   dict(total=1 << 31), dict(Hq=3, Hkv=2), dict(Hq=0), dict(Hkv=0), dict(Hq=65536), dict(window=-2),
                   dict(sinks=-1), dict(scale=math.inf), dict(scale=math.nan), dict(scale=3e38)):
            assert call(**kw) == dg.DG_ERR_INVALID_ARG, kw
        assert call(D=96) == dg.DG_ERR_UNSUPPORTED
        for kw in (dict(q=24), dict(o=24), dict(lse=18), dict(cu=18), dict(ws=264)):
            assert call(**kw) == dg.DG_ERR_ALIGNMENT, kw
        assert call(ws=None) == dg.DG_ERR_WORKSPACE and call(size=need - 1) == dg.DG_ERR_WORKSPACE
        for kw, rc in BAD_CACHES:
            assert call(kv=_kv(**kw)) == rc, kw
        assert call(n=0, q=None) == dg.DG_OK and call(total=0, q=None) == dg.DG_OK
    for kw in (dict(mask=None), dict(words=1), dict(pos=None), dict(mq=65537)):
        assert tree(**kw) == dg.DG_ERR_INVALID_ARG, kw
    assert tree(mask=18) == dg.DG_ERR_ALIGNMENT and tree(pos=18) == dg.DG_ERR_ALIGNMENT
    assert sink(window=-1) == dg.DG_ERR_INVALID_ARG
    # a workspace for the largest call serves the smaller ones
    sizes = [dg.dg_tree_attention_workspace_bytes(n, m, 16, 8, 128) for n in (1, 8, 64, 1000) for m in (1, 8, 64, 1000)]
    assert sizes[-1] == max(sizes)


def test_verify_refusals():
    lib = dg.load()

    def call(x=16, dtype=0, ld=64, tok=16, par=None, probs=None, ldq=0, cu=16, n=1, total=5, V=64, T=16, u=16, un=16, na=16,
             path=16, out=16):
        return lib.dg_verify_drafts(x, dtype, ld, tok, par, probs, ldq, cu, n, total, V, T, u, un, na, path, out, None)

    for kw in (dict(x=None), dict(tok=None), dict(cu=None), dict(T=None), dict(u=None), dict(un=None), dict(na=None),
               dict(path=None), dict(out=None), dict(dtype=7), dict(ld=56), dict(n=-1), dict(n=65536), dict(total=-1),
               dict(total=1 << 31), dict(V=1), dict(V=1 << 30, ld=1 << 30), dict(probs=16, ldq=60),
               dict(par=16, probs=16, ldq=64)):
        assert call(**kw) == dg.DG_ERR_INVALID_ARG, kw
    for kw in (dict(x=24), dict(ld=68), dict(dtype=1, ld=66), dict(probs=24, ldq=64), dict(probs=16, ldq=66), dict(tok=18),
               dict(par=18), dict(cu=18), dict(T=18), dict(u=18), dict(un=18), dict(na=18), dict(path=18), dict(out=18)):
        assert call(**kw) == dg.DG_ERR_ALIGNMENT, kw
    assert call(dtype=1, V=(1 << 29) + 8, ld=(1 << 29) + 8) == dg.DG_ERR_UNSUPPORTED
    assert call(n=0, x=None) == dg.DG_OK


def test_keep_refusals():
    lib = dg.load()

    def call(kv=None, layers=1, stride=0, cu=16, n=4, total=8, Hkv=1, D=128, path=16, na=4096, new=8192):
        c = _kv() if kv is None else kv
        return lib.dg_kv_keep(ctypes.byref(c), layers, stride, cu, n, total, Hkv, D, path, na, new, None)

    for kw in (dict(cu=None), dict(path=None), dict(na=None), dict(new=None), dict(n=-1), dict(n=65536), dict(layers=0),
               dict(layers=65536), dict(total=-1), dict(Hkv=0), dict(layers=2, stride=1 << 55), dict(new=16), dict(new=28),
               dict(new=4096), dict(new=4100, na=4096)):
        assert call(**kw) == dg.DG_ERR_INVALID_ARG, kw
    assert call(D=96) == dg.DG_ERR_UNSUPPORTED
    for kw in (dict(cu=18), dict(path=18), dict(na=4098), dict(new=8194), dict(layers=2, stride=12)):
        assert call(**kw) == dg.DG_ERR_ALIGNMENT, kw
    for kw, rc in BAD_CACHES:
        assert call(kv=_kv(**kw)) == rc, kw
    assert lib.dg_kv_keep(None, 1, 0, 16, 1, 8, 1, 128, 16, 4096, 8192, None) == dg.DG_ERR_INVALID_ARG
    assert call(n=0, cu=None) == dg.DG_OK


def test_python_checks():
    """The Python entry points' own checks of shape, type and layout (host tensors never reach the library)."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kc = z(4, 16, 2, 64)
    ok = dict(k=z(5, 2, 64), v=z(5, 2, 64), k_cache=kc, v_cache=kc, page_table=i(3, 4), cu_q=i(4), kv_len=i(3), q=z(5, 4, 64),
              q_out=z(5, 4, 64), q_norm=z(64, dt=torch.float32), k_norm=z(64, dt=torch.float32), positions=i(5))
    for kw, err in ((dict(q_norm=z(64)), TypeError), (dict(k_norm=z(32, dt=torch.float32)), ValueError),
                    (dict(positions=i(4)), ValueError), (dict(positions=z(5)), TypeError), (dict(q=None, q_out=None), ValueError),
                    (dict(eps="x"), TypeError), (dict(k_cache=z(2, 4, 16, 2, 64)), ValueError)):
        with pytest.raises(err):
            dg.dg_kv_append_norm(**{**ok, **kw})
    with pytest.raises(ValueError, match="device tensors"):
        dg.dg_kv_append_norm(**ok)

    ok = dict(q=z(5, 4, 64), k_cache=kc, v_cache=kc, o=z(5, 4, 64), page_table=i(3, 4), cu_q=i(4), kv_len=i(3), max_q_len=5)
    for call, more in ((dg.dg_tree_attention, dict(tree_mask=i(5, 1))), (dg.dg_sink_attention, dict(window=4, sinks=1))):
        for kw, err in ((dict(o=z(5, 4, 32)), ValueError), (dict(q=z(5, 4, 64, dt=torch.float16)), TypeError),
                        (dict(cu_q=i(3)), ValueError), (dict(lse=z(5, 4)), TypeError), (dict(max_q_len=1 << 40), ValueError),
                        (dict(scale="a"), TypeError), (dict(max_q_len=2.5), TypeError)):
            with pytest.raises(err):
                call(**{**ok, **more, **kw})
        with pytest.raises(ValueError, match="device tensors"):
            call(**ok, **more)
    for kw, err in ((dict(tree_mask=None), TypeError), (dict(tree_mask=i(4, 1)), ValueError), (dict(tree_mask=z(5, 1)), TypeError),
                    (dict(tree_mask=i(5, 1), positions=i(6)), ValueError), (dict(tree_mask=i(5, 2)[:, :1]), ValueError)):
        with pytest.raises(err):
            dg.dg_tree_attention(**ok, **kw)

    f = lambda *s: torch.zeros(s)  # noqa: E731
    ok = dict(logits=z(6, 64), tokens=i(6), cu_q=i(3), temperature=f(2), uniforms=f(6), next_uniforms=f(2), n_accept=i(2),
              path=i(6), out_tokens=i(6))
    for kw, err in ((dict(logits=z(6, 64, dt=torch.float16)), TypeError), (dict(logits=z(6, 8, 8)), ValueError),
                    (dict(logits=z(64, 6).T), ValueError), (dict(tokens=i(5)), ValueError), (dict(cu_q=i(2)), ValueError),
                    (dict(uniforms=f(5)), ValueError), (dict(next_uniforms=None), TypeError), (dict(path=f(6)), TypeError),
                    (dict(draft_probs=f(6, 60)), ValueError), (dict(draft_probs=f(5, 64)), ValueError),
                    (dict(draft_probs=z(6, 64)), TypeError), (dict(draft_probs=f(6, 64), parents=i(6)), ValueError),
                    (dict(V=65), ValueError)):
        with pytest.raises(err):
            dg.dg_verify_drafts(**{**ok, **kw})
    with pytest.raises(ValueError, match="device tensors"):
        dg.dg_verify_drafts(**ok)

    ok = dict(k_cache=kc, v_cache=kc, page_table=i(3, 4), cu_q=i(4), kv_len=i(3), path=i(9), n_accept=i(3), new_len=i(3))
    for kw, err in ((dict(path=None), TypeError), (dict(n_accept=i(2)), ValueError), (dict(new_len=f(3)), TypeError),
                    (dict(k_cache=z(2, 4, 16, 2, 64)), ValueError), (dict(k_cache=z(2, 2, 4, 16, 2, 64)), ValueError)):
        with pytest.raises(err):
            dg.dg_kv_keep(**{**ok, **kw})
    layered = z(2, 4, 16, 2, 64)
    with pytest.raises(ValueError, match="device tensors"):
        dg.dg_kv_keep(**{**ok, "k_cache": layered, "v_cache": layered})


def test_reference_verification():
    """Worked: p = (1/2, 1/4, 1/4); drafts 1, then 0."""
    x = torch.tensor([[math.log(2.0), 0.0, 0.0]] * 3, dtype=torch.float64)
    tok = torch.tensor([0, 1, 0])
    one = lambda u, un, **kw: dref.verify(x, tok, 1.0, torch.tensor(u), torch.tensor(un), **kw)[:2]  # noqa: E731
    assert one([0, 0.2, 0.4], 0.6) == ([0, 1, 2], [1, 0, 1])          # 0.2 < 1/4, 0.4 < 1/2; 0.6 falls into token 1
    assert one([0, 0.3, 0.0], 0.6) == ([0], [0])                      # without token 1: 2/3, 1/3; 0.6 is in the first
    assert one([0, 0.3, 0.0], 0.7) == ([0], [2])
    q = torch.tensor([[0.0] * 3, [0.1, 0.8, 0.1], [0.5, 0.25, 0.25]])
    assert one([0, 0.3, 0.9], 0.5, probs=q) == ([0, 1, 2], [1, 0, 1])  # 0.3 * 0.8 < 1/4; 0.9 * 0.5 < 1/2
    assert one([0, 0.35, 0.9], 0.72, probs=q) == ([0], [0])           # left (0.4, 0, 0.15): 0.72 * 0.55 = 0.396
    assert one([0, 0.35, 0.9], 0.74, probs=q) == ([0], [2])
    # a tree: both children of the root; the second is tried with what the first left, 3/4
    assert one([0, 0.3, 0.6], 0.1, parents=[-1, 0, 0]) == ([0, 2], [0, 0])   # 0.6 * 3/4 = 0.45 < 1/2
    assert one([0, 0.3, 0.7], 0.1, parents=[-1, 0, 0]) == ([0], [2])         # only token 2 is left
    assert dref.verify(x, tok, 0.0, torch.zeros(3), 0.0, parents=[-1, 0, 0])[:2] == ([0, 2], [0, 0])


def test_reference_visibility():
    ok = dref.visible(3, 6, anc=[{0}, {0, 1}, {0, 2}], positions=[3, 4, 4], window=2, sinks=1)
    assert ok.int().tolist() == [[1, 1, 1, 1, 0, 0], [1, 0, 1, 1, 1, 0], [1, 0, 1, 1, 0, 1]]
    assert dref.visible(2, 5, window=1, sinks=1).int().tolist() == [[1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
