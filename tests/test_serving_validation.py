"""Refusals of the paged cache, paged attention and logit-edit calls, on the host: through the C ABI
(nothing is launched) and through the Python entry points' own checks of shape, type and layout; and
the fp64 forms their GPU tests compare with, against the attention oracle and worked values."""
import ctypes

import numpy as np
import pytest
import torch

import entropy_bounded_denoising_gb300 as dg
from entropy_bounded_denoising_gb300 import _native, synth
import oracle

import serving_ref as ref


def _kv(**kw):
    f = dict(k=16, v=16, page_table=16, kv_len=16, n_pages=4, page_stride=16 * 128, slot_stride=128,
             head_stride=128, page_size=16, max_pages=4)
    f.update(kw)
    return _native._PagedKV(*(f[n] for n, _ in _native._PagedKV._fields_))


BAD_CACHES = [(dict(k=None), dg.DG_ERR_INVALID_ARG), (dict(v=None), dg.DG_ERR_INVALID_ARG),
              (dict(page_table=None), dg.DG_ERR_INVALID_ARG), (dict(kv_len=None), dg.DG_ERR_INVALID_ARG),
              (dict(n_pages=0), dg.DG_ERR_INVALID_ARG), (dict(n_pages=1 << 31), dg.DG_ERR_INVALID_ARG),
              (dict(max_pages=0), dg.DG_ERR_INVALID_ARG), (dict(page_size=4), dg.DG_ERR_UNSUPPORTED),
              (dict(page_size=48), dg.DG_ERR_UNSUPPORTED), (dict(page_size=1 << 17), dg.DG_ERR_UNSUPPORTED),
              (dict(slot_stride=120), dg.DG_ERR_INVALID_ARG), (dict(head_stride=0), dg.DG_ERR_INVALID_ARG),
              (dict(page_stride=1 << 39), dg.DG_ERR_INVALID_ARG), (dict(page_stride=-128), dg.DG_ERR_INVALID_ARG),
              (dict(n_pages=1 << 30, page_stride=1 << 38), dg.DG_ERR_INVALID_ARG),
              (dict(k=24), dg.DG_ERR_ALIGNMENT), (dict(v=24), dg.DG_ERR_ALIGNMENT),
              (dict(slot_stride=132), dg.DG_ERR_ALIGNMENT)]


def test_append_refusals():
    lib = dg.load()

    def call(k=16, ldk=128, v=16, ldv=128, q=16, ldq=256, qo=32, cu=16, n=1, total=4, Hq=2, Hkv=1, D=128, w=16,
             rot=128, kv=None):
        c = _kv() if kv is None else kv
        return lib.dg_kv_append(k, ldk, v, ldv, q, ldq, qo, cu, n, total, Hq, Hkv, D, w, rot, 0, ctypes.byref(c), None)

    for kw in (dict(k=None), dict(v=None), dict(cu=None), dict(qo=None), dict(q=None), dict(n=-1), dict(n=65536),
               dict(total=-1), dict(total=1 << 31), dict(Hq=0), dict(Hkv=0), dict(rot=24), dict(rot=144),
               dict(w=None), dict(ldk=120), dict(ldv=64), dict(ldq=128), dict(ldq=1 << 31), dict(qo=16, ldq=264)):
        assert call(**kw) == dg.DG_ERR_INVALID_ARG, kw
    assert call(D=96) == dg.DG_ERR_UNSUPPORTED
    for kw in (dict(k=24), dict(v=24), dict(q=24), dict(qo=24), dict(ldk=132), dict(ldv=132), dict(ldq=260)):
        assert call(**kw) == dg.DG_ERR_ALIGNMENT, kw
    for kw, rc in BAD_CACHES:
        assert call(kv=_kv(**kw)) == rc, kw
    assert lib.dg_kv_append(16, 128, 16, 128, None, 0, None, 16, 1, 4, 1, 1, 128, None, 0, 0, None, None) == dg.DG_ERR_INVALID_ARG
    assert call(n=0, k=None) == dg.DG_OK and call(total=0, k=None) == dg.DG_OK


def test_attention_refusals():
    lib = dg.load()
    need = dg.dg_paged_attention_workspace_bytes(1, 4, 2, 1, 128)
    assert need < 1 << 30

    def call(q=16, o=32, cu=16, causal=16, n=1, mq=4, total=4, Hq=2, Hkv=1, D=128, W=-1, scale=0.1, ws=256,
             wsb=need, kv=None):
        c = _kv() if kv is None else kv
        return lib.dg_paged_attention(q, ctypes.byref(c), o, None, cu, causal, n, mq, total, Hq, Hkv, D, W, scale, ws,
                                      wsb, None)

    for kw in (dict(q=None), dict(o=None), dict(cu=None), dict(causal=None), dict(n=-1), dict(n=65536), dict(mq=0),
               dict(total=-1), dict(total=1 << 31), dict(Hq=3, Hkv=2), dict(Hkv=0), dict(W=-2),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=float("-inf"))):
        assert call(**kw) == dg.DG_ERR_INVALID_ARG, kw
    for d in (0, 96, 512):
        assert call(D=d) == dg.DG_ERR_UNSUPPORTED
    for kw in (dict(q=24), dict(o=24)):
        assert call(**kw) == dg.DG_ERR_ALIGNMENT, kw
    for kw, rc in BAD_CACHES:
        assert call(kv=_kv(**kw)) == rc, kw
    assert call(n=0, q=None) == dg.DG_OK and call(total=0, q=None) == dg.DG_OK


def test_adjust_refusals():
    lib = dg.load()

    def call(x=16, dt=0, ld=64, out=32, ldo=64, n=1, L=4, V=64, p=16, h=16, cuh=16, nh=5, pen=16, bt=16, bv=16, cub=16,
             nb=5, m=16, ms=2, nm=1, mi=16):
        return lib.dg_adjust_logits(x, dt, ld, out, ldo, n, L, V, p, h, cuh, nh, pen, bt, bv, cub, nb, m, ms, nm, mi, None)

    for kw in (dict(x=None), dict(out=None), dict(p=None), dict(dt=2), dict(ld=56), dict(ldo=56), dict(n=-1),
               dict(n=65536), dict(L=0), dict(L=1025), dict(V=1), dict(cuh=None), dict(pen=None), dict(bv=None),
               dict(cub=None), dict(mi=None), dict(ms=1), dict(nm=0), dict(nh=-1), dict(nb=1 << 31),
               dict(out=16, ldo=128)):
        assert call(**kw) == dg.DG_ERR_INVALID_ARG, kw
    for kw in (dict(x=24), dict(out=24), dict(ld=68), dict(ldo=68)):
        assert call(**kw) == dg.DG_ERR_ALIGNMENT, kw
    assert call(dt=1, V=1 << 29, ld=1 << 29, ldo=1 << 29, ms=1 << 24) == dg.DG_ERR_UNSUPPORTED
    assert call(n=0, x=None) == dg.DG_OK


def test_python_checks_come_before_the_device():
    bf = torch.bfloat16
    k = torch.zeros((4, 2, 64), dtype=bf)
    c = torch.zeros((3, 8, 2, 64), dtype=bf)
    table, cu, kl = torch.zeros((1, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q, o = torch.zeros((4, 4, 64), dtype=bf), torch.zeros((4, 4, 64), dtype=bf)
    causal = torch.zeros(1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        dg.dg_kv_append(k, k, c, c, table, cu, kl)
    with pytest.raises(ValueError, match="q and q_out"):
        dg.dg_kv_append(k, k, c, c, table, cu, kl, q=q)
    with pytest.raises(TypeError, match="k_cache"):
        dg.dg_kv_append(k, k, c.float(), c.float(), table, cu, kl)
    with pytest.raises(ValueError, match="one layout"):
        dg.dg_kv_append(k, k, c, torch.zeros((3, 2, 8, 64), dtype=bf).transpose(1, 2), table, cu, kl)
    with pytest.raises(TypeError, match="page_table"):
        dg.dg_kv_append(k, k, c, c, table.long(), cu, kl)
    with pytest.raises(ValueError, match="page_table"):
        dg.dg_paged_attention(q, c, c, o, table[0], cu, kl, causal, 4)
    with pytest.raises(ValueError, match="page_table"):
        dg.dg_paged_attention(q, c, c, o, torch.zeros((1, 6), dtype=torch.int32)[:, ::2], cu, kl, causal, 4)
    x, p = torch.zeros((1, 4, 64)), torch.zeros(36, dtype=torch.uint8)
    with pytest.raises(ValueError, match="come together"):
        dg.dg_adjust_logits(x, p, history=cu)
    with pytest.raises(ValueError, match="come together"):
        dg.dg_adjust_logits(x, p, masks=table)
    with pytest.raises(TypeError, match="out must be"):
        dg.dg_adjust_logits(x, p, x.to(bf))
    with pytest.raises(ValueError, match="device tensor"):
        dg.dg_adjust_logits(x, p)


def test_python_refuses_what_is_not_a_tensor_or_does_not_fit():
    bf = torch.bfloat16
    k, c = torch.zeros((4, 2, 64), dtype=bf), torch.zeros((3, 8, 2, 64), dtype=bf)
    table, cu, kl = torch.zeros((1, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q, causal = torch.zeros((4, 4, 64), dtype=bf), torch.zeros(1, dtype=torch.uint8)
    good = dict(k=k, v=k, k_cache=c, v_cache=c, page_table=table, cu_q=cu, kv_len=kl)
    for name, bad, kind in (("k", None, TypeError), ("v", 3, TypeError), ("k_cache", [c], TypeError), ("v_cache", c[0], ValueError),
                            ("page_table", None, TypeError), ("kv_len", None, TypeError), ("cu_q", kl, ValueError),
                            ("k", k[0], ValueError), ("v", k[:, :1], ValueError), ("v", k.transpose(0, 1), ValueError),
                            ("v", k[:3], ValueError), ("k", torch.zeros((4, 4, 64), dtype=bf)[:, ::2], ValueError),
                            ("k_cache", c.to_sparse(), TypeError), ("kv_len", torch.zeros((1, 1), dtype=torch.int32), ValueError)):
        with pytest.raises(kind):
            dg.dg_kv_append(**{**good, name: bad})
    for kw in (dict(inv_freq=torch.zeros(8)), dict(inv_freq=3), dict(q=q, q_out=q.float()), dict(q=q.float(), q_out=q)):
        with pytest.raises(TypeError):
            dg.dg_kv_append(**good, **kw)
    for kw in (dict(q=q[:3], q_out=q[:3]), dict(q=q, q_out=q[:, :2]), dict(q=q, q_out=q.transpose(0, 1)),
               dict(inv_freq=torch.zeros((1, 8), dtype=torch.float64))):
        with pytest.raises(ValueError):
            dg.dg_kv_append(**good, **kw)
    good = dict(q=q, k_cache=c, v_cache=c, o=q, page_table=table, cu_q=cu, kv_len=kl, causal=causal, max_q_len=4)
    for name, bad, kind in (("q", None, TypeError), ("o", q[:3], ValueError), ("q", q.transpose(0, 1), ValueError),
                            ("causal", kl, TypeError), ("max_q_len", 1.5, TypeError), ("max_q_len", 1 << 31, ValueError),
                            ("lse", torch.zeros(4), ValueError), ("window", 1 << 40, ValueError), ("scale", "1", TypeError)):
        with pytest.raises(kind):
            dg.dg_paged_attention(**{**good, name: bad})
    x, p = torch.zeros((1, 4, 64)), torch.zeros(36, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f32 = torch.zeros
    for args, kw, kind in (((x.double(), p), {}, TypeError), ((x[0], p), {}, ValueError), ((x, p[:35]), {}, ValueError),
                           ((x, None), {}, TypeError), ((None, p), {}, TypeError), ((x, p), dict(V=1.5), TypeError),
                           ((x, p, x[:, :3]), {}, ValueError), ((x, p), dict(masks=i32(2), mask_index=i32(1, 4)), ValueError),
                           ((x, p), dict(masks=i32(1, 2), mask_index=i32(4)), ValueError),
                           ((x, p), dict(masks=i32(0, 2), mask_index=i32(1, 4)), ValueError),
                           ((x, p), dict(history=i32(3), cu_history=i32(2), penalties=f32(3)), ValueError),
                           ((x, p), dict(history=i32(3).long(), cu_history=i32(2), penalties=f32(1, 3)), TypeError),
                           ((x, p), dict(bias_tokens=i32(3), bias_values=f32(2), cu_bias=i32(2)), ValueError)):
        with pytest.raises(kind):
            dg.dg_adjust_logits(*args, **kw)


def test_paged_attention_form_matches_the_attention_oracle():
    """The fp64 form reads the pages as the oracle of dg_attention reads packed keys."""
    b = ref.Batch([(3, 20, True), (5, 13, False), (1, 9, True)], 4, 2, 64, 8, seed=1, device="cpu").fill_keys()
    kk = torch.cat([b.keys(s)[0] for s in range(3)])
    vv = torch.cat([b.keys(s)[1] for s in range(3)])
    cu_kv = np.array([0, 20, 33, 42], np.int32)
    for window in (-1, 0, 4):
        ro, rl = oracle.attention(synth.bf16_bits(b.q), synth.bf16_bits(kk), synth.bf16_bits(vv), b.cu.numpy(), cu_kv,
                                  b.causal.numpy(), window=window)
        for s, (a, _, causal) in enumerate(b.seqs):
            rows = slice(int(b.cu[s]), int(b.cu[s + 1]))
            o, lse, _, _ = ref.attention(b.q[rows], *b.keys(s), causal, window, 1 / 8)
            np.testing.assert_allclose(o.numpy(), ro[rows], rtol=1e-9, atol=1e-12)
            np.testing.assert_allclose(lse.numpy(), rl[rows], rtol=1e-9, atol=1e-12)


def test_rotation_and_edit_forms_on_worked_values():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0]]], dtype=torch.float64)
    w = torch.tensor([np.pi / 2, np.pi], dtype=torch.float64)
    y = ref.rotate(x, torch.tensor([1]), w, False)     # pairs (1, 3) a quarter, (2, 4) half a turn
    np.testing.assert_allclose(y[0, 0], [-3, -2, 1, -4, 5], atol=1e-12)
    y = ref.rotate(x, torch.tensor([3]), w, True)      # pairs (1, 2) three quarters, (3, 4) three halves
    np.testing.assert_allclose(y[0, 0], [2, -1, -3, -4, 5], atol=1e-12)
    words = np.array([[0b0111]], np.uint32)
    y, _, touched = ref.adjusted(torch.tensor([[2.0, -2.0, 1.0, 5.0]]), 4, [0, 1, 0, -1], (2.0, 0.5, 0.25),
                                 [(1, 3.0), (1, -1.0), (9, 5.0)], [0], words)
    assert y[0].tolist() == [2 / 2 - 2 * 0.5 - 0.25, -2 * 2 + 2 - 0.5 - 0.25, 1.0, -float("inf")]
    assert touched[0].tolist() == [True, True, False, True]
