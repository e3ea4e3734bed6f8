"""Host tests of the serving calls (dg_kv_append, dg_paged_attention, dg_adjust_logits) at the edge of what
include/dg.h allows; nothing is launched."""
import ctypes

import pytest
import torch

import entropy_bounded_denoising_gb300 as dg
from entropy_bounded_denoising_gb300 import _native


def _kv(**kw):
    f = dict(k=16, v=16, page_table=16, kv_len=16, n_pages=4, page_stride=16 * 128, slot_stride=128,
             head_stride=128, page_size=16, max_pages=4)
    f.update(kw)
    return _native._PagedKV(*(f[n] for n, _ in _native._PagedKV._fields_))


def _attention(q=16, o=32, lse=None, cu=16, causal=16, n=1, mq=4, total=4, Hq=2, Hkv=1, D=128, W=-1, scale=0.1, ws=256,
               wsb=None, kv=None):
    need = dg.dg_paged_attention_workspace_bytes(n, mq, Hq, Hkv, D)
    c = _kv() if kv is None else kv
    return dg.load().dg_paged_attention(q, ctypes.byref(c), o, lse, cu, causal, n, mq, total, Hq, Hkv, D, W, scale, ws,
                                        need if wsb is None else wsb, None)


def test_scales_whose_log2_form_is_infinite_are_refused():
    for scale in (3e38, -3e38, 1.8e38, float("nan"), float("inf")):
        assert _attention(scale=scale) == dg.DG_ERR_INVALID_ARG
    for scale in (2.0 ** 127, -2.0 ** 127, 0.0):   # past this check: the workspace's is next
        assert _attention(scale=scale, ws=None) == dg.DG_ERR_WORKSPACE
