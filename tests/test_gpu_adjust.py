"""GPU parity of the logit edits (dg_adjust_logits) against their fp64 form, and the edits in front of
the denoising step.  Bound of an edited logit: one rounding to the logits' type (half a step of the value)
and fp32 sums of the terms (2^-24 of their sizes each); everything else bit for bit."""
import math

import numpy as np
import pytest
import torch

import entropy_bounded_denoising_gb300 as dg
from entropy_bounded_denoising_gb300 import synth

import serving_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _params(n, inactive=()):
    p = {"temperature": np.ones(n, np.float32), "beta": np.full(n, 4.0, np.float32), "tau": np.full(n, 0.3, np.float32),
         "k": np.full(n, 2, np.int32), "max_steps": np.full(n, 8, np.int32), "min_accept": np.ones(n, np.int32),
         "step": np.zeros(n, np.int32), "request_id": np.arange(n, dtype=np.uint32),
         "flags": np.full(n, dg.DG_ACTIVE, np.uint32)}
    for c in inactive:
        p["flags"][c] = 0
    return dg.params_tensor(p, DEV)


def _ints(lists):
    cu = np.cumsum([0] + [len(x) for x in lists]).astype(np.int32)
    flat = np.array([t for x in lists for t in x], np.int64)
    return torch.from_numpy(flat).to(torch.int32).to(DEV), torch.from_numpy(cu).to(DEV)


def _case(n, L, V, dtype, *, hist=0, bias=0, masks=0, allowed=0.5, ld=None, ld_out=None, in_place=False, inactive=(),
          seed=0, x=None, status=0, lists=None, mask_rows=None, skip=()):
    rng = np.random.default_rng(seed + V + n)
    per = 8 if dtype == "bf16" else 4
    ld = -(-V // per) * per if ld is None else ld
    if x is None:
        x = torch.randn((n, L, ld), generator=torch.Generator().manual_seed(seed), dtype=torch.float32) * 4
    x = x.to(DT[dtype]).to(DEV)
    kw, h, b = {}, [[] for _ in range(n)], [[] for _ in range(n)]
    pen = np.stack([rng.uniform(0.5, 2.0, n), rng.uniform(-1, 1, n), rng.uniform(-1, 1, n)], 1).astype(np.float32)
    if hist:
        h = [rng.integers(-2, V + 2, max(0, hist - c)).tolist() for c in range(n)]
        h = [list(t) + t[:len(t) // 2] * 2 for t in h]            # repeats
    if bias:
        b = [[(int(t), float(np.float32(v))) for t, v in zip(rng.integers(-2, V + 2, bias), rng.normal(0, 8, bias))]
             for _ in range(n)]
        b = [t + t[:3] + t[:1] for t in b]
    if lists is not None:
        h, b = lists
    if hist or lists is not None:
        kw["history"], kw["cu_history"] = _ints(h)
        kw["penalties"] = torch.from_numpy(pen).to(DEV)
    if bias or lists is not None:
        kw["bias_tokens"], kw["cu_bias"] = _ints([[t for t, _ in c] for c in b])
        kw["bias_values"] = torch.tensor([v for c in b for _, v in c], dtype=torch.float32, device=DEV)
    words = np.zeros((max(1, masks), -(-V // 32) + 1), np.uint32)
    rows = np.full((n, L), -1, np.int32)
    if masks:
        bits = rng.random((masks, words.shape[1] * 32)) < allowed
        bits[0] = False                                           # a mask that leaves nothing
        if masks > 1:
            bits[1] = True                                        # and one that leaves everything
        words = np.packbits(bits, axis=1, bitorder="little").view(np.uint32).reshape(masks, -1)
        rows = rng.integers(-1, masks, (n, L)).astype(np.int32) if mask_rows is None else mask_rows
        kw["masks"] = torch.from_numpy(words.view(np.int32).copy()).to(DEV)
        kw["mask_index"] = torch.from_numpy(rows).to(DEV)
    x0 = x.clone()
    out = x if in_place else torch.full((n, L, ld if ld_out is None else ld_out), 9.0, dtype=x.dtype, device=DEV)
    out0 = out.clone()
    dg.dg_clear_device_status()
    dg.dg_adjust_logits(x, _params(n, inactive), None if in_place else out, V=V, **kw)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == status
    assert in_place or torch.equal(x.view(torch.uint8), x0.view(torch.uint8))
    assert torch.equal(out[..., V:], out0[..., V:])
    for c in range(n):
        if c in inactive or c in skip:
            assert torch.equal(out[c], out0[c]), c
            continue
        want, slack, touched = ref.adjusted(x0[c], V, h[c], pen[c], b[c], [m if m < masks else -1 for m in rows[c]], words)
        got = out[c, :, :V].cpu()
        same = x0[c, :, :V].cpu()
        it = torch.int16 if dtype == "bf16" else torch.int32
        assert torch.equal(got.view(it)[~touched], same.view(it)[~touched]), c
        g = got.double()
        # a value past the type's range rounds to infinity
        ok = (g == want) | (g.isnan() & want.isnan()) | (g.isinf() & (g == want.to(x.dtype).double())) | \
            ((g - want).abs() <= ref.HALF_STEP[x.dtype] * want.abs() + slack * (1 + 2.0 ** -7))
        assert ok[touched].all(), (c, g[touched & ~ok][:4], want[touched & ~ok][:4])
    return out


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,L,V", [(1, 1, 2), (1, 16, 1024), (3, 7, 4099), (2, 130, 2047), (5, 9, 33), (2, 3, 20001)])
def test_adjust(n, L, V, dtype, in_place):
    _case(n, L, V, dtype, hist=50, bias=20, masks=3, in_place=in_place, inactive=(1,) if n > 1 else ())
    _case(n, L, V, dtype, hist=5, in_place=in_place)
    _case(n, L, V, dtype, bias=9, in_place=in_place)
    for allowed in (0.0, 0.01, 0.99, 1.0):
        _case(n, L, V, dtype, masks=4, allowed=allowed, in_place=in_place)
    _case(n, L, V, dtype, in_place=in_place)                      # nothing to do: a copy, or nothing


def test_adjust_strides_and_long_lists():
    _case(2, 5, 1000, "bf16", hist=30, bias=5, masks=2, ld=1024, ld_out=1008)
    _case(2, 5, 1000, "fp32", hist=30, bias=5, masks=2, ld=1004, ld_out=2000)
    _case(2, 3, 5000, "bf16", hist=20000, bias=3000, masks=2)
    _case(70, 2, 300, "bf16", hist=100, bias=10, masks=5, inactive=tuple(range(0, 70, 3)))
    _case(1, 1024, 515, "fp32", hist=40, bias=10, masks=9)


def test_adjust_special_values():
    """Infinite and NaN logits go through the edits as fp32 says, a mask covers them all; biases of
    -inf exclude, the same token many times adds up in list order."""
    for dtype in ("bf16", "fp32"):
        x = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, 1.0, -1.0, torch.finfo(DT[dtype]).max,
                          torch.finfo(DT[dtype]).min, torch.finfo(DT[dtype]).tiny] * 2 + [0.5] * 4).repeat(1, 3, 1)
        hist = [list(range(10)) * 2]
        bias = [[(i, v) for i in (0, 1, 3, 5, 12) for v in (1.5, -0.25, 1e-3)] + [(6, -math.inf), (15, -math.inf)]]
        for in_place in (False, True):
            _case(1, 3, 24, dtype, x=x, lists=(hist, bias), in_place=in_place)
            _case(1, 3, 24, dtype, x=x, lists=(hist, bias), masks=3, in_place=in_place,
                  mask_rows=np.array([[0, 1, 2]], np.int32))
        # 1000 times the same token, whose sum depends on the order of the list
        vals = [float(np.float32(10.0 ** (i % 9 - 4) * (-1) ** i)) for i in range(1000)]
        got = _case(1, 3, 24, dtype, x=x, lists=([[]], [[(20, v) for v in vals]]))
        s = np.float32(0)
        for v in vals:
            s = np.float32(s + np.float32(v))
        want = torch.tensor(np.float32(0.5) + s).to(DT[dtype])
        assert (got[0, :, 20].cpu() == want).all()


def test_adjust_refused_canvases():
    bad = dg.DG_DEV_BAD_PARAM
    n, L, V = 3, 4, 100
    x = torch.randn((n, L, 104), device=DEV)
    hist = torch.arange(9, dtype=torch.int32, device=DEV)
    for cu, pen, who in (([0, 3, 2, 9], None, 1), ([0, 3, 6, 10], None, 2), ([-1, 3, 6, 9], None, 0),
                         ([0, 3, 6, 9], (1, 0.0), 1), ([0, 3, 6, 9], (1, math.nan), 1), ([0, 3, 6, 9], (2, -1.0), 2)):
        p = torch.ones((n, 3), device=DEV)
        if pen:
            p[pen[0], 0] = pen[1]
        out = torch.full_like(x, 9.0)
        dg.dg_clear_device_status()
        dg.dg_adjust_logits(x, _params(n), out, history=hist, cu_history=torch.tensor(cu, dtype=torch.int32, device=DEV),
                            penalties=p, V=V)
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == bad
        assert (out[who] == 9.0).all()
        if cu != [0, 3, 2, 9]:
            assert all((out[c, :, :V] != 9.0).all() for c in range(n) if c != who)
    # a mask row outside the table counts as none
    _case(2, 4, 64, "fp32", masks=2, mask_rows=np.array([[0, 1, 2, -1], [7, 1, 0, 2 ** 31 - 1]], np.int32), status=bad)
    dg.dg_clear_device_status()


def test_adjust_in_a_graph_and_on_a_stream():
    n, L, V = 2, 8, 5000
    x = torch.randn((n, L, V), device=DEV).to(torch.bfloat16)
    hist, cu = _ints([[5, 6, 5], [7]])
    pen = torch.tensor([[1.5, 0.5, 0.25]] * n, device=DEV)
    out = torch.empty_like(x)
    p = _params(n)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    dg.dg_adjust_logits(x, p, out, history=hist, cu_history=cu, penalties=pen, stream=st)
    torch.cuda.synchronize()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.dg_adjust_logits(x, p, out, history=hist, cu_history=cu, penalties=pen)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    hist[3] = 9                                                   # read again at each replay
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], first[0]) and not torch.equal(out[1], first[1])


def test_edits_in_front_of_the_step():
    """The run a served request makes: its pass appended to the cache, attention over the pages, logits
    from the LM head, its edits, the denoising step.  Excluded tokens are never drawn nor argmax, and
    the step's results are those on logits edited by the fp64 form's rules."""
    from helpers import StepBuffers, run_step
    n, L, V, Hq, Hkv, D = 2, 32, 4096, 4, 2, 64
    b = ref.Batch([(L, 100 + L, 0), (L, 60 + L, 0)], Hq, Hkv, D, 16, seed=3).fill_keys()
    qkv = torch.randn((n * L, (Hq + 2 * Hkv) * D), generator=torch.Generator().manual_seed(5)).to(ref.BF16).to(DEV)
    q, k, v = (qkv[:, a * D:e * D].unflatten(1, (e - a, D)) for a, e in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    w = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device=DEV) / (D // 2))
    o = torch.empty((n * L, Hq, D), dtype=ref.BF16, device=DEV)
    dg.dg_clear_device_status()
    dg.dg_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cu, b.kv_len, inv_freq=w, q=q, q_out=b.q)
    dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, L)
    ref.check_attention(b, o, None)
    W = synth.lm_head_weights_int(V, Hq * D, seed=4, device=DEV)
    params = _params(n)
    x = torch.empty((n, L, V), dtype=ref.BF16, device=DEV)
    dg.dg_lm_head_logits(o.view(n, L, Hq * D), W, params, x)
    rng = np.random.default_rng(1)
    keep = rng.random((3, V)) < 0.02
    keep[:, :4] = True
    masks = torch.from_numpy(np.packbits(keep, axis=1, bitorder="little").view(np.int32).copy()).to(DEV)
    index = torch.from_numpy(rng.integers(0, 3, (n, L)).astype(np.int32)).to(DEV)
    hist, cu = _ints([[1, 2, 3, 1], [0]])
    pen = torch.tensor([[1.2, 0.5, 0.25]] * n, device=DEV)
    y = torch.empty_like(x)
    dg.dg_adjust_logits(x, params, y, history=hist, cu_history=cu, penalties=pen, masks=masks, mask_index=index)
    s = StepBuffers.make(n, L, DEV)
    run_step(y, params, 77, s)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == 0
    allowed = keep[index.cpu().numpy()]
    am, acc, smp = s.argmax.cpu().numpy(), s.accept.cpu().numpy().astype(bool), s.sample.cpu().numpy()
    assert np.take_along_axis(allowed, am[..., None], 2).all()
    assert allowed[acc, smp[acc]].all() and acc.any()
    want = torch.stack([ref.adjusted(x[c], V, hist.tolist()[:4] if c == 0 else [0], pen[c].tolist(), [], index[c].tolist(),
                                     masks.cpu().numpy().view(np.uint32))[0] for c in range(n)])
    ok = torch.isfinite(want)
    assert torch.equal(torch.isfinite(y.cpu()), ok)
    assert ((y.cpu().double() - want)[ok].abs() <= 2.0 ** -8 * want[ok].abs() + 2.0 ** -16).all()
    p = torch.softmax(y.double(), -1)
    H = -(p * torch.where(p > 0, p, torch.ones_like(p)).log()).sum(-1)
    assert torch.allclose(s.entropy.double(), H, rtol=1e-5, atol=1e-9)


def test_the_run_in_one_graph():
    """A served pass captured once (append, attention, logits, edits) and replayed with other lengths and
    inputs gives what the calls give one by one."""
    n, L, V, Hq, Hkv, D = 3, 16, 2048, 4, 2, 64
    b = ref.Batch([(L, 90 + L, 0), (L, 40 + L, 1), (L, 300 + L, 0)], Hq, Hkv, D, 16, seed=3).fill_keys()
    w = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device=DEV) / (D // 2))
    qkv = torch.randn((n * L, (Hq + 2 * Hkv) * D), generator=torch.Generator().manual_seed(5)).to(ref.BF16).to(DEV)
    q, k, v = (qkv[:, a * D:e * D].unflatten(1, (e - a, D)) for a, e in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    W = synth.lm_head_weights_int(V, Hq * D, seed=4, device=DEV)
    params = _params(n)
    hist, cu = _ints([[1, 2, 3, 1], [0], [7] * 9])
    pen = torch.tensor([[1.2, 0.5, 0.25]] * n, device=DEV)
    qr, o = torch.empty((n * L, Hq, D), dtype=ref.BF16, device=DEV), torch.empty((n * L, Hq, D), dtype=ref.BF16, device=DEV)
    x = torch.empty((n, L, V), dtype=ref.BF16, device=DEV)

    def run():
        dg.dg_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cu, b.kv_len, inv_freq=w, q=q, q_out=qr)
        dg.dg_paged_attention(qr, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, L)
        dg.dg_lm_head_logits(o.view(n, L, Hq * D), W, params, x)
        dg.dg_adjust_logits(x, params, history=hist, cu_history=cu, penalties=pen)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for lens in ([90 + L, 40 + L, 300 + L], [L, 3 + L, 0], [1 + L, 0, 200 + L]):
        b.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        qkv.mul_(-1)
        for t in (qr, o, x):
            t.zero_()
        kc, vc = b.k_cache.clone(), b.v_cache.clone()
        run()
        torch.cuda.synchronize()
        want = [t.clone() for t in (qr, o, x, b.k_cache, b.v_cache)]
        b.k_cache.copy_(kc)
        b.v_cache.copy_(vc)
        for t in (qr, o, x):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for got, t in zip((qr, o, x, b.k_cache, b.v_cache), want):
            assert torch.equal(got.view(torch.int16), t.view(torch.int16))
        assert torch.isfinite(x).all()
    assert dg.dg_get_device_status() == 0
