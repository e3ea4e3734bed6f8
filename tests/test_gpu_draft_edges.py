"""GPU tests of the calls for drafted tokens at their edges."""
import math

import pytest
import torch

import draft_ref as dref
import serving_ref as ref
from test_gpu_draft import Drafts, _append, _run_attention, _tree_batch

pytestmark = pytest.mark.gpu

import entropy_bounded_denoising_gb300 as dg  # noqa: E402

DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ NaN in sight
def _attend_only(b, mask, pos, window, sinks):
    """o and lse of a batch, without a comparison."""
    o = torch.full((b.total, b.Hq, b.D), 5.0, dtype=ref.BF16, device=DEV)
    lse = torch.full((b.total, b.Hq), 5.0, device=DEV)
    max_q = max(s[0] for s in b.seqs)
    dg.dg_clear_device_status()
    if mask is not None:
        dg.dg_tree_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, mask, max_q, lse=lse, window=window,
                             sinks=sinks, positions=pos if window >= 0 else None)
    else:
        dg.dg_sink_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, max_q, lse=lse, window=window, sinks=sinks)
    assert dg.dg_get_device_status() == 0
    return o, lse


# (nodes, keys) of the sequences: few rows a key head and many; one request over a long context, whose items many CTAs
# share; several whose items are cut between the first tokens and the window; items that one CTA has whole
NAN_CASES = [("few", [(4, 900), (1, 70), (3, 3)]), ("long", [(64, 9000)]), ("cut", [(33, 300)] * 5),
             ("whole", [(64, 64), (40, 41)] * 40)]


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 128), (8, 4, 64), (6, 2, 256)])
@pytest.mark.parametrize("name,seqs", NAN_CASES, ids=[c[0] for c in NAN_CASES])
def test_nan_that_a_row_sees(name, seqs, Hq, Hkv, D, tree):
    """A NaN query, or a NaN key that a row sees, makes that row's o and lse NaN, wherever its item is cut; every other
    row is right."""
    window, sinks = (40, 1) if name == "cut" or not tree else (-1, 0)
    b, oks, mask, pos = _tree_batch(seqs, Hq, Hkv, D, 16, 17, window, sinks)
    if not tree:
        mask, oks = None, [dref.visible(a, m, window=window, sinks=sinks) for a, m in seqs]
    o0, l0 = _run_attention(b, oks, mask=mask, positions=pos if tree and window >= 0 else None, window=window, sinks=sinks)
    cu, group, s = b.cu.tolist(), Hq // Hkv, len(seqs) // 2
    a, m = seqs[s]

    def attend(rows_heads):   # [total, Hq]: the rows that have to be NaN; the rest of the outputs
        o, lse = _attend_only(b, mask, pos, window, sinks)
        assert torch.isnan(o[rows_heads]).all() and torch.isnan(lse[rows_heads]).all()
        o[rows_heads], lse[rows_heads] = o0[rows_heads], l0[rows_heads]
        return o, lse

    # a query: NaN as a whole, and in one dimension
    for row, head, dims in ((cu[s], Hq - 1, slice(0, D)), (cu[s + 1] - 1, 0, slice(D - 1, D))):
        bad = torch.zeros((b.total, Hq), dtype=torch.bool, device=DEV)
        bad[row, head] = True
        old = b.q[row, head].clone()
        b.q[row, head, dims] = math.nan
        o, lse = attend(bad)
        b.q[row, head] = old
        dref.check_attention(b, o, lse, oks)
    # a key of one key head: the first of all (with a window the first token that stays), the context's last, a node
    for j in sorted({0, max(0, m - a - 1), m - 1}):
        at = b.slots(s, [j])
        old = b.k_cache[at[0], at[1], Hkv - 1].clone()
        b.k_cache[at[0], at[1], Hkv - 1] = math.nan
        bad = torch.zeros((b.total, Hq), dtype=torch.bool, device=DEV)
        bad[cu[s]:cu[s + 1], (Hkv - 1) * group:] = oks[s][:, j].to(DEV)[:, None]
        assert bad.any()
        o, lse = attend(bad)
        b.k_cache[at[0], at[1], Hkv - 1] = old
        dref.check_attention(b, o, lse, oks)


# ------------------------------------------------------------------ rounded weights
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 128), (8, 4, 64), (6, 2, 256)])
@pytest.mark.parametrize("name,seqs", NAN_CASES, ids=[c[0] for c in NAN_CASES])
def test_values_that_are_alike_stay_what_they_are(name, seqs, Hq, Hkv, D, tree):
    """Where all values of a dimension are one bf16 number, the output is that number: the rounded weights are divided by
    their own sum.  Over 9000 keys an output is added up in 563 steps of 16 and its sum in fewer, each within 2^-22; with
    the joins and the division less than 2^-12, and half a bf16 step is at least 2^-10, so the last rounding gives the
    number back."""
    window, sinks = (40, 1) if name == "cut" or not tree else (-1, 0)
    b, oks, mask, pos = _tree_batch(seqs, Hq, Hkv, D, 16, 23, window, sinks, q_scale=3.0)
    value = (torch.arange(D, device=DEV) * 0.037 + 1.01).to(ref.BF16)
    b.v_cache[:] = value
    o, _ = _attend_only(b, mask if tree else None, pos, window, sinks)
    assert torch.equal(o, value.expand_as(o)), float((o.double() / value.double() - 1).abs().max())


# ------------------------------------------------------------------ verification
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [50257, 1001, 1000])
def test_verify_columns_of_a_padded_buffer(V, dtype):
    """The first V columns of padded logits and draft rows, for one row as for two, the buffer's last among them."""
    pad = -(-V // 8) * 8
    for sizes in ([1], [2], [1, 1]):
        for at in (0, 3):
            d = Drafts(sizes, V, V + at, T=0.8, dtype=dtype, probs=True)
            want = Drafts(sizes, V, V + at, T=0.8, dtype=dtype, probs=True).run()
            want.check()
            # (columns of other requests before them, now and then)
            buf = torch.full((3 + d.total, pad + at // 3 * 8), math.nan, dtype=dtype, device=DEV)[:, at // 3 * 8:]
            probs = torch.full((3 + d.total, pad + at // 3 * 8), 0.5, device=DEV)[:, at // 3 * 8:]
            rows = slice(at, at + d.total)
            buf[rows, :V], probs[rows, :V] = d.x[:, :V].to(DEV), d.probs[:, :V].to(DEV)
            count, path, out = torch.zeros(len(sizes), **I32), torch.zeros(d.total, **I32), torch.zeros(d.total, **I32)
            dg.dg_verify_drafts(buf[rows, :V], d.tokens.to(DEV), d.cu, d.T.to(DEV), d.u.to(DEV), d.un.to(DEV), count, path, out,
                                draft_probs=probs[rows, :V])
            assert dg.dg_get_device_status() == 0
            assert torch.equal(count, want.n_accept) and torch.equal(path, want.path) and torch.equal(out, want.out)


def test_verify_one_row_without_a_buffer():
    """A row of its own: its columns have to be whole pieces of 16 bytes, whatever stride it names."""
    for V, ok in ((1000, True), (1001, False)):
        row = torch.randn((1, V), device=DEV, dtype=torch.bfloat16)
        for x in (row, row.as_strided((1, V), (V + 7 - (V + 7) % 8 + 8, 1))):   # (a stride with nothing behind it)
            args = (x, torch.zeros(1, **I32), torch.tensor([0, 1], **I32), torch.ones(1, device=DEV), torch.zeros(1, device=DEV),
                    torch.zeros(1, device=DEV), torch.zeros(1, **I32), torch.zeros(1, **I32), torch.zeros(1, **I32))
            if ok:
                dg.dg_verify_drafts(*args)
                assert args[6].item() == 0
            else:
                with pytest.raises(dg.DGError):
                    dg.dg_verify_drafts(*args)
    dg.dg_clear_device_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V", [(3, 700), (40, 700), (200, 700), (500, 700), (700, 700),
                                 (3, 20000), (40, 20000), (100, 20000), (200, 20000), (500, 20000)])
def test_verify_clusters_that_end_apart(n, V, dtype):
    """Sequences of no nodes, refused ones, ones that end at the root and long walks side by side, in clusters of every size,
    again and again on one stream: each as by itself, and no wait runs out."""
    sizes = [(0, 1, 40, 3, 12)[i % 5] for i in range(n)]
    d = Drafts(sizes, V, n, T=0.5, dtype=dtype, near=1.0)
    d.u *= 0.05
    refused = [s for s in range(n) if s % 7 == 3 and sizes[s]]
    for s in refused:
        d.T[s] = -1.0
    d.run()
    d.check(status=dg.DG_DEV_BAD_PARAM if refused else 0, skip=refused)
    n_acc = d.n_accept.tolist()
    assert all(n_acc[s] == -1 for s in refused)
    assert n < 40 or max(n_acc) > 5   # (of three sequences one alone has drafts)
    x, tok, cu, T, u, un, _, _ = d.dev
    want = d.n_accept.clone(), d.path.clone(), d.out.clone()
    for _ in range(20):
        got = [torch.full_like(t, -9) for t in want]
        dg.dg_verify_drafts(x, tok, cu, T, u, un, *got, V=V)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    for s in range(n)[:: max(1, n // 6)]:   # alone, in the largest cluster its row takes
        rows = slice(*d.cu[s:s + 2].tolist())
        got = [torch.full_like(t, -9) for t in (want[0][s:s + 1], want[1][rows], want[2][rows])]
        dg.dg_verify_drafts(x[rows], tok[rows], cu[s:s + 2] - cu[s], T[s:s + 1], u[rows], un[s:s + 1], *got, V=V)
        assert torch.equal(got[0], want[0][s:s + 1]) and torch.equal(got[1], want[1][rows]) and torch.equal(got[2], want[2][rows])
    assert dg.dg_get_device_status() & dg.DG_DEV_TIMEOUT == 0
    dg.dg_clear_device_status()


def test_verify_many_rejected_siblings():
    """A thousand siblings of 2^-24.03 of the mass each, rejected before the one in question: taken off an fp32 sum one by one
    they vanish, 5.8e-5 of it together.  Uniform numbers between the border and where it would then lie, and beyond."""
    us = [0.49999, 0.499995, 0.499999, 0.500001, 0.50001, 0.51, 0.4]
    d = Drafts([1002] * len(us), 1100, 1, T=1.0, dtype=torch.float32, tree=True)
    d.parents[:] = 0
    d.x[:, :1100] = -math.inf
    d.x[:, :2] = 0.0
    d.x[:, 2:1002] = -23.03 * math.log(2)
    d.u[:] = 0.9999
    for s, u in enumerate(us):
        d.tokens[1002 * s + 1:1002 * s + 1001] = torch.arange(2, 1002, dtype=torch.int32)
        d.tokens[1002 * s + 1001] = 1
        d.u[1002 * s + 1001] = u
    d.run().check()
    assert d.n_accept.tolist() == [int(u < 0.5) for u in us]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_verify_against_zero(dtype):
    """u q or u m of 0 is below every probability that is not 0, also below those that fp32 does not hold."""
    V, low = 50, [0.0, -84.5, -88.0, -90.0, -200.0, -600.0, -math.inf]

    def rows(n, **kw):
        d = Drafts(n, V, 3, T=1.0, dtype=dtype, **kw)
        d.x[:, :V] = -math.inf
        d.x[:, :len(low)] = torch.tensor(low, dtype=dtype)
        d.x[:, 10] = 0.0
        return d
    # chains of one draft: u = 0; and a draft whose distribution gave it 0
    d = rows([2] * len(low))
    d.tokens[1::2] = torch.arange(len(low), dtype=torch.int32)
    d.u[1::2] = 0.0
    d.run().check()
    assert d.n_accept.tolist() == [1] * (len(low) - 1) + [0]
    d = rows([2] * len(low), probs=True)
    d.tokens[1::2] = torch.arange(len(low), dtype=torch.int32)
    d.probs[:] = 0.0
    d.u[1::2] = 0.75
    d.run().check()
    assert d.n_accept.tolist() == [1] * (len(low) - 1) + [0]
    # behind siblings that are impossible, rejected, or so near their border that the row is summed exactly
    near = float(torch.nextafter(torch.tensor(0.5), torch.tensor(1.0)))
    d = rows([4] * len(low), tree=True)
    d.parents[:] = 0
    for s in range(len(low)):
        d.tokens[4 * s + 1:4 * s + 4] = torch.tensor([6, 10, s], dtype=torch.int32)
        d.u[4 * s + 1:4 * s + 4] = torch.tensor([0.0, near, 0.0])
    d.run().check()
    assert d.n_accept.tolist() == [1] * (len(low) - 1) + [0]
    assert d.path.view(-1, 4)[:-1, 1].tolist() == [3] * (len(low) - 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_verify_draft_distribution_of_the_targets(dtype):
    """A draft's distribution that is the target's, rounded to fp32: u just below 1 accepts (the rounding is at most 2^-24
    of p, and within 2^-28 of that in one comparison of some 600).  Rejected all the same (a token outside the vocabulary),
    its rounding alone is left, which weights within 2^-31 of p follow within 2^-30; with 1 everywhere nothing is left,
    and the row itself counts."""
    V, n = 400, 40

    def make(**kw):
        d = Drafts([3] * n, V, 5, T=1.0, probs=True, dtype=dtype, **kw)
        for s in range(n):
            for i in (1, 2):
                d.probs[3 * s + i, :V] = torch.softmax(d.x[3 * s + i - 1, :V].double(), 0).float()
        return d
    d = make()
    d.u[:] = 1 - 2.0 ** -24
    d.run().check(allow=1)
    assert (d.n_accept == 2).sum() >= n - 1
    d = make()
    d.tokens[1::3] = V
    d.run()
    assert dg.dg_get_device_status() == 0 and (d.n_accept == 0).all() and (d.out.view(n, 3)[:, 1:] == -1).all()
    for s, t in enumerate(d.out[::3].tolist()):
        p = torch.softmax(d.x[3 * s, :V].double(), 0)
        assert float(p[t] - d.probs[3 * s + 1, t].double()) >= -2.0 ** -30 * float(p[t]), s
    d = make()
    d.tokens[1::3] = -1
    d.probs[1::3] = 1.0
    d.run().check()
    assert (d.n_accept == 0).all()
    d = make()                     # one token that has everything, in the row and in the draft's
    d.x[:, :V] = -math.inf
    d.x[:, 7] = 2.0
    d.tokens[1::3] = 8
    d.probs[1::3] = 0.0
    d.probs[1::3, 7:9] = 1.0
    d.run().check()
    assert (d.out[::3] == 7).all()


# ------------------------------------------------------------------ normed append
@pytest.mark.parametrize("eps", [3.4028234663852886e38, 3.4e38, 2.0 ** 121, 2.0 ** 119])
@pytest.mark.parametrize("scale", [1.0, 1e16, 1.1e18, 1e30])
def test_append_norm_large_eps(scale, eps):
    """eps near fp32's largest number, beside squares whose mean would take their sum past it."""
    _append(ref.Batch([(7, 9, 1), (30, 64, 1)], 3, 1, 64, 16, seed=4, fill=0.0), 64, False, scale=scale, eps=eps)


# ------------------------------------------------------------------ the choice of path
@pytest.mark.parametrize("seqs,Hq,Hkv,D", [([(17, 200), (1, 1), (9, 60)] * 30, 4, 4, 64), ([(18, 200)] * 50, 8, 8, 64),
                                           ([(19, 200), (2, 30)] * 50, 8, 8, 64), ([(5, 90), (1, 2)] * 60, 12, 4, 128),
                                           ([(3, 90), (4, 4)] * 60, 3, 1, 256), ([(2, 90)] * 70, 8, 2, 256),
                                           ([(64, 500)], 8, 8, 128), ([(32, 400), (1, 9)], 16, 8, 64), ([(32, 77)] * 3, 4, 2, 256)])
def test_paths_on_either_side_of_the_rule(seqs, Hq, Hkv, D):
    """Calls near the number of rows, sequences and heads where the kernels for few rows hand over to those for many."""
    for window, sinks in ((-1, 0), (30, 3)):
        b, oks, mask, pos = _tree_batch(seqs, Hq, Hkv, D, 16, 29, window, sinks)
        _run_attention(b, oks, mask=mask, positions=pos, window=window, sinks=sinks)
        w, k = (window, sinks) if window >= 0 else (1000, 0)
        _run_attention(b, [dref.visible(a, m, window=w, sinks=k) for a, m in seqs], window=w, sinks=k)
