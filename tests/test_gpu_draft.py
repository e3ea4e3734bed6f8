"""GPU parity of the calls for drafted tokens against their fp64 forms (draft_ref.py).

Norm: the fp32 norm within (D / 16 + 12) 2^-24 relative (16 squares a lane, a tree over the lanes, division, square root,
two products), the rotation's bound on the normed values, one rounding to bf16 (2^-8).
Attention: see draft_ref.attention.  Verification: tokens and paths equal wherever no comparison came nearer
than 2^-28 to its border; the kernel's weights are within 2^-31.  Copies bit for bit."""
import math

import numpy as np
import pytest
import torch

import entropy_bounded_denoising_gb300 as dg

import draft_ref as dref
import serving_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


def _inv_freq(rot, theta=10000.0):
    return theta ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=DEV) / rot)


# ------------------------------------------------------------------ normed append
def _append(b, rot, interleaved, *, q_norm=True, k_norm=True, eps=1e-6, positions="random", in_place=False, with_q=True,
            scale=1.0, x=None, skip=(), status=0):
    g = torch.Generator(device=DEV).manual_seed(b.total * 7 + rot)
    w = _inv_freq(rot) if rot else None
    qkv = (torch.randn((b.total, (b.Hq + 2 * b.Hkv) * b.D), generator=g, device=DEV) * scale).to(ref.BF16)
    if x is not None:
        qkv = x(qkv)
    cut = lambda lo, h: qkv[:, lo * b.D:(lo + h) * b.D].unflatten(1, (h, b.D))  # noqa: E731
    q, k, v = cut(0, b.Hq), cut(b.Hq, b.Hkv), cut(b.Hq + b.Hkv, b.Hkv)
    if in_place:
        q = q.contiguous()
    q0 = q.clone()
    qn = torch.rand(b.D, generator=g, device=DEV) + 0.5 if q_norm and with_q else None
    kn = torch.rand(b.D, generator=g, device=DEV) * 2 - 1 if k_norm else None
    pos = torch.randint(-1000, 100000, (b.total,), generator=g, **I32) if positions == "random" else positions
    for c in (b.k_cache, b.v_cache):
        c.copy_(torch.randn(c.shape, generator=g, device=DEV).to(ref.BF16))
    kc, vc = b.k_cache.double(), b.v_cache.clone()
    q_out = q if in_place else torch.full((b.total, b.Hq, b.D), 7.0, dtype=ref.BF16, device=DEV)
    before = q_out.clone()
    dg.dg_clear_device_status()
    dg.dg_kv_append_norm(k, v, b.k_cache, b.v_cache, b.table, b.cu, b.kv_len, inv_freq=w, interleaved=interleaved,
                         q=q if with_q else None, q_out=q_out if with_q else None, q_norm=qn, k_norm=kn, eps=eps,
                         positions=pos)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == status
    w = torch.zeros(0, dtype=torch.float64, device=DEV) if w is None else w
    rel = (b.D / 16 + 12) * 2.0 ** -24
    q_ref, q_slack, k_slack = before.double(), torch.zeros(before.shape, dtype=torch.float64, device=DEV), torch.zeros_like(kc)

    def turned(x, weight, p):
        y = dref.normed(x.double(), weight, eps)
        z = ref.rotate(y, p, w, interleaved)
        slack = ref.rotation_bound(y, w, interleaved)
        both = torch.where(slack > 0, slack * 2.0 ** 21, y.abs())
        return z, slack + (rel * both if weight is not None else 0.0) + (2.0 ** -8 * z.abs() if weight is not None else
                                                                       torch.where(slack > 0, 2.0 ** -8 * z.abs(), 0.0))

    cu = b.cu.tolist()
    for s, (a, kl, _) in enumerate(b.seqs):
        if a == 0 or kl == 0 or s in skip:
            continue
        rows = slice(cu[s], cu[s + 1])
        slots = torch.arange(kl - a, kl, device=DEV)
        p = slots if pos is None else pos[rows]
        at = b.slots(s, slots)
        kc[at], k_slack[at] = turned(k[rows], kn, p)
        vc[at] = v[rows]
        if with_q:
            q_ref[rows], q_slack[rows] = turned(q0[rows], qn, p)
    assert torch.equal(b.v_cache.view(torch.int16), vc.view(torch.int16))
    for got, want, slack in ((b.k_cache, kc, k_slack), (q_out, q_ref, q_slack)):
        err = (got.double() - want).abs()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        assert (err <= slack)[~nan].all(), float((err - slack)[~nan].max())
    return b, q_out


SEQS = [(1, 1, 1), (0, 40, 1), (1, 300, 1), (17, 33, 0), (0, 0, 1), (2, 0, 1), (64, 64, 1), (256, 300, 0), (3, 129, 1)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,page,Hq,Hkv,head_major", [(64, 64, 8, 1, 1, False), (64, 16, 16, 7, 1, True),
                                                          (128, 128, 16, 16, 8, False), (128, 64, 64, 5, 5, True),
                                                          (256, 256, 32, 4, 2, False), (256, 48, 128, 24, 3, True)])
def test_append_norm(D, rot, page, Hq, Hkv, head_major, interleaved):
    _append(ref.Batch(SEQS, Hq, Hkv, D, page, seed=D + rot, head_major=head_major, before=3, after=5), rot, interleaved)


def test_append_norm_variants():
    make = lambda seqs=SEQS, **kw: ref.Batch(seqs, 4, 2, 128, 16, seed=9, **kw)  # noqa: E731
    _append(make(), 128, False, q_norm=False)
    _append(make(), 128, True, k_norm=False, in_place=True)
    _append(make(), 0, False, eps=0.5)
    _append(make(after=2), 64, False, with_q=False)
    _append(make(), 128, False, positions=None)
    _append(make([(1, 77, 1)]), 128, False)
    _append(make([(1, 1 + i, 1) for i in range(1500)]), 128, False)
    _append(make([(0, 5, 1)] * 70 + [(2, 9, 1)] + [(0, 0, 1)] * 1100 + [(1, 4, 1)], after=1), 64, False)
    _append(ref.Batch([(2, 9, 1), (1500, 1600, 1)], 64, 8, 128, 16, seed=2), 128, False)   # several rounds of blocks


def test_append_norm_as_append():
    """Without norms and positions: dg_kv_append, bit for bit."""
    for interleaved in (False, True):
        b = ref.Batch(SEQS, 4, 2, 128, 16, seed=5, after=3, fill=0.0)
        g = torch.Generator(device=DEV).manual_seed(1)
        q, k, v = (torch.randn((b.total, h, 128), generator=g, device=DEV).to(ref.BF16) for h in (4, 2, 2))
        res = []
        for call in (dg.dg_kv_append, dg.dg_kv_append_norm):
            b.k_cache.zero_(), b.v_cache.zero_()
            out = torch.zeros_like(q)
            call(k, v, b.k_cache, b.v_cache, b.table, b.cu, b.kv_len, inv_freq=_inv_freq(64), interleaved=interleaved,
                 q=q, q_out=out)
            res.append((out, b.k_cache.clone(), b.v_cache.clone()))
        assert all(torch.equal(x, y) for x, y in zip(*res))


def test_append_norm_sizes_of_values():
    """Rows whose squares leave fp32, tiny rows beside eps, zeros, infinities and NaN."""
    make = lambda: ref.Batch([(7, 9, 1), (30, 64, 1)], 3, 1, 128, 16, seed=4, fill=0.0)  # noqa: E731
    for scale in (1e-30, 1e-19, 1e18, 3e19, 1e30, 1e37):
        _append(make(), 128, False, scale=scale)
        _append(make(), 32, True, scale=scale, eps=2.0 ** -126)

    def odd(x):
        x = x.clone()
        x[0] = 0.0
        x[1, :128] = math.inf
        x[2, 5] = math.inf
        x[3, 130] = math.nan
        x[4] = 3.3e38
        return x
    _append(make(), 0, False, x=odd)
    # a NaN turns with its pair: the other heads are as they are
    b, q = _append(make(), 0, False, x=odd, positions=None)
    assert torch.isfinite(q[4:]).all() and (q[0] == 0).all()


def test_append_norm_refused_sequences():
    b = ref.Batch([(3, 20, 1), (4, 30, 1), (2, 18, 1)], 2, 1, 64, 16, seed=3)
    b.kv_len[1] = 3                       # fewer keys than rows
    b.seqs[1] = (4, 0, 1)
    _append(b, 64, False, skip=(1,), status=dg.DG_DEV_BAD_PARAM)
    b = ref.Batch([(3, 20, 1), (4, 30, 1)], 2, 1, 64, 16, seed=3)
    b.table[1, 1] = b.n_pages             # positions 26 .. 29 lie there: nothing of them is written
    _append(b, 64, False, skip=(1,), status=dg.DG_DEV_BAD_PARAM)


# ------------------------------------------------------------------ attention
def _run_attention(b, oks, *, mask=None, positions=None, window=-1, sinks=0, scale=None, max_q=None, status=0, skip=(),
                   sentinel=5.0, call=None):
    o = torch.full((b.total, b.Hq, b.D), sentinel, dtype=ref.BF16, device=DEV)
    lse = torch.full((b.total, b.Hq), sentinel, device=DEV)
    max_q = max([1] + [s[0] for s in b.seqs]) if max_q is None else max_q
    need = dg.dg_tree_attention_workspace_bytes(len(b.seqs), max_q, b.Hq, b.Hkv, b.D)
    ws = torch.full((max(16, need),), 255, dtype=torch.uint8, device=DEV)
    dg.dg_clear_device_status()
    if mask is not None:
        dg.dg_tree_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, mask, max_q, positions=positions,
                             lse=lse, window=window, sinks=sinks, scale=scale, workspace=ws)
    else:
        dg.dg_sink_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, max_q, lse=lse, window=window,
                             sinks=sinks, scale=scale, workspace=ws)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == status
    dref.check_attention(b, o, lse, oks, scale, sentinel, skip)
    return o, lse


def _tree_batch(seqs, Hq, Hkv, D, page, seed, window=-1, sinks=0, extra_words=0, anc_of=None, **kw):
    """A batch of random trees: seqs [(nodes, keys)]."""
    b = ref.Batch([(a, m, 1) for a, m in seqs], Hq, Hkv, D, page, seed=seed, **kw).fill_keys()
    g = torch.Generator().manual_seed(seed)
    width = -(-max([1] + [a for a, _ in seqs]) // 32) + extra_words
    sets, pos, oks = [set()] * int(b.cu[0]), [0] * int(b.cu[0]), []
    for a, m in seqs:
        _, depth, anc = dref.random_tree(g, a) if a else ([], [], [])
        if anc_of:
            anc = anc_of(a, anc)
        p = [m - a + d for d in depth]
        oks.append(dref.visible(a, m, anc=anc, positions=p, window=window, sinks=sinks) if m and a else None)
        sets += anc
        pos += p
    pad = b.total - len(sets)
    mask = dref.words(sets + [set(range(width * 32))] * pad, width, DEV)
    return b, oks, mask, torch.tensor(pos + [0] * pad, **I32)


TREES = [(1, 1), (5, 5), (8, 300), (0, 40), (33, 64), (0, 0), (3, 0), (64, 500), (2, 65), (61, 1000), (1, 129)]


@pytest.mark.parametrize("window,sinks", [(-1, 0), (40, 0), (100, 70), (0, 1)])
@pytest.mark.parametrize("Hq,Hkv,D,page,head_major", [(16, 8, 128, 16, False), (6, 2, 64, 8, True), (5, 1, 256, 64, False),
                                                      (2, 2, 64, 128, False), (24, 2, 128, 32, True)])
def test_tree_attention(Hq, Hkv, D, page, head_major, window, sinks):
    b, oks, mask, pos = _tree_batch(TREES, Hq, Hkv, D, page, 11, window, sinks, head_major=head_major, before=2, after=3)
    _run_attention(b, oks, mask=mask, positions=pos if window >= 0 else None, window=window, sinks=sinks)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 128), (20, 4, 256), (7, 1, 64), (160, 1, 64), (128, 1, 128)])
def test_tree_attention_sizes(Hq, Hkv, D):
    """Many nodes, odd groups, groups of more heads than a tile has rows, long contexts."""
    b, oks, mask, pos = _tree_batch([(199, 1300), (1, 5000), (128, 128), (130, 700)] if Hq < 100 else [(3, 200), (17, 90)],
                                    Hq, Hkv, D, 32, 5, 300, 20, extra_words=2)
    _run_attention(b, oks, mask=mask, positions=pos, window=300, sinks=20)
    _run_attention(b, [dref.visible(a, m, anc=[{j for j in range(a) if ok[i, m - a + j]} for i in range(a)])
                       for (a, m, _), ok in zip(b.seqs, oks)], mask=mask)


@pytest.mark.parametrize("n,a,m", [(1, 1, 1), (1, 8, 1024), (1, 64, 9000), (3, 300, 333), (200, 1, 70), (1100, 2, 9), (70, 33, 190)])
def test_tree_attention_batches(n, a, m):
    g = torch.Generator().manual_seed(n)
    seqs = [(a, m)] + [(a, a + int(torch.randint(0, m - a + 1, (1,), generator=g))) for _ in range(n - 1)]
    b, oks, mask, _ = _tree_batch(seqs, 8, 2, 128, 16, n + a)
    _run_attention(b, oks, mask=mask)


def test_tree_attention_masks():
    """Rows whose mask leaves nothing, masks that say anything, bits behind the last node."""
    empty = lambda a, anc: [set() if i % 3 == 0 else s | {a, a + 1, 63} for i, s in enumerate(anc)]  # noqa: E731
    seqs = [(30, 30), (10, 10), (1, 1), (12, 80), (64, 64)]
    b, oks, mask, pos = _tree_batch(seqs, 4, 2, 128, 16, 3, anc_of=empty)
    _run_attention(b, oks, mask=mask)
    # every row empty; with a window of 0 and no sinks over context that is farther away
    b, oks, mask, pos = _tree_batch(seqs, 4, 2, 64, 16, 3, 0, 0, anc_of=lambda a, anc: [set() for _ in anc])
    oks = [dref.visible(a, m, anc=[set()] * a, positions=[1000] * a, window=0) for a, m in seqs]
    o, lse = _run_attention(b, oks, mask=mask, positions=torch.full_like(pos, 1000), window=0)
    assert (o == 0).all() and (lse == -math.inf).all()
    # each node sees one other only, the last ones included
    b, oks, mask, _ = _tree_batch([(100, 164), (64, 65)], 4, 1, 128, 16, 6, anc_of=lambda a, anc: [{a - 1 - i} for i in range(a)])
    _run_attention(b, oks, mask=mask)


def test_tree_attention_unseen_values():
    """What no query sees may hold anything: nodes that no mask names, context behind the window, slots past the last key
    and pages that nobody needs."""
    for D, Hq, Hkv in ((64, 4, 2), (128, 16, 8), (256, 3, 1)):
        seqs = [(40, 300), (70, 70), (9, 500)]
        hidden = lambda a, anc: [{j for j in s if j % 5 != 2} | {0} for s in anc]  # noqa: E731
        b, oks, mask, pos = _tree_batch(seqs, Hq, Hkv, D, 16, 8, 50, 3, anc_of=hidden)
        for s, (a, m) in enumerate(seqs):
            unseen = torch.nonzero(~oks[s].any(0))[:, 0]
            assert len(unseen) > 5
            at = b.slots(s, unseen)
            b.k_cache[at] = math.nan
            b.v_cache[at] = torch.tensor([math.inf, -math.inf, math.nan, 3e38] * (D // 4), dtype=ref.BF16, device=DEV)
            for page in range(-(-m // 16)):   # pages out of sight have no entry at all
                if not oks[s][:, page * 16:page * 16 + 16].any():
                    b.table[s, page] = -9
        clean = ref.Batch.keys

        def keys(self, s):
            at = self.table[s].long().clamp(min=0)[torch.arange(seqs[s][1], device=DEV) // 16], torch.arange(seqs[s][1], device=DEV) % 16
            return self.k_cache[at], self.v_cache[at]
        b.keys = keys.__get__(b)
        _run_attention(b, oks, mask=mask, positions=pos, window=50, sinks=3)
        assert clean


def test_tree_attention_scales_and_scores():
    for scale in (0.0, -0.3, 2.0, 1e-30):
        b, oks, mask, _ = _tree_batch([(20, 130), (3, 3), (64, 64)], 4, 2, 128, 16, 21)
        _run_attention(b, oks, mask=mask, scale=scale)
    b, oks, mask, _ = _tree_batch([(20, 400), (50, 61)], 4, 2, 64, 16, 22, q_scale=60.0)   # far apart scores
    _run_attention(b, oks, mask=mask)


def test_tree_attention_refused_sequences():
    seqs = [(4, 40), (5, 50), (6, 60), (7, 70)]
    def fresh():
        return _tree_batch(seqs, 4, 2, 128, 16, 31)
    bad = dg.DG_DEV_BAD_PARAM
    b, oks, mask, _ = fresh()
    b.kv_len[1] = 4                        # fewer keys than queries
    _run_attention(b, oks, mask=mask, status=bad, skip=(1,))
    b, oks, mask, _ = fresh()
    b.kv_len[2] = 10 ** 6                  # more than the table holds
    _run_attention(b, oks, mask=mask, status=bad, skip=(2,))
    b, oks, mask, _ = fresh()
    _run_attention(b, oks, mask=mask, max_q=6, status=bad, skip=(3,))      # more queries than max_q_len
    b, oks, mask, _ = fresh()
    b.cu[4] = 10 ** 6
    _run_attention(b, oks, mask=mask, status=bad, skip=(3,))
    b, oks, mask, _ = fresh()
    b.table[0, 1] = b.n_pages              # a page outside the pool: the others are right
    o = torch.full((b.total, 4, 128), 5.0, dtype=ref.BF16, device=DEV)
    lse = torch.zeros((b.total, 4), device=DEV)
    dg.dg_clear_device_status()
    dg.dg_tree_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, mask, 7, lse=lse)
    assert dg.dg_get_device_status() == bad
    dref.check_attention(b, o, lse, oks, skip=(0,))


@pytest.mark.parametrize("Hq,Hkv,D,page,head_major", [(16, 8, 128, 16, False), (8, 8, 64, 8, True), (5, 1, 256, 64, False)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (17, 4), (64, 64), (200, 100), (1 << 30, 7), (5, 1 << 30)])
def test_sink_attention(Hq, Hkv, D, page, head_major, window, sinks):
    seqs = [(1, 1), (1, 700), (0, 40), (300, 300), (0, 0), (2, 0), (129, 900), (64, 65), (5, 4000)]
    b = ref.Batch([(a, m, 1) for a, m in seqs], Hq, Hkv, D, page, seed=window % 97 + D, head_major=head_major, before=1,
                  after=4).fill_keys()
    oks = [dref.visible(a, m, window=window, sinks=sinks) if a and m else None for a, m in seqs]
    _run_attention(b, oks, window=window, sinks=sinks)


def test_sink_attention_prompts_and_batches():
    b = ref.Batch([(2000, 2300, 1), (1500, 1500, 1), (1, 2222, 1)], 4, 1, 128, 64, seed=1).fill_keys()
    _run_attention(b, [dref.visible(a, m, window=333, sinks=10) for a, m, _ in b.seqs], window=333, sinks=10)
    b = ref.Batch([(1, 1 + 5 * i, 1) for i in range(400)], 8, 4, 64, 16, seed=2).fill_keys()
    _run_attention(b, [dref.visible(a, m, window=100, sinks=4) for a, m, _ in b.seqs], window=100, sinks=4)
    # context between the sinks and the window may hold anything, and have no pages
    b = ref.Batch([(3, 900, 1), (1, 600, 1)], 8, 4, 128, 16, seed=3).fill_keys()
    oks = [dref.visible(a, m, window=70, sinks=5) for a, m, _ in b.seqs]
    k, v = zip(*[b.keys(s) for s in range(2)])
    b.keys = lambda s: (k[s], v[s])
    for s, (a, m, _) in enumerate(b.seqs):
        at = b.slots(s, torch.nonzero(~oks[s].any(0))[:, 0])
        b.k_cache[at] = math.nan
        b.v_cache[at] = math.nan
        b.table[s, 1:(m - a - 70) // 16] = 1 << 30
    _run_attention(b, oks, window=70, sinks=5)


def test_sink_attention_is_causal_attention():
    """A window that reaches everything: dg_paged_attention within its bound."""
    b = ref.Batch([(1, 500, 1), (40, 600, 1), (128, 128, 1)], 8, 2, 128, 16, seed=7).fill_keys()
    o, _ = _run_attention(b, [dref.visible(a, m) for a, m, _ in b.seqs], window=1 << 20, sinks=0)
    o2 = torch.zeros_like(o)
    dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o2, b.table, b.cu, b.kv_len, b.causal, 128)
    ref.check_attention(b, o2, None)


@pytest.mark.parametrize("nodes", [9, 90])
def test_attention_far_pages(nodes):
    """Offsets past 2^31 elements: pages spread over a pool of 2 * 4.3 GB."""
    n_pages, page, H, D = 33000, 64, 8, 128
    k = torch.empty((n_pages, page, H, D), dtype=ref.BF16, device=DEV)   # 2^31 elements: page 32768
    v = torch.empty_like(k)
    b = ref.Batch([(nodes, 200, 1)], 16, H, D, page, seed=2).fill_keys()
    kk, vv = b.keys(0)
    pages = [n_pages - 1, 0, n_pages - 2, 4500]
    b.table = torch.tensor([pages], **I32)
    b.k_cache, b.v_cache, b.n_pages = k, v, n_pages
    at = b.slots(0, range(200))
    k[at], v[at] = kk, vv
    anc = [set(range(i + 1)) for i in range(nodes)]
    _run_attention(b, [dref.visible(nodes, 200, anc=anc)], mask=dref.words(anc, 3, DEV))


# few rows a key head take kernels of their own: the same edges there
SMALL = [(4, 300), (3, 3), (1, 1), (0, 9), (0, 0), (2, 0), (4, 64), (1, 700), (3, 65)]


@pytest.mark.parametrize("window,sinks", [(-1, 0), (40, 0), (100, 70), (0, 1)])
@pytest.mark.parametrize("Hq,Hkv,D,page,head_major", [(16, 8, 128, 16, False), (4, 4, 64, 8, True), (4, 1, 256, 64, False),
                                                      (8, 4, 64, 16, False), (2, 1, 128, 32, True), (3, 1, 256, 8, False)])
def test_small_trees(Hq, Hkv, D, page, head_major, window, sinks):
    b, oks, mask, pos = _tree_batch(SMALL, Hq, Hkv, D, page, 12, window, sinks, head_major=head_major, before=2, after=3)
    _run_attention(b, oks, mask=mask, positions=pos if window >= 0 else None, window=window, sinks=sinks)


@pytest.mark.parametrize("D,page,head_major", [(64, 8, False), (128, 16, True), (128, 128, False), (256, 64, True), (256, 8, False)])
@pytest.mark.parametrize("gap", ["columns", "slots", "heads"])
def test_trees_over_strided_caches(D, page, head_major, gap):
    """Caches with gaps behind their columns, slots or heads."""
    for seqs in ([(70, 200), (5, 5), (40, 333), (1, 64)], [(2, 130), (1, 1)]):
        b, oks, mask, pos = _tree_batch(seqs, 6, 3, D, page, 4, 50, 3, head_major=head_major)
        for name in ("k_cache", "v_cache"):
            old = getattr(b, name)
            n, slots, heads, _ = old.shape
            s, h, d = page + (gap == "slots"), heads + (gap == "heads"), D + (8 if gap == "columns" else 0)
            wide = torch.full((n, h, s, d) if head_major else (n, s, h, d), math.nan, dtype=ref.BF16, device=DEV)
            new = (wide.transpose(1, 2) if head_major else wide)[:, :page, :heads, :D]
            new.copy_(old)
            setattr(b, name, new)
        _run_attention(b, oks, mask=mask, positions=pos, window=50, sinks=3)


def test_small_trees_in_pairs():
    """One or two nodes over heads of 64: two key heads go as one."""
    for window, sinks in ((-1, 0), (30, 5)):
        b, oks, mask, pos = _tree_batch([(2, 200), (1, 1), (2, 2), (1, 90), (2, 1000)], 8, 8, 64, 16, 4, window, sinks)
        _run_attention(b, oks, mask=mask, positions=pos, window=window, sinks=sinks)


def test_small_trees_masks_and_values():
    empty = lambda a, anc: [set() if i % 3 == 0 else s | {a, a + 1, 31} for i, s in enumerate(anc)]  # noqa: E731
    seqs = [(4, 4), (3, 3), (1, 1), (4, 80), (2, 64)]
    for D, Hkv in ((64, 2), (128, 2), (256, 1)):
        b, oks, mask, pos = _tree_batch(seqs, 4 * Hkv, Hkv, D, 16, 3, anc_of=empty)
        _run_attention(b, oks, mask=mask)
        for scale in (0.0, -0.3, 1e-30):
            _run_attention(b, oks, mask=mask, scale=scale)
        # all rows empty
        b, oks, mask, pos = _tree_batch(seqs, 4 * Hkv, Hkv, D, 16, 3, 0, 0, anc_of=lambda a, anc: [set() for _ in anc])
        oks = [dref.visible(a, m, anc=[set()] * a, positions=[1000] * a, window=0) for a, m in seqs]
        o, lse = _run_attention(b, oks, mask=mask, positions=torch.full_like(pos, 1000), window=0)
        assert (o == 0).all() and (lse == -math.inf).all()
        # what nobody sees
        hidden = lambda a, anc: [{j for j in s if j != 1} | {0} for s in anc]  # noqa: E731
        b, oks, mask, pos = _tree_batch([(4, 300), (4, 4), (3, 500)], 4 * Hkv, Hkv, D, 16, 8, 50, 3, anc_of=hidden)
        keys = [b.keys(s) for s in range(3)]
        b.keys = lambda s: keys[s]
        for s, (a, m, _) in enumerate(b.seqs):
            at = b.slots(s, torch.nonzero(~oks[s].any(0))[:, 0])
            b.k_cache[at] = math.nan
            b.v_cache[at] = torch.tensor([math.inf, -math.inf, math.nan, 3e38] * (D // 4), dtype=ref.BF16, device=DEV)
            for page in range(-(-m // 16)):
                if not oks[s][:, page * 16:page * 16 + 16].any():
                    b.table[s, page] = -9
        _run_attention(b, oks, mask=mask, positions=pos, window=50, sinks=3)


def test_tree_positions_before_the_context():
    """A node's position below its context's length counts as that length."""
    for seqs in ([(4, 300), (2, 70)], [(60, 300), (20, 90)]):
        b, _, mask, pos = _tree_batch(seqs, 8, 2, 128, 16, 5)
        low = torch.randint(-1000, 200, pos.shape, **I32)
        oks, at = [], 0
        words = mask.cpu().numpy().view("uint8")
        for a, m in seqs:
            bits = np.unpackbits(words[at:at + a], axis=1, bitorder="little")
            anc = [set(np.nonzero(r)[0].tolist()) for r in bits]
            oks.append(dref.visible(a, m, anc=anc, positions=[max(p, m - a) for p in low[at:at + a].tolist()], window=33, sinks=2))
            at += a
        _run_attention(b, oks, mask=mask, positions=low, window=33, sinks=2)


def test_sink_prompts_unseen_context():
    b = ref.Batch([(100, 900, 1), (40, 600, 1)], 8, 4, 128, 16, seed=3).fill_keys()
    oks = [dref.visible(a, m, window=70, sinks=5) for a, m, _ in b.seqs]
    keys = [b.keys(s) for s in range(2)]
    b.keys = lambda s: keys[s]
    for s, (a, m, _) in enumerate(b.seqs):
        at = b.slots(s, torch.nonzero(~oks[s].any(0))[:, 0])
        b.k_cache[at] = math.nan
        b.v_cache[at] = math.nan
        b.table[s, 1:(m - a - 70) // 16] = 1 << 30
    _run_attention(b, oks, window=70, sinks=5)


# ------------------------------------------------------------------ verification
class Drafts:
    """sizes: nodes of each sequence."""

    def __init__(self, sizes, V, seed, *, dtype=torch.bfloat16, tree=False, probs=False, T=None, std=3.0, pad=0, near=0.6,
                 before=0, after=0):
        g = torch.Generator().manual_seed(seed)
        self.sizes, self.V = sizes, V
        cu = [before]
        for s in sizes:
            cu.append(cu[-1] + s)
        self.total = cu[-1] + after
        self.cu = torch.tensor(cu, **I32)
        ld = -(-V // 8) * 8 + pad
        self.x = torch.full((self.total, ld), math.nan, dtype=dtype)
        self.x[:, :V] = (torch.randn((self.total, V), generator=g) * std).to(dtype)
        n = len(sizes)
        self.T = torch.tensor([0.0 if i % 5 == 4 else 0.3 + 0.2 * (i % 7) for i in range(n)] if T is None else [T] * n)
        self.u = torch.rand(self.total, generator=g)
        self.un = torch.rand(n, generator=g)
        self.tokens = torch.randint(0, V, (self.total,), generator=g, dtype=torch.int32)
        self.parents = self.probs = None
        par = []
        for s, q in enumerate(sizes):
            p = dref.random_tree(g, q, 2)[0] if tree and q else list(range(-1, q - 1))
            par += p
            for i in range(1, q):
                row = self.x[cu[s] + p[i], :V].float()
                if torch.rand(1, generator=g) < near:
                    top = row.topk(min(3, V)).indices
                    self.tokens[cu[s] + i] = int(top[int(torch.randint(0, len(top), (1,), generator=g))])
        if tree:
            self.parents = torch.tensor([-5] * before + [p if p >= 0 else 99999 for p in par] + [-7] * after, dtype=torch.int32)
        if probs:
            self.probs = torch.zeros((self.total, -(-V // 4) * 4))
            for s, q in enumerate(sizes):
                for i in range(1, q):
                    row = self.x[cu[s] + i - 1, :V].float() + 0.7 * torch.randn(V, generator=g)
                    pr = (row / max(float(self.T[s]), 0.1)).softmax(0)
                    self.probs[cu[s] + i, :V] = pr
                    self.tokens[cu[s] + i] = int(torch.multinomial(pr, 1, generator=g))

    def run(self, stream=None, out=None, **kw):
        d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        self.dev = [d(t) for t in (self.x, self.tokens, self.cu, self.T, self.u, self.un, self.parents, self.probs)]
        x, tok, cu, T, u, un, par, probs = self.dev
        self.n_accept = torch.full((len(self.sizes),), -9, **I32)
        self.path, self.out = torch.full((self.total,), -9, **I32), torch.full((self.total,), -9, **I32)
        dg.dg_clear_device_status()
        dg.dg_verify_drafts(x, tok, cu, T, u, un, self.n_accept, self.path, self.out, parents=par, draft_probs=probs, V=self.V,
                            stream=stream)
        torch.cuda.synchronize()
        return self

    def check(self, status=0, skip=(), near=2.0 ** -28, allow=0):
        assert dg.dg_get_device_status() == status
        cu, n_acc, path, out = self.cu.tolist(), self.n_accept.tolist(), self.path.tolist(), self.out.tolist()
        owned, close, accepted = set(), 0, 0
        for s, q in enumerate(self.sizes):
            rows = range(cu[s], cu[s] + q)
            owned |= set(rows)
            if s in skip:
                continue
            if q == 0:
                assert n_acc[s] == -1
                continue
            lo = cu[s]
            sl = slice(lo, lo + q)
            p, t, gap = dref.verify(self.x[sl, :self.V], self.tokens[sl], float(self.T[s]), self.u[sl], self.un[s].double(),
                                    None if self.parents is None else self.parents[sl].tolist(),
                                    None if self.probs is None else self.probs[sl, :self.V])
            if gap < near:
                close += 1
                continue
            assert n_acc[s] == len(p) - 1, (s, n_acc[s], p)
            assert path[lo:lo + q] == p + [-1] * (q - len(p)), s
            assert out[lo:lo + q] == t + [-1] * (q - len(t)), (s, out[lo:lo + q], t, gap)
            accepted += n_acc[s]
        assert close <= allow
        assert all(path[i] == -9 and out[i] == -9 for i in range(self.total) if i not in owned)
        return accepted


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [2, 7, 1000, 4097, 32768, 152063])
@pytest.mark.parametrize("kind", ["chain", "probs", "tree"])
def test_verify(kind, V, dtype):
    sizes = [6, 1, 0, 9, 2, 5, 5, 3, 7, 1, 33, 12]
    d = Drafts(sizes, V, V + len(kind), dtype=dtype, tree=kind == "tree", probs=kind == "probs", pad=8, before=2, after=3)
    # a draw of a thousand tokens comes within 2^-28 of a border once in some ten thousand; of 2^17, in a thousand
    d.run().check(allow=1 if V > 30000 else 0)


def test_verify_many_and_large():
    d = Drafts([4] * 300, 500, 5, tree=True)
    assert d.run().check() > 50
    d = Drafts([1] * 1000 + [3], 64, 6)
    d.run().check()
    d = Drafts([1024, 3, 1000], 50, 7, tree=True, std=0.5)
    d.run().check()
    d = Drafts([4, 3], 262144, 8, probs=True, std=2.0)
    d.run().check(allow=1)
    d = Drafts([2], 1 << 21, 9, dtype=torch.float32)
    d.run().check(allow=1)


def test_verify_flat_and_peaked():
    """All tokens alike (every border counts), one token that has everything, masked tokens."""
    d = Drafts([1] * 200, 2048, 1, T=1.0, std=0.0)
    d.run().check()
    want = (d.un.double() * 2048).floor().int()
    assert torch.equal(d.out.cpu(), want)
    d = Drafts([5, 4], 3000, 2, T=0.05, std=30.0, tree=True)
    d.run().check()
    d = Drafts([5, 4, 6, 6], 3000, 3, tree=True)
    d.x[:, :3000][:, torch.arange(3000) % 3 != 1] = -math.inf
    d.run().check()
    d = Drafts([3, 3], 300, 3)
    d.x[:, :300] = -math.inf
    d.x[:, 17] = -5.0
    d.tokens[:] = 17
    d.run().check()
    assert d.n_accept.tolist() == [2, 2] and d.out.tolist() == [17] * 6


def test_verify_borders():
    """Uniform numbers right at a probability's border, where fp32 sums do not decide."""
    V = 5000
    for tree in (False, True):
        d = Drafts([4] * 64, V, 12, T=0.7, tree=tree, near=1.0)
        cu = d.cu.tolist()
        for s in range(64):      # the first child's border, a little below or above
            p = torch.softmax(d.x[cu[s], :V].double() / float(d.T[s].double()), 0)
            b = float(p[int(d.tokens[cu[s] + 1])])
            near = torch.tensor(b, dtype=torch.float32)
            steps = (s % 5) - 2
            for _ in range(abs(steps)):
                near = torch.nextafter(near, torch.tensor(2.0 if steps > 0 else 0.0))
            d.u[cu[s] + 1] = near
        d.run().check(allow=3)
    # and the draws: at the border of token 40 of a flat row of 64, one step either way
    d = Drafts([1] * 3, 64, 1, T=1.0, std=0.0)
    e = torch.tensor(40 / 64)
    d.un = torch.stack([torch.nextafter(e, torch.tensor(0.0)), e, torch.nextafter(e, torch.tensor(1.0))])
    d.run()
    assert d.out.tolist() == [39, 40, 40]
    d.un = torch.tensor([0.0, 1 - 2.0 ** -24, 2.0 ** -149])
    d.run()
    assert d.out.tolist() == [0, 63, 0]


def test_verify_odd_drafts():
    V = 400
    d = Drafts([6, 6, 6], V, 3, T=1.0)
    d.tokens[1] = -1
    d.tokens[7] = V
    d.tokens[13] = 2 ** 31 - 1
    d.run().check()
    assert d.n_accept.tolist() == [0, 0, 0]
    # children with one token, several times
    d = Drafts([40] * 20, V, 4, T=0.5, tree=True)
    d.parents[:] = 0
    d.tokens[:] = torch.arange(800, dtype=torch.int32) % 3
    d.u[:] = 0.9999
    d.run().check()
    # every token a rejected child but one; and all of them (then the row itself counts)
    for last in (0, 1):
        d = Drafts([65 + last - 1 + 1], 64, 4, T=1.0, tree=True, std=0.1)
        d.parents[:] = 0
        d.tokens[1:] = torch.arange(d.total - 1, dtype=torch.int32)[:] % 64
        d.u[:] = 1 - 2.0 ** -24
        if not last:
            d.tokens[64] = 5
        d.run().check(near=2.0 ** -20, allow=1)
    # the draft's distribution is the target's, or zero where it was drawn, or no distribution at all
    d = Drafts([3] * 40, V, 5, T=1.0, probs=True, dtype=torch.float32)
    for s in range(40):
        for i in (1, 2):
            d.probs[3 * s + i, :V] = torch.softmax(d.x[3 * s + i - 1, :V].double(), 0).float()
    d.u[:] = 1 - 2.0 ** -24
    d.run()
    d = Drafts([3] * 40, V, 5, T=1.0, probs=True)
    for s in range(40):
        d.probs[3 * s + 1, :V] = [0.0, 1.0, 7.0, -1.0, math.nan, math.inf, 2.0 ** -140][s % 7]
    d.u[1::3] = 0.99
    d.run().check()


def test_verify_temperatures():
    """Temperatures at the ends of their range: the largest token alone, and all tokens but the masked ones alike."""
    V = 640
    for dtype in (torch.bfloat16, torch.float32):
        d = Drafts([4] * 30, V, 6, T=2.0 ** -64, dtype=dtype)
        d.x[:, 5] = 100.0
        d.run().check()
        assert (d.out.view(30, 4)[:, 0] == 5).all()
        d = Drafts([1] * 50, V, 6, T=2.0 ** 64, dtype=dtype)
        d.x[:, :V] = torch.where(torch.arange(V) % 2 == 0, torch.full_like(d.x[:, :V], -math.inf), d.x[:, :V])
        d.run()
        assert dg.dg_get_device_status() == 0
        want = ((d.un.double() * (V // 2)).floor() * 2 + 1).int()
        assert torch.equal(d.out.cpu(), want)
    d = Drafts([1] * 50, V, 6, T=1.0, dtype=torch.float32, std=1e38)   # differences past fp32
    over = torch.isinf(d.x).any(1).tolist()                             # some rows hold an infinity
    d.run().check(status=1, skip=[s for s in range(50) if over[s]])
    d.x = d.x.clamp(-3e38, 3e38)
    d.run().check()


def test_verify_nothing():
    d = Drafts([0, 0], 16, 1)
    d.run().check()
    assert d.n_accept.tolist() == [-1, -1]
    z = torch.zeros(0, **I32)
    dg.dg_verify_drafts(torch.zeros((0, 16), device=DEV), z, z.new_zeros(1), torch.zeros(0, device=DEV),
                        torch.zeros(0, device=DEV), torch.zeros(0, device=DEV), z, z.clone(), z.clone())


def test_verify_distribution():
    """20000 chains from one pair of distributions: the first token produced has the target's."""
    n, V = 20000, 12
    g = torch.Generator().manual_seed(0)
    x = torch.randn((1, 16), generator=g).expand(2 * n, 16).contiguous()
    p = torch.softmax(x[0, :V].double(), 0)
    for probs in (True, False):
        q = torch.softmax(torch.randn(V, generator=g).double(), 0)
        tok = torch.zeros(2 * n, dtype=torch.int32)
        tok[1::2] = torch.multinomial(q, n, replacement=True, generator=g).int()
        qq = torch.zeros((2 * n, V))
        qq[1::2] = q.float()
        count, path, out = torch.zeros(n, **I32), torch.zeros(2 * n, **I32), torch.zeros(2 * n, **I32)
        dg.dg_verify_drafts(x.to(DEV), tok.to(DEV), torch.arange(0, 2 * n + 1, 2, **I32), torch.ones(n, device=DEV),
                            torch.rand(2 * n, generator=g).to(DEV), torch.rand(n, generator=g).to(DEV), count, path, out,
                            draft_probs=qq.to(DEV) if probs else None, V=V)
        got = torch.bincount(out[::2].cpu().long(), minlength=V).double()
        chi2 = float(((got - n * p) ** 2 / (n * p)).sum())
        assert chi2 < 40.0    # 11 degrees of freedom: 40 is passed once in 30000 times
        accept = float((count == 1).double().mean())
        want = float(torch.minimum(p, q).sum()) if probs else float((p * q).sum())
        assert abs(accept - want) < 5 * math.sqrt(want * (1 - want) / n)


def test_verify_refused_and_bad_rows():
    bad = dg.DG_DEV_BAD_PARAM
    V = 100
    def one(change, tree=True, status=bad, T=0.8):
        d = Drafts([5, 6, 4], V, 9, T=T, tree=tree)
        change(d)
        d.run().check(status=status, skip=(1,))
        return d
    def refused(d):
        assert d.n_accept[1] == -1 and (d.path[5:11] == -1).all() and (d.out[5:11] == -1).all()
    for change in (lambda d: d.parents.__setitem__(7, 2), lambda d: d.parents.__setitem__(7, -1),
                   lambda d: d.parents.__setitem__(10, 10 ** 9), lambda d: d.T.__setitem__(1, -1.0),
                   lambda d: d.T.__setitem__(1, math.nan), lambda d: d.T.__setitem__(1, math.inf),
                   lambda d: d.T.__setitem__(1, 1e-30), lambda d: d.u.__setitem__(8, 1.0),
                   lambda d: d.u.__setitem__(10, -0.1), lambda d: d.un.__setitem__(1, math.nan)):
        refused(one(change))
    d = Drafts([5, 6, 4], V, 9, tree=False)
    d.cu[3] = 1000                          # a sequence that ends behind the rows
    d.run()
    assert dg.dg_get_device_status() == bad and d.n_accept[2] == -1 and (d.path[11:] == -9).all()
    # greedy requests do not read the random numbers
    d = Drafts([5, 6], V, 9, T=0.0, tree=True)
    d.u[:] = math.nan
    d.un[:] = 7.0
    d.run().check()
    # rows: bad ones count only on the walk
    for value, status in ((math.nan, dg.DG_DEV_NAN_INF_ROW), (math.inf, dg.DG_DEV_NAN_INF_ROW)):
        for T in (0.8, 0.0):
            d = one(lambda d: d.x[5].__setitem__(77, value), status=status, T=T)   # the root's row
            assert d.n_accept[1] == 0 and d.path[5:11].tolist() == [0] + [-1] * 5 and (d.out[5:11] == -1).all()
    d = one(lambda d: d.x[5, :V].fill_(-math.inf), status=dg.DG_DEV_EMPTY_ROW)
    assert d.n_accept[1] == 0 and (d.out[5:11] == -1).all()
    d = Drafts([3, 3], V, 2, T=1.0)
    d.tokens[1] = d.tokens[4] = -1          # both end at the root
    d.x[1:3] = math.nan
    d.x[4:] = math.nan
    d.run()
    assert dg.dg_get_device_status() == 0 and d.n_accept.tolist() == [0, 0]
    d = Drafts([1200, 3], 40, 2, tree=True)   # more nodes than a walk takes
    d.run()
    assert dg.dg_get_device_status() == bad and d.n_accept[0] == -1 and (d.path[:1200] == -1).all()
    dg.dg_clear_device_status()


# ------------------------------------------------------------------ kept paths
def _keep(seqs, layers, Hkv, D, page, paths, *, seed=0, head_major=False, bad=(), status=0, change=None):
    """seqs [(nodes, keys)]; paths: kept nodes of each sequence (None: n_accept -1)."""
    b = ref.Batch([(a, m, 1) for a, m in seqs], 1, Hkv, D, page, seed=seed, head_major=head_major, before=1, after=2)
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (layers, b.n_pages, Hkv, page, D) if head_major else (layers, b.n_pages, page, Hkv, D)
    make = lambda: torch.randn(shape, generator=g, device=DEV).to(ref.BF16)  # noqa: E731
    kc, vc = make(), make()
    if head_major:
        kc, vc = kc.transpose(2, 3), vc.transpose(2, 3)
    path, count, lens = [-3], [], []
    for (a, m), p in zip(seqs, paths):
        p = [] if p is None else p
        path += (p + [-1] * a)[:a] if a >= len(p) else p[:a]
        count.append(len(p) - 1)
    path += [-3] * 2
    args = dict(path=torch.tensor(path, **I32), count=torch.tensor(count, **I32))
    if change:
        change(b, args)
    want_k, want_v = kc.clone(), vc.clone()
    for s, ((a, m), p) in enumerate(zip(seqs, paths)):
        if p is None or s in bad:
            lens.append(m)
            continue
        lens.append(m - a + len(p))
        src, dst = b.slots(s, [m - a + x for x in p]), b.slots(s, range(m - a, m - a + len(p)))
        for want, old in ((want_k, kc), (want_v, vc)):
            want[:, dst[0], dst[1]] = old[:, src[0], src[1]]
    new_len = torch.full((len(seqs),), -9, **I32)
    dg.dg_clear_device_status()
    ck, cv = (kc, vc) if layers > 1 else (kc[0], vc[0])
    dg.dg_kv_keep(ck, cv, b.table, b.cu, b.kv_len, args["path"], args["count"], new_len)
    assert dg.dg_get_device_status() == status
    assert torch.equal(kc.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(vc.view(torch.int16), want_v.view(torch.int16))
    for s in bad:
        lens[s] = int(b.kv_len[s])
    assert new_len.tolist() == lens


@pytest.mark.parametrize("layers,Hkv,D,page,head_major", [(1, 1, 64, 8, False), (3, 2, 128, 16, True), (2, 8, 256, 64, False),
                                                          (5, 3, 64, 8, True)])
def test_keep(layers, Hkv, D, page, head_major):
    seqs = [(1, 1), (8, 30), (16, 16), (0, 9), (60, 300), (5, 70), (300, 333), (7, 7), (4, 4)]
    every = list(range(300))
    paths = [[0], [0, 2, 3, 7], [1, 2, 3, 4, 5, 15], None, [0, 1, 2, 10, 11, 12, 40, 59], [4], every[:1] + every[3::2], None,
             [0, 1, 2, 3]]
    _keep(seqs, layers, Hkv, D, page, paths, head_major=head_major, seed=layers)


def test_keep_long_and_many():
    _keep([(1000, 1010), (900, 2000)], 2, 1, 64, 16, [list(range(1, 1000)), list(range(0, 900, 3))])
    g = torch.Generator().manual_seed(0)
    paths = [sorted(torch.randperm(20, generator=g)[:1 + i % 9].tolist()) for i in range(700)]
    _keep([(20, 20 + i % 50) for i in range(700)], 1, 2, 64, 8, paths)


def test_keep_refused():
    bad = dg.DG_DEV_BAD_PARAM
    seqs, paths = [(8, 30), (8, 40), (8, 50)], [[0, 3, 5], [0, 2, 6], [1, 2, 7]]
    run = lambda change: _keep(seqs, 2, 2, 64, 16, paths, bad=(1,), status=bad, change=change)  # noqa: E731
    run(lambda b, a: a["path"].__setitem__(1 + 8 + 2, 2))       # twice the same
    run(lambda b, a: a["path"].__setitem__(1 + 8 + 2, 8))       # past the last node
    run(lambda b, a: a["path"].__setitem__(1 + 8, -1))
    run(lambda b, a: a["count"].__setitem__(1, 8))
    run(lambda b, a: a["count"].__setitem__(1, -2))
    run(lambda b, a: b.kv_len.__setitem__(1, 7))
    run(lambda b, a: b.kv_len.__setitem__(1, 10 ** 6))
    run(lambda b, a: b.table.__setitem__((1, 2), b.n_pages))    # nodes 0 .. 7 lie in slots 32 .. 39
    # a page that no moved node needs may be anything
    _keep(seqs, 1, 2, 64, 16, paths, change=lambda b, a: b.table.__setitem__((2, 0), -1))


# ------------------------------------------------------------------ the calls as they are used
def _pass(seed=1, n=5, D=128, Hq=8, Hkv=2, V=600, layers=2, page=16):
    """One drafting pass over random trees: its state, ready to be run."""
    g = torch.Generator().manual_seed(seed)
    sizes = [6 + 5 * i for i in range(n)]
    ctx = [10 + 37 * i for i in range(n)]
    seqs = [(a, a + c, 1) for a, c in zip(sizes, ctx)]
    b = ref.Batch(seqs, Hq, Hkv, D, page, seed=seed, fill=0.0).fill_keys()
    d = Drafts(sizes, V, seed, tree=True, near=0.9, std=1.5)
    d.u *= 0.02                             # most drafts are likely tokens: let them pass
    par = d.parents.tolist()
    sets, pos, at = [], [], 0
    for a, c in zip(sizes, ctx):
        depth, anc = [0], [{0}]
        for i in range(1, a):
            p = par[at + i]
            depth.append(depth[p] + 1)
            anc.append(anc[p] | {i})
        sets += anc
        pos += [c + x for x in depth]
        at += a
    s = dict(b=b, d=d, sizes=sizes, ctx=ctx, pos=torch.tensor(pos, **I32), mask=dref.words(sets, -(-max(sizes) // 32), DEV),
             sets=sets)
    rnd = lambda *shape: torch.randn(shape, generator=g).to(ref.BF16).to(DEV)  # noqa: E731
    s["qkv"] = [(rnd(b.total, Hq, D), rnd(b.total, Hkv, D), rnd(b.total, Hkv, D)) for _ in range(layers)]
    s["k"] = torch.stack([b.k_cache] * layers)
    s["v"] = torch.stack([b.v_cache] * layers)
    s["o"] = torch.zeros((layers, b.total, Hq, D), dtype=ref.BF16, device=DEV)
    s["q_out"] = torch.zeros((b.total, Hq, D), dtype=ref.BF16, device=DEV)
    s["norm"] = (torch.rand(D, generator=g) + 0.5).to(DEV), (torch.rand(D, generator=g) + 0.5).to(DEV)
    s["w"] = _inv_freq(D)
    s["ws"] = torch.zeros(max(16, dg.dg_tree_attention_workspace_bytes(n, max(sizes), Hq, Hkv, D)), dtype=torch.uint8, device=DEV)
    s["x"], s["tok"], s["T"], s["u"], s["un"], s["par"] = (t.to(DEV) for t in (d.x, d.tokens, d.T, d.u, d.un, d.parents))
    s["count"], s["path"], s["out"], s["new_len"] = (torch.zeros(k, **I32) for k in (n, b.total, b.total, n))
    return s


def _step(s, stream=None, verify=True):
    b = s["b"]
    for layer, (q, k, v) in enumerate(s["qkv"]):
        dg.dg_kv_append_norm(k, v, s["k"][layer], s["v"][layer], b.table, b.cu, b.kv_len, inv_freq=s["w"], q=q,
                             q_out=s["q_out"], q_norm=s["norm"][0], k_norm=s["norm"][1], positions=s["pos"], stream=stream)
        dg.dg_tree_attention(s["q_out"], s["k"][layer], s["v"][layer], s["o"][layer], b.table, b.cu, b.kv_len, s["mask"],
                             max(s["sizes"]), workspace=s["ws"], stream=stream)
    if verify:
        dg.dg_verify_drafts(s["x"], s["tok"], b.cu, s["T"], s["u"], s["un"], s["count"], s["path"], s["out"],
                            parents=s["par"], V=s["d"].V, stream=stream)
        dg.dg_kv_keep(s["k"], s["v"], b.table, b.cu, b.kv_len, s["path"], s["count"], s["new_len"], stream=stream)


def test_a_drafting_pass():
    """Append, attend, verify, keep: the cache is then what appending the accepted tokens one after another makes it, and
    the accepted nodes' outputs are those of causal attention over it."""
    s = _pass()
    b, n = s["b"], len(s["sizes"])
    k0, v0 = s["k"].clone(), s["v"].clone()
    _step(s)
    torch.cuda.synchronize()
    cu, count, path = b.cu.tolist(), s["count"].tolist(), s["path"].tolist()
    assert sum(count) > 3 and s["new_len"].tolist() == [c + a + 1 for c, a in zip(s["ctx"], count)]
    rows = [cu[i] + path[cu[i] + j] for i in range(n) for j in range(count[i] + 1)]
    cu2 = torch.tensor([0] + torch.tensor([a + 1 for a in count]).cumsum(0).tolist(), **I32)
    for layer, (q, k, v) in enumerate(s["qkv"]):
        q2 = torch.zeros((len(rows), *q.shape[1:]), dtype=ref.BF16, device=DEV)
        kc, vc = k0[layer].clone(), v0[layer].clone()
        dg.dg_kv_append_norm(k[rows].contiguous(), v[rows].contiguous(), kc, vc, b.table, cu2, s["new_len"], inv_freq=s["w"],
                             q=q[rows].contiguous(), q_out=q2, q_norm=s["norm"][0], k_norm=s["norm"][1])
        for i in range(n):
            at = b.slots(i, range(s["ctx"][i] + count[i] + 1))
            assert torch.equal(kc[at], s["k"][layer][at]) and torch.equal(vc[at], s["v"][layer][at])
        o2, lse = torch.zeros_like(q2), torch.zeros(q2.shape[:2], device=DEV)
        dg.dg_paged_attention(q2, kc, vc, o2, b.table, cu2, s["new_len"], torch.ones(n, dtype=torch.uint8, device=DEV),
                              max(count) + 1, lse=lse)
        b2 = b
        for i in range(n):
            m, a = s["ctx"][i] + count[i] + 1, count[i] + 1
            at = b2.slots(i, range(m))
            sel = slice(int(cu2[i]), int(cu2[i + 1]))
            ro, _, bound, _ = dref.attention(q2[sel], kc[at], vc[at], dref.visible(a, m).to(DEV), 1 / math.sqrt(b.D))
            got = s["o"][layer][rows][sel]
            assert ((got.double() - ro).abs() <= bound).all() and ((o2[sel].double() - ro).abs() <= bound).all()


def test_a_pass_in_a_graph_and_on_streams():
    """Captured and replayed, on another stream, and beside another pass: bit for bit what one call after another gives."""
    a, ref_a = _pass(2), _pass(2)
    _step(ref_a)
    torch.cuda.synchronize()
    same = ("o", "k", "v", "count", "path", "out", "new_len", "q_out")
    k0, v0 = a["k"].clone(), a["v"].clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    _step(a, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a[x], ref_a[x]) for x in same)
    a["k"].copy_(k0), a["v"].copy_(v0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(a)
    for _ in range(3):
        a["k"].copy_(k0), a["v"].copy_(v0)
        for x in ("o", "count", "path", "out", "new_len"):
            a[x].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a[x], ref_a[x]) for x in same)
    # two passes at once, each with its own workspace
    c, ref_c = _pass(3, n=7), _pass(3, n=7)
    _step(ref_c)
    a["k"].copy_(k0), a["v"].copy_(v0)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        _step(a, stream=s1, verify=False)
        _step(c, stream=s2, verify=False)
    _step(a, stream=s1)
    _step(c, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(a[x], ref_a[x]) for x in same) and all(torch.equal(c[x], ref_c[x]) for x in same)
