"""GPU tests of dg_paged_attention's query tiles in the ways they run: with no more items than CTAs every CTA finds
its item by itself (one kernel); with more, a plan kernel lists them (two), to be taken round robin where they
all cost the same and from a counter where they do not, several by each CTA.  An item is 128 queries of a sequence
and a query head; the CTAs are two an SM for heads of 64 and 128, one for heads of 256."""
import math

import pytest
import torch

import entropy_bounded_denoising_gb300 as dg

import serving_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAD = dg.DG_DEV_BAD_PARAM
H = 8

# (queries, keys, causal); the longest has 257 queries: three tiles
FEW = [(130, 200, 1), (140, 500, 0), (1, 1, 1), (257, 300, 0), (131, 0, 1)]
RAGGED = [(130, 200, 1), (140, 500, 0), (1, 1, 1), (133, 133, 1), (0, 40, 0), (257, 300, 0), (131, 0, 1), (257, 900, 1),
          (5, 700, 0), (256, 256, 1)] * 5
EQUAL = [(257, 400, 0)] * 45
WAYS = {"by itself": FEW, "counter": RAGGED, "round robin": EQUAL}
ways = pytest.mark.parametrize("way", list(WAYS))
heads = pytest.mark.parametrize("D", [64, 128, 256])


def _batch(way, D, seqs=None, **kw):
    seqs = WAYS[way] if seqs is None else seqs
    return ref.Batch(seqs, H, H, D, 16, seed=D + len(seqs), before=1, after=2, **kw).fill_keys()


def _items(b, max_q):
    return len(b.seqs) * -(-max_q // 128) * b.Hq


def _attend(b, way, window=-1, scale=None, max_q=257, workspace=None, stream=None):
    """The call, and that it went its way."""
    o = torch.full(b.q.shape, 7.0, dtype=ref.BF16, device=DEV)
    lse = torch.full(b.q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (_items(b, max_q) > sms * (1 if b.D == 256 else 2)) == (way != "by itself")
    launches = dg.dg_launch_count()
    dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, max_q, lse=lse, window=window,
                          scale=scale, workspace=workspace, stream=stream)
    assert dg.dg_launch_count() - launches == (1 if way == "by itself" else 2)
    return o, lse


def _checked(b, way, window=-1, scale=None, status=0, skip=(), max_q=257):
    dg.dg_clear_device_status()
    o, lse = _attend(b, way, window, scale, max_q)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == status
    dg.dg_clear_device_status()
    ref.check_attention(b, o, lse, window, scale, sentinel=7.0, skip=skip)
    return o, lse


@ways
@heads
def test_scales_and_windows(D, way):
    b = _batch(way, D)
    for scale in (None, 0.0, -0.1, 1.0):
        _checked(b, way, scale=scale)
    for window in (0, 1, 100):
        _checked(b, way, window)


@ways
@heads
def test_refused_sequences(D, way):
    """Lengths and offsets out of range, a page outside the pool, more queries than the call says: reported, and
    the other sequences are right."""
    n = len(WAYS[way])
    b = _batch(way, D)
    b.kv_len[1] = b.seqs[1][0] - 1
    b.kv_len[n - 2] = -5
    _checked(b, way, status=BAD, skip=(1, n - 2))
    b = _batch(way, D, extra_columns=0)
    b.kv_len[1] = b.table.shape[1] * 16 + 1
    _checked(b, way, status=BAD, skip=(1,))
    b = _batch(way, D)
    b.cu[n] = b.total + 1
    b.cu[n - 1] = 3
    _checked(b, way, status=BAD, skip=(n - 1, n - 2))
    for page in (-1, b.n_pages, 2 ** 31 - 1):
        b = _batch(way, D)
        b.table[1, 7] = page
        dg.dg_clear_device_status()
        o, lse = _attend(b, way)
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == BAD
        ref.check_attention(b, o, lse, skip=(1,))
    b = _batch(way, D)
    dg.dg_clear_device_status()
    o, lse = _attend(b, way, max_q=256 if way == "by itself" else 200)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == BAD
    long = [s for s, (a, _, _) in enumerate(b.seqs) if a > 200]
    ref.check_attention(b, o, lse, skip=long)
    for s in long[:2]:                        # their first rows are there
        rows = slice(int(b.cu[s]), int(b.cu[s]) + 200)
        ro, _, bound, _ = ref.attention(b.q[int(b.cu[s]):int(b.cu[s + 1])], *b.keys(s), b.seqs[s][2], -1, D ** -0.5)
        assert ((o[rows].double() - ro[:200]).abs() <= bound[:200]).all()
    dg.dg_clear_device_status()


@ways
@heads
def test_nothing_but_sequences_without_keys(D, way):
    _checked(_batch(way, D, [(257, 0, 1)] * (3 if way == "by itself" else 45)), way)
    _checked(_batch(way, D, [(0, 50, 1)] * (3 if way == "by itself" else 45) + [(1, 0, 0)]), way)


@ways
@heads
@pytest.mark.parametrize("page", [8, 32, 128])
def test_slots_that_no_query_sees_hide(D, way, page):
    """Slots before the window, and stale ones past kv_len, hold NaN; table entries of dropped pages are invalid."""
    n = 4 if way == "by itself" else 50
    seqs = [(257, 1000 if way == "round robin" else 600 + 37 * (i % 11), i % 2) for i in range(n)]
    b = ref.Batch(seqs, H, H, D, page, seed=page).fill_keys()
    want, lse = _checked(b, way, 90)
    for s, (a, kl, _) in enumerate(b.seqs):
        gone = b.slots(s, range(kl - a - 90))
        b.k_cache[gone] = math.nan
        b.v_cache[gone] = math.nan
        b.table[s, :(kl - a - 90) // page] = -3
    dg.dg_clear_device_status()
    o, l = _attend(b, way, 90)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == 0 and torch.equal(o, want) and torch.equal(l, lse)


@ways
@heads
def test_nan_stays_where_it_belongs(D, way):
    """A query of NaN shows in its row and head alone, NaN keys and infinite values in their head's."""
    b = _batch(way, D)
    o0, l0 = _checked(b, way)
    s, bad = 1, 5
    row = int(b.cu[s]) + 3
    at = b.slots(s, [0, b.seqs[s][1] // 2])
    q, k, v = b.q[row, 2].clone(), b.k_cache[at], b.v_cache[at]     # to be put back
    b.q[row, 2] = math.nan
    b.k_cache[at[0], at[1], bad] = math.nan
    b.v_cache[at[0], at[1], bad] = math.inf
    o, lse = _attend(b, way)
    assert torch.isnan(o[row, 2]).all() and torch.isnan(lse[row, 2])
    mine = slice(int(b.cu[s]), int(b.cu[s + 1]))
    assert not torch.isfinite(o[mine, bad]).any() and torch.isnan(lse[mine, bad]).all()
    b.q[row, 2], b.k_cache[at], b.v_cache[at] = q, k, v
    o[row, 2], lse[row, 2], o[mine, bad], lse[mine, bad] = o0[row, 2], l0[row, 2], o0[mine, bad], l0[mine, bad]
    ref.check_attention(b, o, lse, sentinel=7.0)


@ways
@heads
def test_repeats_streams_and_workspaces(D, way):
    """The same bits again, whatever the workspace held, and from two calls at once on two streams."""
    bs = [_batch(way, D), _batch(way, D, list(reversed(WAYS[way])))]
    want = [_checked(b, way) for b in bs]
    need = dg.dg_paged_attention_workspace_bytes(len(bs[0].seqs), 257, H, H, D)
    for byte in (0, 255, 127):
        ws = torch.full((need,), byte, dtype=torch.uint8, device=DEV)
        for b, (o0, l0) in zip(bs, want):
            o, lse = _attend(b, way, workspace=ws)
            assert torch.equal(o, o0) and torch.equal(lse, l0)
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(4):
        torch.cuda.synchronize()
        got = [_attend(b, way, stream=st) for b, st in zip(bs, streams)]
        torch.cuda.synchronize()
        for (o, l), (o0, l0) in zip(got, want):
            assert torch.equal(o, o0) and torch.equal(l, l0)


@ways
@heads
def test_graphs_that_share_a_workspace(D, way):
    """Two captured calls on one workspace, replayed in turn and after their lengths changed."""
    bs = [_batch(way, D), _batch(way, D, list(reversed(WAYS[way])))]
    ws = torch.empty(dg.dg_paged_attention_workspace_bytes(len(bs[0].seqs), 257, H, H, D), dtype=torch.uint8, device=DEV)
    outs, graphs = [], []
    for b in bs:
        _attend(b, way, workspace=ws)
        torch.cuda.synchronize()
        o, lse = torch.full(b.q.shape, 7.0, dtype=ref.BF16, device=DEV), torch.full(b.q.shape[:2], 7.0, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, 257, lse=lse, workspace=ws)
        outs.append((o, lse))
        graphs.append(g)
    dg.dg_clear_device_status()
    for turn in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b, (o, lse) in zip(bs, outs):
            ref.check_attention(b, o, lse, sentinel=7.0)
            # other lengths: an empty slot becomes a sequence of its queries' keys, others lose some, or all
            b.seqs = [(a, kl if turn == 1 or s % 3 == 1 else 0 if s % 3 == 2 else a, c) for s, (a, kl, c) in enumerate(b.seqs)]
            b.kv_len.copy_(torch.tensor([kl for _, kl, _ in b.seqs], dtype=torch.int32))
            for s, (a, kl, _) in enumerate(b.seqs):    # pages for a slot that had none: a full one of another's
                used = -(-kl // b.page_size)
                assert used <= b.table.shape[1]
                b.table[s, :used] = torch.where(b.table[s, :used] < 0, b.table[1, 0], b.table[s, :used])
    assert dg.dg_get_device_status() == 0


@pytest.mark.parametrize("D,Hq,Hkv,n", [(64, 4, 2, 1), (64, 16, 8, 1), (128, 4, 2, 1), (128, 16, 8, 1), (256, 4, 1, 1), (256, 8, 8, 2)])
def test_causal_prompts_of_thousands_of_rows(D, Hq, Hkv, n):
    """Prompts after some context: one of 2500 rows, and two at once."""
    b = ref.Batch([(2500 - 400 * i, 2611 + 300 * i, 1) for i in range(n)], Hq, Hkv, D, 64, seed=D, after=1).fill_keys()
    for window in (-1, 700):
        o, lse = torch.full(b.q.shape, 7.0, dtype=ref.BF16, device=DEV), torch.full(b.q.shape[:2], 7.0, device=DEV)
        dg.dg_clear_device_status()
        dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, 2500, lse=lse, window=window)
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == 0
        ref.check_attention(b, o, lse, window, sentinel=7.0)
