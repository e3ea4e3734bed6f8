"""GPU parity of the paged cache's calls (dg_kv_append, dg_paged_attention) against their fp64 forms.

Append: |got - ref| <= 2^-8 |ref| (one rounding to bf16) + 2^-21 (|a| + |b|) (fp32 sines, cosines and
rotation); values, unrotated dimensions and every slot that is not appended bit for bit.
Attention: see serving_ref.attention; rows of no sequence, and of refused ones, bit for bit."""
import math

import pytest
import torch

import entropy_bounded_denoising_gb300 as dg

import serving_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inv_freq(rot, theta=10000.0):
    return theta ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=DEV) / rot)


# ------------------------------------------------------------------ append
def _append(b, rot, interleaved, *, fused=True, in_place=False, with_q=True, w=None, status=0, skip=()):
    """Append a random pass to batch b and compare everything it may and may not write."""
    g = torch.Generator(device=DEV).manual_seed(b.total + rot)
    w = _inv_freq(rot) if w is None and rot else w
    width = (b.Hq + 2 * b.Hkv) * b.D
    qkv = torch.randn((b.total, width), generator=g, device=DEV).to(ref.BF16)
    cut = lambda lo, h: qkv[:, lo * b.D:(lo + h) * b.D].unflatten(1, (h, b.D))  # noqa: E731
    q, k, v = cut(0, b.Hq), cut(b.Hq, b.Hkv), cut(b.Hq + b.Hkv, b.Hkv)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q0 = q.clone()
    for c in (b.k_cache, b.v_cache):
        c.copy_(torch.randn(c.shape, generator=g, device=DEV).to(ref.BF16))
    kc0, vc0 = b.k_cache.clone(), b.v_cache.clone()
    q_out = q if in_place else torch.full((b.total, b.Hq, b.D), 7.0, dtype=ref.BF16, device=DEV)
    dg.dg_clear_device_status()
    dg.dg_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cu, b.kv_len, inv_freq=w, interleaved=interleaved,
                    q=q if with_q else None, q_out=q_out if with_q else None)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == status
    w = torch.zeros(0, dtype=torch.float64, device=DEV) if w is None else w
    kc, vc = kc0.double(), vc0.clone()
    slack = torch.zeros_like(kc)
    qr = q0.double() if in_place else torch.full(q0.shape, 7.0, dtype=torch.float64, device=DEV)
    q_slack = torch.zeros_like(qr)
    cu = b.cu.tolist()
    for s, (a, kl, _) in enumerate(b.seqs):
        if a == 0 or kl == 0 or s in skip:
            continue
        rows = slice(cu[s], cu[s + 1])
        p = torch.arange(kl - a, kl, device=DEV)
        at = b.slots(s, p)
        kc[at] = ref.rotate(k[rows].double(), p, w, interleaved)
        slack[at] = ref.rotation_bound(k[rows].double(), w, interleaved)
        vc[at] = v[rows]
        qr[rows] = ref.rotate(q0[rows].double(), p, w, interleaved)
        q_slack[rows] = ref.rotation_bound(q0[rows].double(), w, interleaved)
    assert torch.equal(b.v_cache.view(torch.int16), vc.view(torch.int16))

    def near(got, want, slack):
        turned = slack > 0
        assert torch.equal(got.double()[~turned], want[~turned])
        err = (got.double() - want).abs()
        assert (err <= 2.0 ** -8 * want.abs() + slack)[turned].all(), float(err.max())

    near(b.k_cache, kc, slack)
    if with_q:
        near(q_out, qr, q_slack)
    else:
        assert (q_out == 7.0).all()


SEQS = [(1, 1, 1), (0, 40, 1), (1, 300, 1), (17, 33, 0), (0, 0, 1), (2, 0, 1), (64, 64, 1), (256, 300, 0), (3, 129, 1)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,page,Hq,Hkv,head_major", [(64, 64, 8, 1, 1, False), (64, 16, 16, 7, 1, True),
                                                          (128, 128, 16, 16, 8, False), (128, 64, 64, 5, 5, True),
                                                          (256, 256, 32, 4, 2, False), (256, 48, 128, 24, 3, True)])
def test_append(D, rot, page, Hq, Hkv, head_major, interleaved):
    b = ref.Batch(SEQS, Hq, Hkv, D, page, seed=D + rot, head_major=head_major, before=3, after=5)
    _append(b, rot, interleaved)


def test_append_variants():
    make = lambda seqs=SEQS, **kw: ref.Batch(seqs, 4, 2, 128, 16, seed=9, **kw)  # noqa: E731
    _append(make(), 128, False, fused=False, in_place=True)
    _append(make(after=2), 0, False)                         # no rotation: copies
    _append(make(), 128, True, with_q=False)
    _append(make([(1, 77, 1)]), 128, False)                  # one token
    _append(make([(1, 1 + i, 1) for i in range(1500)]), 128, False)   # more sequences than a search round
    _append(make([(0, 5, 1)] * 70 + [(2, 9, 1)] + [(0, 0, 1)] * 1100 + [(1, 4, 1)], after=1), 64, False)
    # frequencies of more than a turn, of either sign, and none
    w = torch.tensor([0.0, -1.0, 7.5, 100.0, 1e-9, 3.0, -0.25, 6.283185307179586], dtype=torch.float64, device=DEV)
    _append(make(), 16, True, w=w)
    # value and key rows that are parts of wider rows of their own
    b = make()
    _append(b, 128, False, fused=True)


def test_append_far_positions():
    """Positions near 2^31: the angle's reduction is exact, so the bound is that of near positions.  The
    reference reduces position * frequency modulo a turn in integers."""
    D, page, far = 64, 65536, (1 << 31) - 3
    cols = far // page + 1
    table = torch.full((1, cols), -1, dtype=torch.int32, device=DEV)
    table[0, (far - 5) // page:] = 0
    cache = [torch.zeros((1, page, 1, D), dtype=ref.BF16, device=DEV) for _ in range(2)]
    g = torch.Generator(device=DEV).manual_seed(3)
    k = torch.randn((5, 1, D), generator=g, device=DEV).to(ref.BF16)
    # frequencies that are whole numbers of 2^-40 turns: exact in double, with exact angles
    turns = [(3 ** j * 1234567) % (1 << 40) for j in range(D // 2)]
    w = torch.tensor([t / 2.0 ** 40 * 2 * math.pi for t in turns], dtype=torch.float64, device=DEV)
    dg.dg_clear_device_status()
    dg.dg_kv_append(k, k, *cache, table, torch.tensor([0, 5], dtype=torch.int32, device=DEV),
                    torch.tensor([far], dtype=torch.int32, device=DEV), inv_freq=w)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == 0
    for i in range(5):
        p = far - 5 + i
        ang = torch.tensor([(p * t % (1 << 40)) / 2.0 ** 40 * 2 * math.pi for t in turns], dtype=torch.float64, device=DEV)
        want = ref.rotate(k[i:i + 1].double(), torch.ones(1, device=DEV), ang, False)[0, 0]
        got = cache[0][0, p % page, 0].double()
        # w / 2 pi carries 2^-52 relative (two roundings in double): p 2^-52 turns on the way here
        slack = ref.rotation_bound(k[i:i + 1].double(), ang, False)[0, 0] * (1 + 2 * math.pi * p * 2.0 ** -52 * 2.0 ** 21)
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + slack).all(), i


def test_append_leaves_refused_sequences_out():
    bad = dg.DG_DEV_BAD_PARAM
    # fewer keys than queries; more keys than the table holds; a page outside the pool
    b = ref.Batch([(4, 20, 1), (5, 16, 1), (3, 30, 1)], 2, 1, 64, 16, seed=2)
    b.kv_len[1] = 4
    _append(b, 64, False, status=bad, skip=(1,))
    b = ref.Batch([(4, 20, 1), (5, 16, 1), (3, 30, 1)], 2, 1, 64, 16, seed=2, extra_columns=0)
    b.kv_len[2] = 33
    _append(b, 64, False, status=bad, skip=(2,))
    for page in (-1, b.n_pages, 2 ** 31 - 1):
        b = ref.Batch([(4, 20, 1), (5, 16, 1), (3, 30, 1)], 2, 1, 64, 16, seed=2)
        b.table[1, 0] = page
        _append(b, 64, False, status=bad, skip=(1,))
    # offsets outside the rows
    b = ref.Batch([(4, 20, 1), (5, 16, 1), (3, 30, 1)], 2, 1, 64, 16, seed=2)
    b.cu[3] = b.total + 1
    _append(b, 64, False, status=bad, skip=(2,))
    dg.dg_clear_device_status()


def test_append_past_32_bit_offsets():
    """A cache of more than 2^32 bytes and 2^31 elements: the last page."""
    D, Hkv, page = 128, 8, 64
    n_pages = (1 << 31) // (D * Hkv * page) + 2
    kc = torch.zeros((n_pages, page, Hkv, D), dtype=ref.BF16, device=DEV)
    vc = torch.zeros_like(kc)
    k = torch.randn((1, Hkv, D), device=DEV).to(ref.BF16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    dg.dg_kv_append(k, k, kc, vc, i32(n_pages - 1)[None], i32(0, 1), i32(64))
    torch.cuda.synchronize()
    for c in (kc, vc):
        assert torch.equal(c[n_pages - 1, 63], k[0])
        c[n_pages - 1, 63] = 0
        assert not c.any()


# ------------------------------------------------------------------ attention
def _attend(b, window=-1, scale=None, *, max_q=None, status=0, skip=(), lse=True, **kw):
    o = torch.full(b.q.shape, 7.0, dtype=ref.BF16, device=DEV)
    l = torch.full(b.q.shape[:2], 7.0, dtype=torch.float32, device=DEV) if lse else None
    dg.dg_clear_device_status()
    mq = max([1] + [s[0] for s in b.seqs]) if max_q is None else max_q
    dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, mq, lse=l, window=window,
                          scale=scale, **kw)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == status
    ref.check_attention(b, o, l, window, scale, sentinel=7.0, skip=skip)
    return o, l


TOKENS = [(1, 1, 1), (1, 7, 1), (1, 64, 0), (1, 65, 1), (0, 50, 1), (1, 0, 1), (1, 1000, 1), (1, 129, 0), (0, 0, 0)]
DRAFTS = [(5, 5, 1), (1, 33, 1), (4, 200, 1), (3, 0, 1), (5, 1023, 1), (2, 2, 0), (5, 77, 0)]
MIXED = [(300, 300, 1), (256, 700, 0), (256, 700, 1), (5, 5, 1), (17, 40, 0), (3, 0, 0), (128, 128, 0), (1, 600, 1)]


@pytest.mark.parametrize("window", [-1, 0, 1, 100])
@pytest.mark.parametrize("seqs", [TOKENS, DRAFTS, MIXED], ids=["tokens", "drafts", "mixed"])
@pytest.mark.parametrize("D,page,Hq,Hkv,head_major", [(64, 8, 8, 8, True), (128, 16, 16, 8, False), (128, 64, 6, 2, True),
                                                      (256, 32, 7, 1, False), (256, 128, 16, 4, True)])
def test_attention(D, page, Hq, Hkv, head_major, seqs, window):
    b = ref.Batch(seqs, Hq, Hkv, D, page, seed=D + len(seqs) + window, head_major=head_major, before=2, after=3).fill_keys()
    _attend(b, window)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (9, 1), (17, 1), (40, 1), (71, 1), (64, 2)])
def test_attention_head_groups(Hq, Hkv):
    b = ref.Batch([(1, 150, 1), (2, 90, 1)], Hq, Hkv, 64, 16, seed=Hq, after=1).fill_keys()
    _attend(b)
    _attend(b, lse=False)


@pytest.mark.parametrize("D,q_len,kv", [(64, 1, 30011), (128, 1, 100003), (256, 3, 20000), (128, 256, 5000)])
def test_attention_long(D, q_len, kv):
    """One long context: split over its length and joined; with a window the first pages drop out."""
    b = ref.Batch([(q_len, kv, 1)], 4, 2, D, 64, seed=kv, after=1).fill_keys()
    _attend(b)
    _attend(b, 4000)
    b.table[0, :(kv - q_len - 4000) // 64] = -1     # pages that no query sees may be gone
    o = torch.zeros_like(b.q)
    dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, q_len, window=4000)
    assert dg.dg_get_device_status() == 0 and torch.isfinite(o).all() and o[:q_len].abs().sum() > 0


def test_attention_many_sequences():
    seqs = [(1, (37 * i) % 200, 1) for i in range(700)]
    _attend(ref.Batch(seqs, 2, 1, 64, 16, seed=5, after=1).fill_keys())


def test_attention_scores_of_any_size():
    """Scales that make one key win, all keys alike (scale 0) and the least similar win (negative);
    keys with infinities give no NaN where their scores are -inf."""
    b = ref.Batch([(1, 500, 1), (4, 90, 1), (200, 200, 0)], 4, 2, 128, 16, seed=8).fill_keys()
    for scale in (0.0, -0.1, 1.0, 3.0):
        _attend(b, scale=scale)
    b = ref.Batch([(1, 500, 1), (4, 90, 1)], 4, 2, 128, 16, seed=8).fill_keys()
    b.q.abs_().clamp_(min=0.01)
    for s, gone in ((0, [0, 3, 250, 499]), (1, [0, 1, 80])):
        b.k_cache[b.slots(s, gone)] = -math.inf
    _attend(b)


def test_attention_refused_sequences_and_rows():
    bad = dg.DG_DEV_BAD_PARAM
    for q in (1, 5, 40):
        seqs = [(q, 200, 1), (q, 100, 1), (q, 300, 1)]
        b = ref.Batch(seqs, 2, 1, 64, 16, seed=2).fill_keys()
        if q > 1:
            b.kv_len[1] = q - 1
            _attend(b, status=bad, skip=(1,))
        b = ref.Batch(seqs, 2, 1, 64, 16, seed=2, extra_columns=0).fill_keys()
        b.kv_len[2] = 305
        _attend(b, status=bad, skip=(2,))
        b = ref.Batch(seqs, 2, 1, 64, 16, seed=2).fill_keys()
        b.kv_len[0] = -1
        _attend(b, status=bad, skip=(0,))
        b = ref.Batch(seqs, 2, 1, 64, 16, seed=2).fill_keys()
        b.cu[3] = b.total + 1
        _attend(b, status=bad, skip=(2,))
        # a page outside the pool: reported, the other sequences are right
        for page in (-1, 1 << 30):
            b = ref.Batch(seqs, 2, 1, 64, 16, seed=2).fill_keys()
            b.table[1, 3] = page
            o = torch.zeros_like(b.q)
            dg.dg_clear_device_status()
            dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, q)
            torch.cuda.synchronize()
            assert dg.dg_get_device_status() == bad
            ref.check_attention(b, o, None, skip=(1,))
    # more queries than the call says: reported, the first ones are right
    b = ref.Batch([(9, 200, 1)], 2, 1, 64, 16, seed=2).fill_keys()
    o = torch.zeros_like(b.q)
    dg.dg_clear_device_status()
    dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, 4)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == bad
    k, v = b.keys(0)
    ro, _, bound, _ = ref.attention(b.q, k, v, True, -1, 1 / 8)
    assert ((o.double() - ro).abs() <= bound)[:4].all()
    dg.dg_clear_device_status()


def _tiles(D, seqs=None, **kw):
    """A batch of many rows a key head, which takes the query tiles."""
    seqs = [(130, 200, 1), (140, 500, 0), (1, 1, 1), (133, 133, 1), (0, 40, 0), (257, 300, 0), (131, 0, 1)] if seqs is None else seqs
    return ref.Batch(seqs, 8, 8, D, 16, seed=D + len(seqs), before=1, after=2, **kw).fill_keys()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_tiles_scales_and_refusals(D):
    """The query tiles with every sign of the scale, with refused sequences, a page outside the pool, more
    queries than the call says, and nothing but sequences without keys."""
    bad = dg.DG_DEV_BAD_PARAM
    b = _tiles(D)
    for scale in (None, 0.0, -0.1, 1.0):
        _attend(b, scale=scale)
    b = _tiles(D)
    b.kv_len[1] = 139
    _attend(b, status=bad, skip=(1,))
    b = _tiles(D, extra_columns=0)
    b.kv_len[1] = 32 * 16 + 1
    _attend(b, status=bad, skip=(1,))
    b = _tiles(D)
    b.kv_len[3] = -5
    b.cu[7] = b.total + 1
    b.cu[6] = 3
    _attend(b, status=bad, skip=(3, 5, 6))
    for page in (-1, b.n_pages, 2 ** 31 - 1):
        b = _tiles(D)
        b.table[1, 7] = page
        o = torch.full(b.q.shape, 7.0, dtype=ref.BF16, device=DEV)
        dg.dg_clear_device_status()
        dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, 257)
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == bad
        ref.check_attention(b, o, None, skip=(1,))
    b = _tiles(D)
    dg.dg_clear_device_status()
    o = torch.zeros_like(b.q)
    dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, 256)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == bad
    ref.check_attention(b, o, None, skip=(5,))
    b = _tiles(D, [(200, 0, 1)] * 6)
    _attend(b)


def test_attention_tiles_hide_what_no_query_sees():
    """Slots of a sequence before its window, and its own stale slots past kv_len, hold NaN: windows that end
    inside a page and a tile, page sizes below and above the tile's, table entries of dropped pages invalid."""
    for page in (8, 32, 128):
        b = ref.Batch([(150, 1000, c) for c in (0, 1, 0, 1, 1, 0)], 8, 8, 128, page, seed=page).fill_keys()
        want, lse = _attend(b, 90)
        for s, (a, kl, _) in enumerate(b.seqs):
            first = kl - a - 90
            gone = b.slots(s, range(first))
            b.k_cache[gone] = math.nan
            b.v_cache[gone] = math.nan
            b.table[s, :first // page] = -3
        o = torch.empty_like(want)
        dg.dg_clear_device_status()
        dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, 150, window=90)
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == 0 and torch.equal(o, want)


def test_attention_thousands_of_sequences():
    """More sequences than a block reads at once, most of them empty or short."""
    seqs = [(1, (7 * i) % 40, 1) if i % 3 else (0, 9, 1) for i in range(3000)]
    b = ref.Batch(seqs, 2, 1, 64, 8, seed=6, after=1).fill_keys()
    o = torch.full(b.q.shape, 7.0, dtype=ref.BF16, device=DEV)
    dg.dg_clear_device_status()
    dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, 1)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == 0
    pick = set(range(0, 3000, 37)) | {0, 1, 2, 2998, 2999}
    ref.check_attention(b, o, None, skip=[s for s in range(3000) if s not in pick])


def test_offsets_out_of_order_are_refused():
    """Offsets that go back: the rows they claim are left alone or belong to a sound sequence; nothing outside
    the tables is read."""
    b = ref.Batch([(4, 20, 1), (5, 16, 1), (3, 30, 1)], 2, 1, 64, 16, seed=2, extra_columns=0).fill_keys()
    for cu in ([0, 9, 4, 12], [0, -5, 9, 12], [5, 4, 3, 2], [0, 2 ** 31 - 1, 9, 12], [-7, 4, 9, 12]):
        b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        q, o = b.q.clone(), torch.zeros_like(b.q)
        dg.dg_clear_device_status()
        dg.dg_kv_append(q[:, :1].contiguous(), q[:, 1:].contiguous(), b.k_cache.clone(), b.v_cache.clone(), b.table, b.cu,
                        b.kv_len, inv_freq=_inv_freq(64), q=q, q_out=o)
        dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, 5)
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == dg.DG_DEV_BAD_PARAM
    dg.dg_clear_device_status()


def test_longest_sequences():
    """Sequences at the limit of kv_len, of which a window shows the last two pages: appended to and read by
    either path; one key more is refused by the attention."""
    last, page, D, H, W = (1 << 31) - (1 << 16), 65536, 64, 8, 100
    for rows in (1, 640):
        b = ref.Batch([(rows, rows + W, 1)], H, H, D, 1024, seed=rows)
        kc, vc = (torch.zeros((2, page, H, D), dtype=ref.BF16, device=DEV) for _ in range(2))
        table = torch.full((1, last // page + 1), -1, dtype=torch.int32, device=DEV)
        table[0, last // page - 2:last // page] = torch.tensor([0, 1])
        g = torch.Generator(device=DEV).manual_seed(rows)
        k, v = (torch.randn((rows + W, H, D), generator=g, device=DEV).to(ref.BF16) for _ in range(2))
        cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        cu_all = torch.tensor([0, rows + W], dtype=torch.int32, device=DEV)
        causal = torch.ones(1, dtype=torch.uint8, device=DEV)
        for kl, status in ((last, 0), (last + 1, dg.DG_DEV_BAD_PARAM)):
            kv_len = torch.tensor([kl], dtype=torch.int32, device=DEV)
            o, lse = torch.full((rows, H, D), 7.0, dtype=ref.BF16, device=DEV), torch.full((rows, H), 7.0, device=DEV)
            dg.dg_clear_device_status()
            if not status:
                dg.dg_kv_append(k, v, kc, vc, table, cu_all, kv_len)
            dg.dg_paged_attention(b.q, kc, vc, o, table, cu, kv_len, causal, rows, lse=lse, window=W)
            torch.cuda.synchronize()
            assert dg.dg_get_device_status() == status
            if status:
                assert (o == 7.0).all() and (lse == 7.0).all()
                continue
            assert torch.equal(kc[1, -(rows + W):], k) and torch.equal(vc[1, -(rows + W):], v)
            ro, rl, bound, lbound = ref.attention(b.q, k, v, True, W, 1 / 8)
            assert ((o.double() - ro).abs() <= bound).all() and ((lse.double() - rl).abs() <= lbound).all()
    dg.dg_clear_device_status()


@pytest.mark.parametrize("rows", [1, 640])
def test_attention_past_32_bit_offsets(rows):
    """The last pages of a cache of more than 2^32 bytes and 2^31 elements, by either path."""
    D, H, page = 64, 8, 64
    n_pages = (1 << 31) // (D * H * page) + 16
    small = ref.Batch([(rows, 700, 1)], H, H, D, page, seed=1, extra_columns=0).fill_keys()
    kc, vc = (torch.full((n_pages, page, H, D), math.nan, dtype=ref.BF16, device=DEV) for _ in range(2))
    used = small.table.flatten().long()
    far = torch.arange(n_pages - used.numel(), n_pages, dtype=torch.int32, device=DEV)
    kc[far.long()], vc[far.long()] = small.k_cache[used], small.v_cache[used]
    o = torch.zeros_like(small.q)
    dg.dg_paged_attention(small.q, kc, vc, o, far[None], small.cu, small.kv_len, small.causal, rows)
    ref.check_attention(small, o, None)


@pytest.mark.parametrize("rows", [5, 640])
def test_attention_nan_queries_stay_in_their_rows(rows):
    """A query of NaN: its rows of o and lse are NaN, by either path; all others are right."""
    b = ref.Batch([(rows, 700, 1), (1, 900, 1)], 8, 8, 64, 16, seed=rows).fill_keys()
    o0, l0 = _attend(b)
    q = b.q[2, 3].clone()
    b.q[2, 3] = math.nan
    o, lse = _attend_only(b)
    assert torch.isnan(o[2, 3]).all() and torch.isnan(lse[2, 3])
    b.q[2, 3], o[2, 3], lse[2, 3] = q, o0[2, 3], l0[2, 3]
    ref.check_attention(b, o, lse)


@pytest.mark.parametrize("rows,D,Hq,Hkv", [(1, 64, 8, 8), (2, 64, 8, 4), (1, 64, 3, 3), (8, 64, 2, 2), (1, 128, 8, 4), (300, 64, 16, 8)])
def test_attention_heads_do_not_meet(rows, D, Hq, Hkv):
    """NaN keys and infinite values that one key head may see: its query heads alone show them."""
    b = ref.Batch([(rows, 700, 0), (1, 90, 1)], Hq, Hkv, D, 16, seed=rows + D).fill_keys()
    want, lse = _attend(b)
    bad, group = Hkv - 1 if Hkv == 3 else 1, Hq // Hkv
    at = b.slots(0, [0, 100, 699])
    b.k_cache[at[0], at[1], bad] = math.nan
    b.v_cache[at[0], at[1], bad] = math.inf
    o, l = _attend_only(b)
    mine = slice(bad * group, (bad + 1) * group)
    assert not torch.isfinite(o[:rows, mine]).any() and torch.isnan(l[:rows, mine]).all()
    o[:rows, mine], l[:rows, mine] = want[:rows, mine], lse[:rows, mine]
    b.k_cache[at[0], at[1], bad] = 0
    for s in range(2):   # the other heads against fp64
        sl = slice(int(b.cu[s]), int(b.cu[s + 1]))
        k, v = (t.nan_to_num(0, 0, 0) for t in b.keys(s))
        ro, rl, bound, lbound = ref.attention(b.q[sl], k, v, bool(b.causal[s]), -1, D ** -0.5)
        clean = [h for h in range(Hq) if s or not mine.start <= h < mine.stop]
        assert ((o[sl].double() - ro).abs() <= bound)[:, clean].all()
        assert ((l[sl].double() - rl).abs() <= lbound)[:, clean].all()


def test_attention_repeats_bit_for_bit():
    for seqs in (TOKENS * 5, [(1, 50000, 1)], MIXED):
        b = ref.Batch(seqs, 8, 4, 128, 16, seed=4).fill_keys()
        o0, l0 = _attend(b)
        for _ in range(8):
            o, lse = _attend_only(b)
            assert torch.equal(o.view(torch.int16)[:b.cu[-1]], o0.view(torch.int16)[:b.cu[-1]])
            assert torch.equal(lse, l0)


def _attend_only(b, workspace=None, stream=None):
    o = torch.full(b.q.shape, 7.0, dtype=ref.BF16, device=DEV)
    lse = torch.full(b.q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, max(s[0] for s in b.seqs),
                          lse=lse, workspace=workspace, stream=stream)
    return o, lse


def test_attention_workspace_needs_no_contents_and_is_checked():
    b = ref.Batch([(1, 3000, 1), (1, 20, 1)], 8, 4, 128, 16, seed=4).fill_keys()
    need = dg.dg_paged_attention_workspace_bytes(2, 1, 8, 4, 128)
    o0, l0 = _attend(b)
    for byte in (0, 255, 127):
        ws = torch.full((max(16, need),), byte, dtype=torch.uint8, device=DEV)
        o, lse = _attend_only(b, ws)
        torch.cuda.synchronize()
        assert torch.equal(o, o0) and torch.equal(lse, l0)
    if need:
        with pytest.raises(dg.DGError, match="WORKSPACE"):
            _attend_only(b, torch.empty(need - 1, dtype=torch.uint8, device=DEV))
        with pytest.raises(dg.DGError, match="ALIGNMENT"):
            _attend_only(b, torch.empty(need + 8, dtype=torch.uint8, device=DEV)[8:])


@pytest.mark.parametrize("q", [1, 100, 400])
def test_attention_on_streams_and_in_graphs(q):
    """Two calls at once on two streams, and a captured call replayed after its inputs changed: one token,
    and rows for the split keys (100) and for the query tiles (400)."""
    bs = [ref.Batch([(q, 5000 + 500 * i, 1)] * 3, 8, 4, 128, 16, seed=i).fill_keys() for i in range(2)]
    want = [_attend(b) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(3):
        torch.cuda.synchronize()
        got = [_attend_only(b, stream=st) for b, st in zip(bs, streams)]
        torch.cuda.synchronize()
        for (o, l), (o0, l0) in zip(got, want):
            assert torch.equal(o, o0) and torch.equal(l, l0)
    b = bs[0]
    need = dg.dg_paged_attention_workspace_bytes(3, q, 8, 4, 128)
    ws = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
    o, lse = torch.zeros_like(b.q), torch.zeros(b.q.shape[:2], device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, q, lse=lse, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])
    # the same graph with other lengths: an empty slot, one key more than the queries, a shorter one
    b.seqs = [(q, 0, 1), (q, q + 1, 1), (q, 2777, 1)]
    b.kv_len.copy_(torch.tensor([0, q + 1, 2777], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    ref.check_attention(b, o, lse)


def test_calls_from_two_threads_at_once():
    """Threads that append to their own caches and attend, each on its own stream, without workspaces."""
    import threading
    bs = [ref.Batch([(q, 1500 + 100 * q, 1)] * 5, 8, 4, 64, 16, seed=q).fill_keys() for q in (1, 3, 300)]
    want = [_attend(b) for b in bs]
    got, streams = [None] * 3, [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()

    def run(i):
        b = bs[i]
        rows = torch.cat([torch.arange(kl - a, kl) for a, kl, _ in b.seqs])
        at = b.table[torch.arange(5, device=DEV).repeat_interleave(b.seqs[0][0]), rows.to(DEV) // 16].long(), rows.to(DEV) % 16
        with torch.cuda.stream(streams[i]):
            k, v = b.k_cache[at], b.v_cache[at]      # what the cache holds: appended again, it stays the same
            for _ in range(30):
                dg.dg_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cu, b.kv_len)
                got[i] = _attend_only(b)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == 0
    for (o, lse), (o0, l0) in zip(got, want):
        assert torch.equal(o, o0) and torch.equal(lse, l0)


def test_append_then_attend_step_by_step():
    """Tokens appended one by one and read back, as a decoding loop does, against the packed form."""
    n, Hq, Hkv, D, page, steps = 3, 4, 2, 64, 8, 20
    g = torch.Generator(device=DEV).manual_seed(1)
    pages = steps // page + 1
    table = torch.randperm(n * pages, generator=torch.Generator().manual_seed(2)).view(n, pages).to(torch.int32).to(DEV)
    kc, vc = (torch.full((n * pages, page, Hkv, D), float("nan"), dtype=ref.BF16, device=DEV) for _ in range(2))
    cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    causal = torch.ones(n, dtype=torch.uint8, device=DEV)
    w = _inv_freq(D)
    keys, values = [], []
    kv_len = torch.zeros(n, dtype=torch.int32, device=DEV)
    for step in range(steps):
        x = torch.randn((n, (Hq + 2 * Hkv) * D), generator=g, device=DEV).to(ref.BF16)
        q, k, v = (x[:, a * D:e * D].unflatten(1, (e - a, D)) for a, e in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        kv_len += 1
        qr, o = torch.empty((n, Hq, D), dtype=ref.BF16, device=DEV), torch.empty((n, Hq, D), dtype=ref.BF16, device=DEV)
        dg.dg_kv_append(k, v, kc, vc, table, cu, kv_len, inv_freq=w, q=q, q_out=qr)
        dg.dg_paged_attention(qr, kc, vc, o, table, cu, kv_len, causal, 1)
        keys.append(ref.rotate(k.double(), torch.full((n,), step, device=DEV), w, False).to(ref.BF16))
        values.append(v)
        for s in range(n):
            kk, vv = torch.stack([t[s] for t in keys]), torch.stack([t[s] for t in values])
            ro, _, bound, _ = ref.attention(qr[s:s + 1], kk, vv, True, -1, 1 / 8)
            # a key rounded the other way than fp64's is a step of 2^-7 off: rare, and the scores move by
            # at most 2^-7 |q| |k| / 8 for one dimension
            kmax = 2.0 ** -7 * float((qr[s].abs().max() * kk.abs().max())) / 8
            assert ((o[s].double() - ro[0]).abs() <= bound[0] + 2 * kmax * vv.abs().max()).all(), (step, s)
    assert dg.dg_get_device_status() == 0
