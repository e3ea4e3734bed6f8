"""GPU tests of the serving calls (dg_kv_append, dg_paged_attention, dg_adjust_logits) where their arguments
are at the edge of what include/dg.h allows, or past it: what is reported, what is left alone."""
import math

import numpy as np
import pytest
import torch

import entropy_bounded_denoising_gb300 as dg

import serving_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAD = dg.DG_DEV_BAD_PARAM


# ------------------------------------------------------------------ sequences that are refused
def _three(seqs=((4, 20, 1), (5, 16, 1), (3, 30, 1))):
    return ref.Batch(list(seqs), 2, 1, 64, 16, seed=2, extra_columns=0).fill_keys()


def _claims(b):
    """Per row of q: the sound sequences that claim it."""
    cu, kl = b.cu.tolist(), b.kv_len.tolist()
    cap = b.table.shape[1] * b.page_size
    claims = [[] for _ in range(b.total)]
    for s, n in enumerate(kl):
        q0, q1 = cu[s], cu[s + 1]
        if 0 <= q0 <= q1 <= b.total and 0 < n <= cap and q1 - q0 <= n:
            for t in range(q0, q1):
                claims[t].append(s)
    return claims


def _append_copies(b):
    """Appends random rows without rotation; every row goes to the slot of a sound sequence that claims it or,
    where the offsets go back, nowhere; nothing else changes.  Returns the status."""
    g = torch.Generator(device=DEV).manual_seed(7)
    q, k, v = (torch.randn((b.total, h, 64), generator=g, device=DEV).to(ref.BF16) for h in (2, 1, 1))
    o = torch.full_like(q, 7.0)
    before = b.k_cache.clone(), b.v_cache.clone()
    dg.dg_clear_device_status()
    dg.dg_kv_append(k, v, b.k_cache, b.v_cache, b.table, b.cu, b.kv_len, q=q, q_out=o)
    torch.cuda.synchronize()
    status = dg.dg_get_device_status()
    cu, kl = b.cu.tolist(), b.kv_len.tolist()
    ordered = all(x <= y for x, y in zip(cu, cu[1:]))
    same = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))  # noqa: E731
    free = torch.ones(b.k_cache.shape[:2], dtype=torch.bool, device=DEV)   # slots that no row may write
    for t, claims in enumerate(_claims(b)):
        written = not same(o[t], torch.full_like(o[t], 7.0))
        assert not written or same(o[t], q[t])
        assert written == bool(claims) if ordered else claims or not written
        at = [b.slots(s, [kl[s] - (cu[s + 1] - cu[s]) + t - cu[s]]) for s in claims]
        if written:
            assert any(same(b.k_cache[x][0], k[t]) and same(b.v_cache[x][0], v[t]) for x in at)
        for x in at:
            free[x] = False
    for now, was in zip((b.k_cache, b.v_cache), before):
        assert same(now[free], was[free])
    return status


@pytest.mark.parametrize("cu", [[5, 4, 3, 2], [0, 9, 4, 12], [0, -5, 9, 12], [0, 4, 12, 62], [-7, 4, 9, 12],
                                [0, 2 ** 31 - 1, 9, 12], [12, 0, 0, 0]])
def test_bad_offsets_are_reported_by_each_call(cu):
    b = _three()
    b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    assert _append_copies(b) == BAD
    o = torch.full(b.q.shape, 7.0, dtype=ref.BF16, device=DEV)
    dg.dg_clear_device_status()
    dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, 9)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == BAD
    for t, claims in enumerate(_claims(b)):
        if not claims:
            assert (o[t] == 7.0).all(), t
        elif len(claims) == 1:
            s = claims[0]
            at = b.slots(s, range(int(b.kv_len[s])))
            rows = slice(int(b.cu[s]), int(b.cu[s + 1]))
            ro, _, bound, _ = ref.attention(b.q[rows], b.k_cache[at], b.v_cache[at], True, -1, 1 / 8)
            assert ((o[t].double() - ro[t - rows.start]).abs() <= bound[t - rows.start]).all(), t
    dg.dg_clear_device_status()


@pytest.mark.parametrize("kv_len", [-1, 33, 2 ** 31 - 1])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_append_reports_bad_lengths_of_sequences_without_rows(which, kv_len):
    seqs = [(4, 20, 1), (5, 16, 1), (3, 30, 1)]
    seqs[which] = (0, 16, 1)
    b = _three(seqs)
    assert _append_copies(b) == 0
    b.kv_len[which] = kv_len
    assert _append_copies(b) == BAD
    dg.dg_clear_device_status()


@pytest.mark.parametrize("rows", [1, 40])
def test_append_checks_thousands_of_sequences(rows):
    """More sequences than the grid has threads, of which the last ones have no rows."""
    for bad in (None, 0, 1, 2999, 5555, 5999):
        b = ref.Batch([(rows, 50, 1)] + [(0, 3, 1)] * 5999, 2, 1, 64, 64, seed=2, extra_columns=0).fill_keys()
        if bad is not None:
            b.kv_len[bad] = -1
        assert _append_copies(b) == (0 if bad is None else BAD), bad
    dg.dg_clear_device_status()


# ------------------------------------------------------------------ angles
def _pi(bits):
    """floor(pi 2^bits): 16 atan(1 / 5) - 4 atan(1 / 239), in integers with 64 bits to spare."""
    one = 1 << (bits + 64)

    def atan(n):
        total, power, k = 0, one // n, 1
        while power:
            total += power // k if k % 4 == 1 else -(power // k)
            power //= n * n
            k += 2
        return total

    return (16 * atan(5) - 4 * atan(239)) >> 64


def _angle(w, p):
    """w p modulo a turn, in radians: the double w taken exactly."""
    n, d = w.as_integer_ratio()
    turn = 2 * _pi(400)                       # of 2^-400 radians
    r = ((n * p) << 400) // d % turn
    return r / (1 << 400)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size", [1e-3, 1.0, 3.9999, 4.0, 100.0, 1e6, 1e12, 2.0 ** 52])
def test_far_positions_with_frequencies_of_many_turns(size, interleaved):
    """Positions near 2^31 and frequencies up to 2^53 of either sign: the bound is that of near positions."""
    D, page, far = 64, 65536, (1 << 31) - 3
    table = torch.full((1, far // page + 1), -1, dtype=torch.int32, device=DEV)
    table[0, (far - 5) // page:] = 0
    cache = [torch.zeros((1, page, 1, D), dtype=ref.BF16, device=DEV) for _ in range(2)]
    k = torch.randn((5, 1, D), generator=torch.Generator().manual_seed(3)).to(ref.BF16).to(DEV)
    w = [size * (1 + (j * 0.6180339887498949) % 1 * 0.999) * (-1) ** (j // 2) for j in range(D // 2)]
    dg.dg_clear_device_status()
    dg.dg_kv_append(k, k, *cache, table, torch.tensor([0, 5], dtype=torch.int32, device=DEV),
                    torch.tensor([far], dtype=torch.int32, device=DEV),
                    inv_freq=torch.tensor(w, dtype=torch.float64, device=DEV), interleaved=interleaved)
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == 0
    for i in range(5):
        p = far - 5 + i
        ang = torch.tensor([_angle(x, p) for x in w], dtype=torch.float64, device=DEV)
        want = ref.rotate(k[i:i + 1].double(), torch.ones(1, device=DEV), ang, interleaved)[0, 0]
        got = cache[0][0, p % page, 0].double()
        # two units of 2^-64 of a turn a position: 2 pi 2^-32 radians at most, next to 2^-22 for sine and cosine
        slack = ref.rotation_bound(k[i:i + 1].double(), ang, interleaved)[0, 0] * (1 + 2 * math.pi * 2.0 ** -32 * 2.0 ** 21)
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + slack).all(), i


def test_frequencies_without_an_angle_are_refused():
    """Frequencies of 2^53 and more, infinite ones and NaN raise the status and turn nothing; those beside them do."""
    w = [0.5, 2.0 ** 53, -2.0 ** 53, 1e300, math.inf, -math.inf, math.nan, 2.0 ** 53 - 1]
    b = ref.Batch([(3, 40, 1), (1, 9, 1)], 2, 1, 64, 16, seed=4).fill_keys()
    k = torch.randn((4, 1, 64), generator=torch.Generator().manual_seed(1)).to(ref.BF16).to(DEV)
    for j in range(8):
        f = torch.zeros(8, dtype=torch.float64, device=DEV)
        f[j] = w[j]
        dg.dg_clear_device_status()
        dg.dg_kv_append(k, k, b.k_cache, b.v_cache, b.table, b.cu, b.kv_len, inv_freq=f)
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == (0 if j in (0, 7) else BAD), w[j]
        got = b.k_cache[b.slots(1, [8])][0]
        assert torch.equal(got, k[3]) != (j in (0, 7)), w[j]
    dg.dg_clear_device_status()


# ------------------------------------------------------------------ scores
@pytest.mark.parametrize("rows,n", [(1, 2), (300, 2), (256, 24)])
@pytest.mark.parametrize("size", [2.0 ** 56, 2.0 ** 60, 1.0])
def test_scales_that_undo_large_queries_and_keys(rows, n, size):
    """Queries and keys of 2^56 and a scale of 2^-114 are scores like any others; scales of 0 and next to it weigh
    every key alike."""
    b = ref.Batch([(rows, 500, 0)] * n, 8, 8, 64, 16, seed=rows).fill_keys()
    b.q.mul_(size)
    b.k_cache.mul_(size)
    for scale in (2.0 ** -2 / size ** 2, -2.0 ** -2 / size ** 2, 2.0 ** -140, 0.0):
        o = torch.full(b.q.shape, 7.0, dtype=ref.BF16, device=DEV)
        lse = torch.full(b.q.shape[:2], 7.0, device=DEV)
        dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, rows, lse=lse, scale=scale)
        for s in (0, n - 1):
            sl = slice(int(b.cu[s]), int(b.cu[s + 1]))
            ro, rl, bound, lbound = ref.attention(b.q[sl], *b.keys(s), False, -1, scale)
            assert ((o[sl].double() - ro).abs() <= bound).all() and ((lse[sl].double() - rl).abs() <= lbound).all(), scale


# ------------------------------------------------------------------ logit edits
def _active(n):
    p = np.zeros((n, dg.PARAM_BYTES // 4), np.int32)
    p[:, 0] = np.float32(1.0).view(np.int32)
    p[:, -1] = dg.DG_ACTIVE
    return torch.from_numpy(p.view(np.uint8).reshape(-1)).to(DEV)


def _ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_repetitions_without_a_normal_reciprocal_are_refused():
    """x / repetition is x times the rounded reciprocal: right to 2^-23 where that is a normal number, refused
    where it is not."""
    x = torch.tensor([[[1e-30, 3.0, 1e30, -1e-30, -3.0, -1e30, 0.0, 7.0]]], device=DEV)
    for rep, sound in ((2.0 ** -126, 1), (2.0 ** 126, 1), (1e-37, 1), (8e37, 1), (1.7, 1), (2.0 ** -127, 0), (1e-39, 0),
                       (2.0 ** 126 * (1 + 2.0 ** -23), 0), (3e38, 0), (math.inf, 0), (math.nan, 0), (0.0, 0), (-2.0, 0)):
        out = torch.full_like(x, 9.0)
        dg.dg_clear_device_status()
        dg.dg_adjust_logits(x, _active(1), out, history=_ints(*range(7)), cu_history=_ints(0, 7),
                            penalties=torch.tensor([[rep, 0.0, 0.0]], device=DEV))
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == (0 if sound else BAD), rep
        if not sound:
            assert (out == 9.0).all(), rep
            continue
        r = float(torch.tensor(rep, dtype=torch.float32))
        for t, v in enumerate(x[0, 0].tolist()):
            want = v if t == 7 else v / r if v > 0 else v * r
            got = float(out[0, 0, t])
            # fp32: beyond its range infinity, below it steps of 2^-149
            assert got == want or (abs(want) >= 3.4e38 and got == math.copysign(math.inf, want)) or \
                abs(got - want) <= 2.0 ** -23 * abs(want) + 2.0 ** -149, (rep, v, got)
    dg.dg_clear_device_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,lens,kinds", [(2, [1, 2, 700], 2), (5000, [1023, 1024, 1025, 0, 3000], 40), (5000, [4097, 2], 5000),
                                          (70001, [2, 9000, 2048], 4500), (3001, [6000, 6000, 1], 1)])
def test_repeated_biases_add_up_in_list_order(V, lens, kinds, dtype):
    """Lists in which tokens come many times, anywhere: the fp32 sum in list order, bit for bit."""
    n, L = len(lens), 3
    g = torch.Generator().manual_seed(V + kinds)
    cu = np.cumsum([0] + lens)
    pool = torch.randperm(V + 2, generator=g)[:kinds] - 1                   # -1 and V among them: ignored
    tok = pool[torch.randint(0, len(pool), (int(cu[-1]),), generator=g)].to(torch.int32)
    val = (torch.randn(int(cu[-1]), generator=g) * 10.0 ** torch.randint(-3, 4, (int(cu[-1]),), generator=g)).float()
    ld = -(-V // 8) * 8
    x = torch.randn((n, L, ld), generator=g).to(dtype)
    for in_place in (False, True):
        xd = x.to(DEV)
        out = xd if in_place else torch.full_like(xd, 9.0)
        dg.dg_clear_device_status()
        dg.dg_adjust_logits(xd, _active(n), None if in_place else out, bias_tokens=tok.to(DEV), bias_values=val.to(DEV),
                            cu_bias=torch.from_numpy(cu.astype(np.int32)).to(DEV), V=V)
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == 0
        for c in range(n):
            s = np.zeros(V, np.float32)
            for t, v in zip(tok[cu[c]:cu[c + 1]].tolist(), val[cu[c]:cu[c + 1]].numpy()):
                if 0 <= t < V:
                    s[t] = np.float32(s[t] + v)
            seen = torch.zeros(V, dtype=torch.bool)
            seen[[t for t in tok[cu[c]:cu[c + 1]].tolist() if 0 <= t < V]] = True
            want = torch.where(seen, x[c, :, :V].float() + torch.from_numpy(s), x[c, :, :V].float()).to(dtype)
            assert torch.equal(out[c, :, :V].cpu(), want), c


def test_repeated_biases_take_no_more_than_a_few_times_as_long():
    """4000 tokens given twice against 8000 given once: the entries of a token lie 4000 apart."""
    V, L = 32768, 16
    x = torch.randn((1, L, V), device=DEV)
    out, params, cu = torch.empty_like(x), _active(1), _ints(0, 8000)
    tok = torch.randperm(V, device=DEV)[:8000].to(torch.int32)
    val = torch.randn(8000, device=DEV)

    def best(tokens):
        times = []
        for _ in range(8):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            dg.dg_adjust_logits(x, params, out, bias_tokens=tokens, bias_values=val, cu_bias=cu)
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        return min(times)

    once, twice = best(tok), best(tok[:4000].repeat(2))
    print(f"once {once * 1000:.1f} us, twice {twice * 1000:.1f} us")
    assert twice < 10 * once, (once, twice)   # 80 times before such lists were read by the whole block


# ------------------------------------------------------------------ workspaces
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_workspace_serves_a_programs_calls(D):
    """A buffer of the size of the largest call, for tokens, drafts and canvases one after another."""
    ws = torch.empty(dg.dg_paged_attention_workspace_bytes(70, 300, 16, 8, D), dtype=torch.uint8, device=DEV)
    for n, rows in ((70, 1), (1, 1), (5, 5), (3, 40), (2, 300), (70, 2), (24, 200)):
        b = ref.Batch([(rows, rows + 90, 1)] * n, 16, 8, D, 16, seed=n).fill_keys()
        o, lse = torch.full_like(b.q, 7.0), torch.full(b.q.shape[:2], 7.0, device=DEV)
        dg.dg_paged_attention(b.q, b.k_cache, b.v_cache, o, b.table, b.cu, b.kv_len, b.causal, rows, lse=lse, workspace=ws)
        ref.check_attention(b, o, lse, skip=range(3, n))


@pytest.mark.parametrize("rows", [1, 300])
def test_caches_whose_strides_differ_where_the_extent_is_one(rows):
    b = ref.Batch([(rows, 400, 1)] * 3, 8, 1, 64, 16, seed=rows).fill_keys()
    ends = []
    for v in (b.v_cache, b.v_cache.transpose(1, 2).contiguous().transpose(1, 2)):
        b.v_cache = v
        assert _append_copies(b) == 0
        o = torch.zeros_like(b.q)
        dg.dg_paged_attention(b.q, b.k_cache, v, o, b.table, b.cu, b.kv_len, b.causal, rows)
        ref.check_attention(b, o, None)
        ends.append(o)
    assert torch.equal(*ends)
