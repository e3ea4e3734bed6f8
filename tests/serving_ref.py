"""Plain fp64 forms of the serving operators (paged cache append, paged attention, logit edits) and
the batches their tests run, in torch on any device, written from the definitions in include/dg.h."""
from __future__ import annotations

import math

import numpy as np
import torch

BF16 = torch.bfloat16
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # relative, of one rounding


class Batch:
    """A paged batch: seqs = [(q_len, kv_len, causal)]; `before` / `after` rows of q that no sequence
    owns; pages in random order, the table's unused entries invalid, `spare` pages nobody owns."""

    def __init__(self, seqs, Hq, Hkv, D, page_size, *, seed, head_major=False, before=0, after=0, spare=2,
                 device="cuda", fill=float("nan"), extra_columns=2, q_scale=2.0):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.seqs, self.Hq, self.Hkv, self.D, self.page_size = seqs, Hq, Hkv, D, page_size
        ql = [s[0] for s in seqs]
        self.cu = torch.tensor(np.cumsum([before] + ql), dtype=torch.int32)
        self.total = int(self.cu[-1]) + after
        self.kv_len = torch.tensor([s[1] for s in seqs], dtype=torch.int32)
        self.causal = torch.tensor([int(s[2]) for s in seqs], dtype=torch.uint8)
        used = [-(-s[1] // page_size) for s in seqs]
        n_pages = sum(used) + spare
        order = torch.randperm(n_pages, generator=g).tolist()
        width = max(used + [1]) + extra_columns
        self.table = torch.full((len(seqs), width), -7, dtype=torch.int32)
        k = 0
        for s, u in enumerate(used):
            for j in range(u):
                self.table[s, j] = order[k]
                k += 1
        self.n_pages = n_pages
        shape = (n_pages, Hkv, page_size, D) if head_major else (n_pages, page_size, Hkv, D)
        make = lambda: (lambda t: t.transpose(1, 2) if head_major else t)(  # noqa: E731
            torch.full(shape, fill, dtype=BF16, device=device))
        self.k_cache, self.v_cache = make(), make()
        self.device = device
        self.g = g
        self.q = (torch.randn((self.total, Hq, D), generator=g) * q_scale).to(BF16).to(device)
        for name in ("cu", "kv_len", "causal", "table"):
            setattr(self, name, getattr(self, name).to(device))

    def slots(self, s, positions):
        """Page and slot indices of positions of sequence s."""
        p = torch.as_tensor(positions, device=self.device, dtype=torch.long)
        return self.table[s].long()[p // self.page_size], p % self.page_size

    def fill_keys(self):
        """Random keys and values in every slot a sequence owns; the rest keeps its fill."""
        for s, (_, kl, _) in enumerate(self.seqs):
            if kl:
                at = self.slots(s, range(kl))
                for c in (self.k_cache, self.v_cache):
                    c[at] = torch.randn((kl, self.Hkv, self.D), generator=self.g).to(BF16).to(self.device)
        return self

    def keys(self, s):
        at = self.slots(s, range(self.seqs[s][1]))
        return self.k_cache[at], self.v_cache[at]


def rotate(x, pos, w, interleaved):
    """x [t, h, D] float64 with its first 2 len(w) dimensions rotated by pos * w."""
    r = 2 * w.numel()
    y = x.clone()
    ang = pos.double()[:, None, None] * w.double()
    ia = torch.arange(0, r, 2, device=x.device) if interleaved else torch.arange(r // 2, device=x.device)
    ib = ia + (1 if interleaved else r // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * ang.cos() - b * ang.sin()
    y[..., ib] = a * ang.sin() + b * ang.cos()
    return y


def rotation_bound(x, w, interleaved):
    """What fp32 may lose of a rotated value before its rounding: sines and cosines within 2^-22, two
    products and a sum."""
    r = 2 * w.numel()
    m = torch.zeros_like(x)
    ia = torch.arange(0, r, 2, device=x.device) if interleaved else torch.arange(r // 2, device=x.device)
    ib = ia + (1 if interleaved else r // 2)
    both = x[..., ia].abs() + x[..., ib].abs()
    m[..., ia] = both
    m[..., ib] = both
    return 2.0 ** -21 * m


def attention(q, k, v, causal, window, scale):
    """One sequence in fp64: q [a, Hq, D], k, v [m, Hkv, D] -> o, lse, and per output the bound that
    the kernels' arithmetic gives: weights rounded to bf16 before the product with v (half a step of each),
    scores from fp32 sums of D products, weights and sums in fp32, the output rounded to bf16."""
    a, Hq, D = q.shape
    m, Hkv, _ = k.shape
    rep = Hq // Hkv
    q, k, v = q.double(), k.double().repeat_interleave(rep, 1), v.double().repeat_interleave(rep, 1)
    x = torch.einsum("ahd,mhd->ham", q, k) * scale
    mag = torch.einsum("ahd,mhd->ham", q.abs(), k.abs()) * abs(scale)
    pos = torch.arange(m - a, m, device=q.device)[:, None]
    j = torch.arange(m, device=q.device)[None, :]
    ok = torch.ones((a, m), dtype=torch.bool, device=q.device)
    if causal:
        ok &= j <= pos
    if window >= 0:
        ok &= (j >= pos - window) & (j <= pos + window)
    x = x.masked_fill(~ok, -math.inf)
    mag = mag.masked_fill(~ok | mag.isinf(), 0.0)
    lse = torch.logsumexp(x, -1)
    p = (x - lse[..., None]).exp()
    v0 = torch.where(ok.any(0)[:, None, None], v, torch.zeros_like(v))
    o = torch.einsum("ham,mhd->ahd", p, v0)
    wide = torch.einsum("ham,mhd->ahd", p, v0.abs())
    ds = (D + 4) * 2.0 ** -24 * mag.amax(-1) + (m + 8) * 2.0 ** -24 + 2.0 ** -20    # per head and row
    ds = ds.T[..., None]
    bound = 2.0 ** -8 * wide + 2 * ds * wide + 2.0 ** -8 * o.abs()
    return o, lse.T, bound, ds[..., 0] + 2.0 ** -21 * lse.T.abs()


def check_attention(b, o, lse, window=-1, scale=None, sentinel=None, skip=()):
    """Every row of the batch against fp64; rows of no sequence (and of `skip`) keep the sentinel."""
    scale = 1.0 / math.sqrt(b.D) if scale is None else scale
    owned = torch.zeros(b.total, dtype=torch.bool)
    cu = b.cu.tolist()
    for s, (a, kl, causal) in enumerate(b.seqs):
        if s in skip:
            continue
        rows = slice(cu[s], cu[s + 1])
        owned[rows] = True
        if a == 0:
            continue
        if kl == 0:
            assert (o[rows] == 0).all(), s
            if lse is not None:
                assert (lse[rows] == -math.inf).all(), s
            continue
        k, v = b.keys(s)
        ro, rl, bound, lbound = attention(b.q[rows], k, v, causal, window, scale)
        err = (o[rows].double() - ro).abs()
        assert torch.isfinite(o[rows]).all(), s
        assert (err <= bound).all(), (s, float((err / bound).max()))
        if lse is not None:
            le = (lse[rows].double() - rl).abs()
            assert (le <= lbound).all(), (s, float((le / lbound).max()))
    if sentinel is not None:
        assert (o[~owned.to(o.device)] == sentinel).all()
        if lse is not None:
            assert (lse[~owned.to(o.device)] == sentinel).all()


def adjusted(x, V, history, penalties, bias, mask_rows, words):
    """One canvas in fp64: x [L, >=V]; history a list of tokens, penalties (rep, freq, pres), bias a list
    of (token, value), mask_rows [L] row of `words` or -1.  Returns (y [L, V], bound before the last
    rounding, touched [L, V])."""
    y = x[:, :V].double().cpu().clone()
    size = torch.zeros_like(y)
    touched = torch.zeros(y.shape, dtype=torch.bool)
    count = {}
    for t in history:
        if 0 <= t < V:
            count[t] = count.get(t, 0) + 1
    add = {}
    mag = {}
    for t, val in bias:
        if 0 <= t < V:
            add[t] = add.get(t, 0.0) + float(val)
            mag[t] = mag.get(t, 0.0) + abs(float(val))
    rep, freq, pres = (float(np.float32(p)) for p in penalties)
    for t in set(count) | set(add):
        z = y[:, t]
        if t in count:
            z = torch.where(z > 0, z / rep, z * rep)
        more = abs(freq) * count.get(t, 0) + abs(pres) + mag.get(t, 0.0) if t in count else mag.get(t, 0.0)
        size[:, t] = z.abs() + more
        z = z + (add.get(t, 0.0) - (freq * count[t] + pres if t in count else 0.0))
        y[:, t] = z
        touched[:, t] = True
    for i, m in enumerate(mask_rows):
        if m >= 0:
            bits = np.unpackbits(words[m].view(np.uint8), bitorder="little")[:V].astype(bool)
            y[i, ~torch.from_numpy(bits)] = -math.inf
            touched[i, ~torch.from_numpy(bits)] = True
    n_terms = 4 + max([0] + [sum(1 for b in bias if b[0] == t) for t in add])
    return y, n_terms * 2.0 ** -24 * size, touched
