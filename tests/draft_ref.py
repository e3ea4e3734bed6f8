"""Plain fp64 forms of the calls for drafted tokens (normed append, tree and sink attention, verification, kept
paths) in torch on any device, written from the definitions in include/dg.h."""
from __future__ import annotations

import math

import numpy as np
import torch

import serving_ref as ref


def random_tree(g, q, wide=3):
    """Parents, depths and ancestor sets of a random tree of q nodes, the root first."""
    parent, depth, anc = [-1], [0], [{0}]
    for i in range(1, q):
        lo = max(0, i - 1 - int(torch.randint(0, 2 * wide, (1,), generator=g)))
        p = int(torch.randint(lo, i, (1,), generator=g))
        parent.append(p)
        depth.append(depth[p] + 1)
        anc.append(anc[p] | {i})
    return parent, depth, anc


def words(sets, width, device):
    """Sets of node numbers as rows of `width` 32-bit words (numbers past them are left out)."""
    m = np.zeros((len(sets), width * 32), np.uint8)
    for i, s in enumerate(sets):
        for j in s:
            if j < width * 32:
                m[i, j] = 1
    return torch.from_numpy(np.packbits(m, axis=1, bitorder="little").view(np.int32).copy()).to(device)


def normed(x, w, eps):
    """x [t, h, D] float64 (None weights: as it is)."""
    return x if w is None else x * w.double() / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def attention(q, k, v, ok, scale):
    """One sequence in fp64: q [a, Hq, D], k, v [m, Hkv, D], ok [a, m] -> o, lse and their bounds: weights
    rounded to bf16 before the product with v (half a step of each, at most 2^-8), the output's own rounding (2^-8),
    fp32 scores of D products, fp32 weights and sums of m keys."""
    a, Hq, D = q.shape
    m, Hkv, _ = k.shape
    rep = Hq // Hkv
    q, k, v = q.double(), k.double().repeat_interleave(rep, 1), v.double().repeat_interleave(rep, 1)
    seen = ok.any(0)
    k = torch.where(seen[:, None, None], k, torch.zeros_like(k))
    v = torch.where(seen[:, None, None], v, torch.zeros_like(v))
    x = torch.einsum("ahd,mhd->ham", q, k) * scale
    mag = (torch.einsum("ahd,mhd->ham", q.abs(), k.abs()) * abs(scale)).masked_fill(~ok, 0.0)
    x = x.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = (x - lse[..., None]).exp().masked_fill(~ok, 0.0)
    o = torch.einsum("ham,mhd->ahd", p, v)
    wide = torch.einsum("ham,mhd->ahd", p, v.abs())
    ds = (D + 4) * 2.0 ** -24 * mag.amax(-1) + (m + 8) * 2.0 ** -24 + 2.0 ** -20
    ds = ds.T[..., None]
    bound = 2.0 ** -8 * wide + 2 * ds * wide + 2.0 ** -8 * o.abs()
    return o, lse.T, bound, ds[..., 0] + 2.0 ** -21 * lse.T.abs().nan_to_num(0, 0, 0)


def visible(a, m, *, anc=None, positions=None, window=-1, sinks=0):
    """[a, m]: what each of a sequence's last a queries sees of its m keys; anc: sets of nodes (None: causal)."""
    ctx = m - a
    j = torch.arange(m)[None, :]
    pos = torch.arange(ctx, m) if positions is None else torch.as_tensor(positions)
    ok = torch.ones((a, m), dtype=torch.bool)
    if window >= 0:
        ok = (j >= pos[:, None] - window) | (j < sinks)
    if anc is None:
        return ok & (j <= torch.arange(ctx, m)[:, None])
    for i in range(a):
        ok[i, ctx:] = False
        for n in anc[i]:
            if n < a:
                ok[i, ctx + n] = True
    return ok


def check_attention(b, o, lse, oks, scale=None, sentinel=None, skip=()):
    """Every row of batch b against fp64, sequence s with visibility oks[s]; rows of no sequence (and of `skip`)
    keep the sentinel."""
    scale = 1.0 / math.sqrt(b.D) if scale is None else scale
    owned = torch.zeros(b.total, dtype=torch.bool)
    cu = b.cu.tolist()
    for s, (a, kl, _) in enumerate(b.seqs):
        if s in skip:
            continue
        rows = slice(cu[s], cu[s + 1])
        owned[rows] = True
        if a == 0:
            continue
        if kl == 0:
            assert (o[rows] == 0).all() and (lse[rows] == -math.inf).all(), s
            continue
        k, v = b.keys(s)
        ro, rl, bound, lbound = attention(b.q[rows], k, v, oks[s].to(o.device), scale)
        none = torch.isinf(rl)
        assert torch.isfinite(o[rows]).all(), s
        err = (o[rows].double() - ro).abs()
        assert (err <= bound).all(), (s, float((err / bound).max()))
        assert (lse[rows][none] == -math.inf).all()
        le = (lse[rows].double() - rl).abs()[~none]
        assert (le <= lbound[~none]).all(), (s, float((le / lbound[~none]).max()))
    if sentinel is not None:
        assert (o[~owned.to(o.device)] == sentinel).all()
        assert (lse[~owned.to(o.device)] == sentinel).all()


def verify(logits, tokens, T, u, u_next, parents=None, probs=None):
    """One sequence: logits [q, V] -> (path, tokens with the next one, gap): gap is how near, relative to the mass
    compared, some comparison came to its border."""
    x = logits.double().cpu()
    q, V = x.shape
    tokens, u = tokens.tolist(), u.double().tolist()
    path, out, gap = [0], [], math.inf
    while True:
        node = path[-1]
        p = torch.softmax(x[node] / T, 0) if T else None
        best = int(x[node].argmax())
        left, gone, moved, rejected = 1.0, [], False, None
        for c in range(node + 1, q):
            if (parents[c] if parents is not None else c - 1) != node:
                continue
            t = tokens[c]
            if T == 0:
                moved = t == best
            else:
                pt = float(p[t]) if 0 <= t < V and t not in gone else 0.0
                if probs is not None:
                    lhs = u[c] * (float(probs[c, t].double().clamp(0, 1).nan_to_num(0)) if 0 <= t < V else 1.0)
                else:
                    lhs = u[c] * left
                moved = lhs < pt
                if lhs != pt:
                    gap = min(gap, abs(lhs - pt) / max(lhs, pt))
                if not moved:
                    rejected = c
                    if 0 <= t < V and t not in gone:
                        gone.append(t)
                        left -= pt
            if moved:
                path.append(c)
                out.append(t)
                break
        if not moved:
            break
    if T == 0:
        return path, out + [best], gap
    r = p.clone()
    if probs is not None and rejected is not None:
        r = (p - probs[rejected].double().cpu().nan_to_num(0).clamp(0, 1)).clamp(min=0)
    elif probs is None and gone:
        r[gone] = 0
    if float(r.sum()) == 0:
        r = p
    edge = r.cumsum(0)
    at = float(u_next) * float(edge[-1])
    nxt = int(torch.searchsorted(edge, at, right=True))
    gap = min(gap, float((edge - at).abs().min()) / float(edge[-1]))
    return path, out + [nxt], gap


__all__ = ["random_tree", "words", "normed", "attention", "visible", "check_attention", "verify", "ref"]
