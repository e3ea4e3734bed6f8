"""The serving operators around the denoising step, as cases to be timed: keys and values appended
to a paged cache with the position rotation on the way (``dg_kv_append``), attention over the paged
cache (``dg_paged_attention``) and a request's penalties, biases and grammar masks on the logits
(``dg_adjust_logits``).  Each has its plain form in elementary torch operations."""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
ACTIVE = 1            # flag bit of a canvas that takes part in the step


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one step of 64 causal requests, one new token each: latency counts
        dict(name="append 64 tokens", op="append", n=64, q=1, kv=1024, hq=16, hkv=8, d=128, rot=128,
             page=16, head_major=False, interleaved=False),
        # a denoising pass of 8 canvases, its keys rewritten in place after their context
        dict(name="append 8 canvases", op="append", n=8, q=256, kv=2304, hq=16, hkv=8, d=128, rot=128,
             page=64, head_major=False, interleaved=False),
        # ragged prompts with wide heads, half of each rotated, pages that keep a head's slots together
        dict(name="append ragged prompts", op="append", n=33, q=1531, kv=1531, hq=16, hkv=8, d=256, rot=128,
             page=32, head_major=True, interleaved=True),
        # one request, one token: the latency of the call
        dict(name="token of 1, 1k keys", op="attention", n=1, q=1, kv=1024, hq=16, hkv=8, d=128, page=16,
             causal=True, window=-1, head_major=False),
        # a step of 64 requests with ragged contexts
        dict(name="tokens of 64, 8k keys", op="attention", n=64, q=1, kv=8192, hq=16, hkv=8, d=128, page=16,
             causal=True, window=-1, head_major=False),
        # one very long context: split over its length
        dict(name="token of 1, 128k keys", op="attention", n=1, q=1, kv=131072, hq=16, hkv=4, d=256, page=64,
             causal=True, window=-1, head_major=True),
        # many short reads through a sliding window; MHA heads of 64
        dict(name="tokens of 250, window", op="attention", n=250, q=1, kv=2500, hq=8, hkv=8, d=64, page=32,
             causal=True, window=1000, head_major=False),
        # five drafted tokens a request, verified in one call
        dict(name="5 drafts of 32, 4k keys", op="attention", n=32, q=5, kv=4096, hq=16, hkv=8, d=128, page=16,
             causal=True, window=-1, head_major=True),
        # the denoising batch: 8 canvases of 256 after 2048 tokens of context, bidirectional
        dict(name="8 canvases, 2k context", op="attention", n=8, q=256, kv=2304, hq=16, hkv=8, d=128, page=64,
             causal=False, window=-1, head_major=False),
        # one canvas over a small vocabulary: history, bias, one grammar mask for all positions
        dict(name="edits of 1 canvas, 32k", op="adjust", n=1, L=256, V=32768, dtype="bf16", hist=300, bias=16,
             masks=1, allowed=0.3, in_place=False, idle=False),
        # the batched step: 8 canvases, a grammar mask per position that allows few tokens, fp32 logits
        # of an odd vocabulary width and a quarter of the canvases converged
        dict(name="edits of 8, fp32 ragged", op="adjust", n=8, L=256, V=152063, dtype="fp32", hist=4096, bias=300,
             masks=64, allowed=0.5, in_place=False, idle=True),
        # the batched step's logits masked where they are, few tokens allowed at each position
        dict(name="grammar of 8 in place", op="adjust", n=8, L=256, V=262144, dtype="bf16", hist=0, bias=0,
             masks=256, allowed=0.01, in_place=True, idle=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "adjust"])
    if op == "append":
        d = rng.choice([64, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        q = rng.choice([1, 1, _log(rng, 2, 1500)])
        n = max(1, min(_log(rng, 1, 256), 40000 // q))
        return dict(op=op, n=n, q=q, kv=q + _log(rng, 1, 900), hq=hkv * rng.choice([1, 2, 4]), hkv=hkv, d=d,
                    rot=rng.choice([d, d // 2]), page=rng.choice([8, 16, 32, 64, 128]),
                    head_major=rng.random() < 0.5, interleaved=rng.random() < 0.5)
    if op == "attention":
        d = rng.choice([64, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        kind = rng.choice(["one", "one", "few", "canvas"])
        q = 1 if kind == "one" else rng.randint(2, 8) if kind == "few" else rng.choice([256, rng.randint(33, 300)])
        kv = q + _log(rng, 1, 100000 if kind == "one" else 4000)
        n = max(1, min(_log(rng, 1, 256), (8192 * 64 * 8 * 128 if kind == "one" else 1 << 26) // (kv * hkv * d),
                       40 if kind == "few" else 10 if kind == "canvas" else 256))
        return dict(op=op, n=n, q=q, kv=kv, hq=hkv * rng.choice([1, 2, 4, 8] if kind == "one" else [1, 2, 4]),
                    hkv=hkv, d=d, page=rng.choice([8, 16, 32, 64, 128]),
                    causal=kind != "canvas" or rng.random() < 0.3, window=rng.choice([-1, -1, _log(rng, 16, 2000)]),
                    head_major=rng.random() < 0.5)
    in_place = rng.random() < 0.3
    V = _log(rng, 1000, 262144)
    n = max(1, min(_log(rng, 1, 16), (1 << 29) // (256 * V)))
    return dict(op=op, n=n, L=rng.choice([16, 256, rng.randint(1, 256)]), V=V, dtype=rng.choice(["bf16", "fp32"]),
                hist=0 if in_place else _log(rng, 1, 8000), bias=0 if in_place else _log(rng, 1, 300),
                masks=rng.choice([1, 16, 200]), allowed=rng.choice([0.01, 0.5, 0.95]), in_place=in_place,
                idle=n > 3 and rng.random() < 0.3)


def _lengths(case):
    """Ragged (q_len, kv_len) of a case's sequences, the first one the longest; part of the case, not of
    the seed."""
    rng = np.random.default_rng(case["n"] * 1000003 + case["kv"])
    n, q, kv = case["n"], case["q"], case["kv"]
    if q <= 8 or q == 256:                 # tokens and canvases: whole
        ql = np.full(n, q)
        ctx = np.maximum(0, (kv - q) * rng.uniform(0.3, 1.0, n)).astype(np.int64)
    else:                                  # prompts: ragged, some with context before them
        ql = np.maximum(1, q * rng.uniform(0.2, 1.0, n)).astype(np.int64)
        ctx = ((kv - q) * rng.uniform(0.0, 1.0, n)).astype(np.int64)
    if q == 256 and kv == 2304:            # the denoising batch has one context length
        ctx[:] = kv - q
    ql[0], ctx[0] = q, kv - q
    return ql, ql + ctx


def _seen(case):
    """Per sequence: the number of keys that some query may see, and of allowed (query, key) pairs."""
    ql, kl = _lengths(case)
    keys = pairs = 0
    W = case["window"]
    for a, b in zip(ql.tolist(), kl.tolist()):
        pos = np.arange(b - a, b)
        lo = np.maximum(0, pos - W) if W >= 0 else np.zeros_like(pos)
        hi = pos if case["causal"] else np.minimum(b - 1, pos + W) if W >= 0 else np.full_like(pos, b - 1)
        keys += int(hi.max() - lo.min() + 1)
        pairs += int((hi - lo + 1).sum())
    return keys, pairs


def work(case):
    if case["op"] == "append":
        total = int(_lengths(case)[0].sum())
        one = total * (case["hq"] + 2 * case["hkv"]) * case["d"]
        return {"bytes": 2.0 * 2 * one, "flops": 6.0 * total * (case["hq"] + case["hkv"]) * case["rot"] / 2}
    if case["op"] == "attention":
        total = int(_lengths(case)[0].sum())
        keys, pairs = _seen(case)
        return {"bytes": 4.0 * keys * case["hkv"] * case["d"] + 4.0 * total * case["hq"] * case["d"] + 4.0 * total * case["hq"],
                "flops": 4.0 * pairs * case["hq"] * case["d"]}
    es = 2 if case["dtype"] == "bf16" else 4
    n = _active(case).sum()
    vals = float(n) * case["L"] * case["V"]
    bits = min(case["masks"], int(n) * case["L"]) * case["V"] / 8
    if case["in_place"]:                   # the forbidden tokens are written, nothing is read but the bits
        return {"bytes": vals * (1 - case["allowed"]) * es + bits, "flops": 0.0}
    return {"bytes": vals * (1 + case["allowed"]) * es + bits, "flops": vals}


# ------------------------------------------------------------------ inputs
def _active(case):
    a = np.ones(case["n"], bool)
    if case["idle"]:
        a[3::4] = False
    return a


def _pages(case, kl, g):
    """A page table [n, width] over a pool in random order; -1 where a sequence has no page."""
    page = case["page"]
    used = -(-kl // page)
    width = int(used.max()) + 1
    pool = int(used.sum()) + 3
    order = torch.randperm(pool, generator=g, device=DEV)
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(used)[:-1]])).to(DEV)
    col = torch.arange(width, device=DEV)
    idx = start[:, None] + col
    table = torch.where(col < torch.from_numpy(used).to(DEV)[:, None], order[idx.clamp(max=pool - 1)], -1)
    return table.to(torch.int32), pool


def _pool(case, pool, fill):
    """A cache [pool, page, hkv, d], stored token by token or head by head."""
    hkv, d, page = case["hkv"], case["d"], case["page"]
    shape = (pool, hkv, page, d) if case["head_major"] else (pool, page, hkv, d)
    t = fill(shape)
    return t.transpose(1, 2) if case["head_major"] else t


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    s = {"case": case}
    if case["op"] in ("append", "attention"):
        ql, kl = _lengths(case)
        total = int(ql.sum())
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        s["table"], pool = _pages(case, kl, g)
        s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)).to(DEV)
        s["kv_len"] = torch.from_numpy(kl.astype(np.int32)).to(DEV)
        s["max_q"] = int(ql.max())
        if case["op"] == "append":
            # q, k and v side by side, as a fused projection leaves them
            qkv = normal(total, (hq + 2 * hkv) * d)
            s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
            s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
            s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
            s["q_out"] = torch.zeros((total, hq, d), dtype=torch.bfloat16, device=DEV)
            zeros = lambda shape: torch.zeros(shape, dtype=torch.bfloat16, device=DEV)  # noqa: E731
            s["k_cache"], s["v_cache"] = _pool(case, pool, zeros), _pool(case, pool, zeros)
            j = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
            s["inv_freq"] = 10000.0 ** (-2.0 * j / case["rot"])
        else:
            spread = torch.empty((total, 1, 1), device=DEV).uniform_(0.5, 4.0, generator=g)
            s["q"] = (normal(total, hq, d) * spread).to(torch.bfloat16)
            fill = lambda shape: normal(*shape)  # noqa: E731
            s["k_cache"], s["v_cache"] = _pool(case, pool, fill), _pool(case, pool, fill)
            s["causal"] = torch.full((case["n"],), int(case["causal"]), dtype=torch.uint8, device=DEV)
            s["o"] = torch.zeros((total, hq, d), dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.zeros((total, hq), dtype=torch.float32, device=DEV)
        return s
    n, L, V = case["n"], case["L"], case["V"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    ld = -(-V // 8) * 8
    s["x"] = torch.randn((n, L, ld), generator=g, device=DEV, dtype=dt).mul_(4.0)
    s["out"] = s["x"] if case["in_place"] else torch.zeros((n, L, ld), dtype=dt, device=DEV)
    s["active"] = torch.from_numpy(_active(case)).to(DEV)
    rec = np.zeros((n, 9), np.int32)       # the step's per-canvas records: only the flags matter here
    rec[:, 0] = np.float32(1.0).view(np.int32)
    rec[:, 8] = np.where(_active(case), ACTIVE, 0)
    s["params"] = torch.from_numpy(rec.view(np.uint8).reshape(-1)).to(DEV)
    rng = np.random.default_rng(seed)
    if case["hist"]:
        hl = np.maximum(0, case["hist"] * rng.uniform(0.5, 1.0, n)).astype(np.int64)
        hl[0] = case["hist"]
        s["cu_hist"] = torch.from_numpy(np.concatenate([[0], np.cumsum(hl)]).astype(np.int32)).to(DEV)
        # token frequencies fall off as in text: many repeats of few tokens
        u = torch.rand((int(hl.sum()),), generator=g, device=DEV, dtype=torch.float64)
        s["hist"] = (V ** u).long().clamp(max=V - 1).to(torch.int32)
        pen = np.stack([rng.uniform(1.0, 1.5, n), rng.uniform(0.0, 0.5, n), rng.uniform(0.0, 1.0, n)], 1)
        s["penalties"] = torch.from_numpy(pen.astype(np.float32)).to(DEV)
    if case["bias"]:
        nb = min(case["bias"], V)
        s["cu_bias"] = torch.arange(n + 1, dtype=torch.int32, device=DEV) * nb
        tok = np.stack([rng.permutation(V)[:nb] for _ in range(n)])
        s["bias_tok"] = torch.from_numpy(tok.reshape(-1).astype(np.int32)).to(DEV)
        s["bias_val"] = torch.empty((n * nb,), device=DEV).uniform_(-20.0, 20.0, generator=g)
    M, words = case["masks"], -(-V // 32)
    keep = torch.rand((M, words * 32), generator=g, device=DEV) < case["allowed"]
    keep[:, 0] = True
    shifts = torch.arange(32, device=DEV, dtype=torch.int64)
    bits = (keep.view(M, words, 32).long() << shifts).sum(-1)
    s["masks"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    pick = torch.randint(0, M, (n, L), generator=g, device=DEV, dtype=torch.int32)
    pick[torch.rand((n, L), generator=g, device=DEV) < (0.0 if case["in_place"] else 0.05)] = -1
    s["mask_index"] = pick
    return s


# ------------------------------------------------------------------ plain forms
def _owner(s):
    """Of every packed token: its sequence, its index there and its position."""
    cu = s["cu"].long()
    tok = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    i = tok - cu[seq]
    return seq, i, (s["kv_len"].long() - (cu[1:] - cu[:-1]))[seq] + i


def _rotated(x, pos, w, interleaved):
    """x [t, h, d] in fp32 with its first 2 len(w) dims rotated by pos * w; angles in 64 bits."""
    r = 2 * w.numel()
    ang = pos.double()[:, None] * w[None, :]
    c, sn = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    x = x.float()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * c - b * sn, a * sn + b * c
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y, x[..., r:]], -1).to(torch.bfloat16)


def _plain_append(s):
    case = s["case"]
    seq, _, pos = _owner(s)
    page = s["table"].long()[seq, pos // case["page"]]
    slot = pos % case["page"]
    s["k_cache"][page, slot] = _rotated(s["k"], pos, s["inv_freq"], case["interleaved"])
    s["v_cache"][page, slot] = s["v"]
    s["q_out"].copy_(_rotated(s["q"], pos, s["inv_freq"], case["interleaved"]))


def _plain_attention(s):
    case = s["case"]
    n, d, hkv = case["n"], case["d"], case["hkv"]
    grp = case["hq"] // hkv
    table = s["table"].long().clamp(min=0)
    k = s["k_cache"][table].float().flatten(1, 2)           # [n, keys, hkv, d]
    v = s["v_cache"][table].float().flatten(1, 2)
    cu, kl = s["cu"].long(), s["kv_len"].long()
    ql = cu[1:] - cu[:-1]
    i = torch.arange(s["max_q"], device=DEV)
    j = torch.arange(k.shape[1], device=DEV)
    pos = (kl - ql)[:, None] + i
    hi = pos if case["causal"] else (kl - 1)[:, None].expand_as(pos)
    lo = torch.zeros_like(pos)
    if case["window"] >= 0:
        lo = pos - case["window"]
        hi = torch.minimum(hi, pos + case["window"])
    ok = (j <= hi[..., None]) & (j >= lo[..., None]) & (j < kl[:, None, None])
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float().unflatten(2, (hkv, grp))
    x = torch.einsum("nqhgd,nkhd->nhgqk", q, k) / math.sqrt(d)
    x = x.masked_fill(~ok[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = (x - m).exp()
    z = x.sum(-1)
    o = torch.einsum("nhgqk,nkhd->nqhgd", x, v) / z.permute(0, 3, 1, 2)[..., None].clamp(min=1e-30)
    lse = (m[..., 0] + z.log()).permute(0, 3, 1, 2)
    seq, at, _ = _owner(s)
    s["o"].copy_(o[seq, at].flatten(1, 2))
    s["lse"].copy_(lse[seq, at].flatten(1, 2))


def _plain_adjust(s):
    case = s["case"]
    n, V = case["n"], case["V"]
    x = s["x"][..., :V]
    y = x.float()
    if "hist" in s:
        c = torch.searchsorted(s["cu_hist"][1:].contiguous(), torch.arange(s["hist"].numel(), device=DEV, dtype=torch.int32), right=True)
        count = torch.zeros((n, V), device=DEV)
        count.index_put_((c, s["hist"].long()), torch.ones((), device=DEV), accumulate=True)
        count = count[:, None, :]
        rep, freq, pres = (s["penalties"][:, k, None, None] for k in range(3))
        y = torch.where(count > 0, torch.where(y > 0, y / rep, y * rep) - freq * count - pres, y)
    if "bias_tok" in s:
        c = torch.searchsorted(s["cu_bias"][1:].contiguous(), torch.arange(s["bias_tok"].numel(), device=DEV, dtype=torch.int32), right=True)
        bias = torch.zeros((n, V), device=DEV)
        bias.index_put_((c, s["bias_tok"].long()), s["bias_val"], accumulate=True)
        y = y + bias[:, None, :]
    bit = torch.arange(32, device=DEV, dtype=torch.int32)
    allowed = ((s["masks"][..., None] >> bit) & 1).bool().flatten(1)[:, :V]
    pick = s["mask_index"].long()
    y = y.masked_fill(~(allowed[pick.clamp(min=0)] | (pick < 0)[..., None]), -math.inf)
    s["out"][..., :V] = torch.where(s["active"][:, None, None], y.to(x.dtype), s["out"][..., :V])


def run(s):
    case = s["case"]
    if own:
        import entropy_bounded_denoising_gb300 as dg
    if case["op"] == "append":
        if own:
            dg.dg_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"],
                            inv_freq=s["inv_freq"], interleaved=case["interleaved"], q=s["q"], q_out=s["q_out"])
        else:
            _plain_append(s)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if case["op"] == "attention":
        if own:
            if "workspace" not in s:       # scratch that a program keeps beside its cache
                need = dg.dg_paged_attention_workspace_bytes(case["n"], s["max_q"], case["hq"], case["hkv"], case["d"])
                s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
            dg.dg_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["o"], s["table"], s["cu"], s["kv_len"],
                                  s["causal"], s["max_q"], lse=s["lse"], window=case["window"], workspace=s["workspace"])
        else:
            _plain_attention(s)
        return {"o": s["o"], "lse": s["lse"]}
    if own:
        dg.dg_adjust_logits(s["x"], s["params"], s["out"], history=s.get("hist"), cu_history=s.get("cu_hist"),
                            penalties=s.get("penalties"), bias_tokens=s.get("bias_tok"), bias_values=s.get("bias_val"),
                            cu_bias=s.get("cu_bias"), masks=s["masks"], mask_index=s["mask_index"], V=case["V"])
    else:
        _plain_adjust(s)
    return {"logits": s["out"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_append(s):
    case = s["case"]
    ql, kl = _lengths(case)
    r = case["rot"]
    w = torch.tensor([10000.0 ** (-2.0 * j / r) for j in range(r // 2)], dtype=torch.float64, device=DEV)
    first = torch.arange(r // 2, device=DEV) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else r // 2)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    qo = s["q"].double()
    table = s["table"].cpu().numpy()
    at = 0
    for b in range(case["n"]):
        rows = slice(at, at + int(ql[b]))
        at += int(ql[b])
        p = np.arange(kl[b] - ql[b], kl[b])
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           torch.from_numpy(p).to(DEV).double()[:, None] * w)[:, None, :]

        def rotate(x):
            y = x.clone()
            z = torch.complex(x[..., first], x[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return y

        page = torch.from_numpy(table[b][p // case["page"]].astype(np.int64)).to(DEV)
        slot = torch.from_numpy(p % case["page"]).to(DEV)
        kc[page, slot] = rotate(s["k"][rows].double())
        vc[page, slot] = s["v"][rows].double()
        qo[rows] = rotate(s["q"][rows].double())
    return {"q": qo, "k_cache": kc, "v_cache": vc}


def _exact_attention(s):
    case = s["case"]
    ql, kl = _lengths(case)
    hq, hkv, d, W = case["hq"], case["hkv"], case["d"], case["window"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    at = 0
    for b in range(case["n"]):
        a, m = int(ql[b]), int(kl[b])
        where = s["table"][b, :-(-m // case["page"])].long()
        k = s["k_cache"][where].reshape(-1, hkv, d)[:m].double()
        v = s["v_cache"][where].reshape(-1, hkv, d)[:m].double()
        dist = torch.arange(m, device=DEV)[None, :] - torch.arange(m - a, m, device=DEV)[:, None]  # key - query
        out = dist > 0 if case["causal"] else torch.zeros_like(dist, dtype=torch.bool)
        if W >= 0:
            out = out | (dist.abs() > W)
        for h in range(hq):
            x = s["q"][at:at + a, h].double() @ k[:, h * hkv // hq].T / d ** 0.5
            x[out] = -math.inf
            z = torch.logsumexp(x, 1)
            lse[at:at + a, h] = z
            o[at:at + a, h] = (x - z[:, None]).exp() @ v[:, h * hkv // hq]
        at += a
    return {"o": o, "lse": lse}


def _exact_adjust(s):
    case = s["case"]
    n, L, V = case["n"], case["L"], case["V"]
    res = s["out"].double()
    words = s["masks"].cpu().numpy().view(np.uint8)
    table = torch.from_numpy(np.unpackbits(words, axis=1, bitorder="little")[:, :V].astype(bool)).to(DEV)
    cuh = s["cu_hist"].tolist() if "hist" in s else None
    cub = s["cu_bias"].tolist() if "bias_tok" in s else None
    for c in np.nonzero(_active(case))[0].tolist():
        y = s["x"][c, :, :V].double()
        if cuh:
            times = torch.bincount(s["hist"][cuh[c]:cuh[c + 1]].long(), minlength=V).double()
            rep, freq, pres = s["penalties"][c].double()
            seen = torch.nonzero(times)[:, 0]
            z = y[:, seen]
            y[:, seen] = torch.maximum(z, torch.zeros_like(z)) / rep + torch.minimum(z, torch.zeros_like(z)) * rep \
                - freq * times[seen] - pres
        if cub:
            t = s["bias_tok"][cub[c]:cub[c + 1]].long()
            y[:, t] += s["bias_val"][cub[c]:cub[c + 1]].double()
        for i, m in enumerate(s["mask_index"][c].tolist()):
            if m >= 0:
                y[i][~table[m]] = -math.inf
        res[c, :, :V] = y
    return {"logits": res}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "adjust": _exact_adjust}[case["op"]](s)
