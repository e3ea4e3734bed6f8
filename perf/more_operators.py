"""The operators of a drafting pass over the paged cache, as cases to be timed: queries and keys normed
for each head, rotated by given positions and appended (``dg_kv_append_norm``), attention for trees of
drafted tokens (``dg_tree_attention``) and through a sliding window with first tokens that stay visible
(``dg_sink_attention``), verification of the drafts against the target's probabilities from given
random numbers (``dg_verify_drafts``), and the accepted path kept in the cache (``dg_kv_keep``).  Each
has its plain form in elementary torch operations."""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one step of 64 causal requests, a new token each: latency counts
        dict(name="norm 64 tokens", op="norm", n=64, q=1, kv=1024, hq=16, hkv=8, d=128, rot=128, page=16,
             head_major=False, interleaved=False, tree=False),
        # trees of 61 drafts, each rotated by its depth, wide heads of which half turns
        dict(name="norm trees of 32", op="norm", n=32, q=61, kv=800, hq=16, hkv=4, d=256, rot=128, page=32,
             head_major=True, interleaved=True, tree=True),
        # ragged prompts
        dict(name="norm ragged prompts", op="norm", n=33, q=1531, kv=1531, hq=16, hkv=8, d=128, rot=128, page=64,
             head_major=False, interleaved=False, tree=False),
        # one request's small tree: the latency of the call
        dict(name="tree of 1, 8 nodes, 1k keys", op="tree", n=1, q=8, kv=1024, hq=16, hkv=8, d=128, page=16,
             window=-1, sinks=0, head_major=False),
        # a batch of requests with trees of 64 nodes over long contexts
        dict(name="trees of 32, 64 nodes, 4k keys", op="tree", n=32, q=64, kv=4096, hq=16, hkv=8, d=128, page=16,
             window=-1, sinks=0, head_major=False),
        # wide heads, an odd group and tree, a sliding window over the context
        dict(name="trees of 9, 199 nodes, window", op="tree", n=9, q=199, kv=9001, hq=20, hkv=4, d=256, page=64,
             window=2500, sinks=0, head_major=True),
        # a step of 64 requests through a window, the first tokens in sight
        dict(name="tokens of 64, window and sinks", op="sink", n=64, q=1, kv=8192, hq=16, hkv=8, d=128, page=16,
             window=1024, sinks=4, head_major=False),
        # prompts that go on behind a long context
        dict(name="prompts of 2, window and sinks", op="sink", n=2, q=4000, kv=8000, hq=8, hkv=4, d=64, page=64,
             window=1500, sinks=70, head_major=False),
        # one request's chain of 5 drafts with the draft model's probabilities, small vocabulary
        dict(name="verify 1 chain of 5, 32k", op="verify", n=1, q=6, V=32768, dtype="bf16", tree=False, probs=True),
        # a batch of trees, drafts without probabilities, large vocabulary; some requests greedy
        dict(name="verify 64 trees of 32, 262k", op="verify", n=64, q=32, V=262144, dtype="bf16", tree=True,
             probs=False),
        # one request's accepted path, every layer's cache in one call
        dict(name="keep 1 path, 12 layers", op="keep", n=1, q=16, kv=100, hkv=8, d=128, page=16, layers=12,
             head_major=False),
        # a batch of trees
        dict(name="keep 250 paths, 8 layers", op="keep", n=250, q=61, kv=90, hkv=8, d=128, page=32, layers=8,
             head_major=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "tree", "tree", "sink", "verify", "verify", "keep"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([8, 16, 32, 64, 128])
    major = rng.random() < 0.5
    if op == "norm":
        tree = rng.random() < 0.5
        q = _log(rng, 2, 200) if tree else rng.choice([1, _log(rng, 2, 1500)])
        n = max(1, min(_log(rng, 1, 256), 30000 // q))
        return dict(op=op, n=n, q=q, kv=q + _log(rng, 1, 900), hq=hkv * rng.choice([1, 2, 4]), hkv=hkv, d=d,
                    rot=rng.choice([d, d // 2, 0]), page=page, head_major=major, interleaved=rng.random() < 0.5, tree=tree)
    if op == "tree":
        q = _log(rng, 1, 220)
        kv = q + _log(rng, 1, 9000)
        n = max(1, min(_log(rng, 1, 64), (32 * 4096 * 8 * 128) // (kv * hkv * d), (1 << 28) // (kv * q * hkv * group)))
        w = rng.choice([-1, -1, _log(rng, 200, 4000)])
        return dict(op=op, n=n, q=q, kv=kv, hq=hkv * group, hkv=hkv, d=d, page=page, window=w,
                    sinks=rng.choice([0, _log(rng, 1, 100)]) if w >= 0 else 0, head_major=major)
    if op == "sink":
        q = rng.choice([1, 1, _log(rng, 2, 3000)])
        kv = q + _log(rng, 1, 9000)
        n = max(1, min(_log(rng, 1, 200), (64 * 8192 * 8 * 128) // (kv * hkv * d), (1 << 28) // (kv * q * hkv * group)))
        return dict(op=op, n=n, q=q, kv=kv, hq=hkv * group, hkv=hkv, d=d, page=page, window=_log(rng, 16, 4000),
                    sinks=_log(rng, 1, 150), head_major=major)
    if op == "verify":
        tree = rng.random() < 0.5
        V = _log(rng, 1000, 262144)
        q = _log(rng, 1, 64) if tree else rng.randint(1, 9)
        n = max(1, min(_log(rng, 1, 100), (1 << 29) // (q * V)))
        return dict(op=op, n=n, q=q, V=V, dtype=rng.choice(["bf16", "fp32"]), tree=tree, probs=not tree and rng.random() < 0.7)
    q = _log(rng, 1, 200)
    layers = rng.randint(1, 12)
    n = max(1, min(_log(rng, 1, 250), (250 * 90 * 8 * 8 * 128) // ((q + 100) * layers * hkv * d)))
    return dict(op=op, n=n, q=q, kv=q + rng.randint(0, 100), hkv=hkv, d=d, page=page, layers=layers, head_major=major)


def _lengths(case):
    """Ragged (q_len, kv_len) of a case's sequences, the first one the longest; part of the case, not of
    the seed."""
    rng = np.random.default_rng(case["n"] * 1000003 + case["kv"])
    n, q, kv = case["n"], case["q"], case["kv"]
    ql = np.full(n, q) if q <= 8 or q == 64 else np.maximum(1, q * rng.uniform(0.5, 1.0, n)).astype(np.int64)
    ctx = ((kv - q) * rng.uniform(0.3, 1.0, n)).astype(np.int64)
    ql[0], ctx[0] = q, kv - q
    return ql, ql + ctx


def _rows(case):
    """Rows of logits that a sequence's walk has to read on average, by the inputs' making: the root's, and
    one more for every draft accepted (0.7 of those of a chain with probabilities, fewer without)."""
    depth = min(case["q"] - 1, 8)
    a = 0.7 if case["probs"] else 0.4
    return sum(a ** i for i in range(depth + 1))


def work(case):
    if case["op"] == "norm":
        total = int(_lengths(case)[0].sum())
        one = total * (case["hq"] + 2 * case["hkv"]) * case["d"]
        return {"bytes": 2.0 * 2 * one, "flops": total * (case["hq"] + case["hkv"]) * (4.0 * case["d"] + 3.0 * case["rot"])}
    if case["op"] in ("tree", "sink"):
        ql, kl = _lengths(case)
        total = int(ql.sum())
        W = case["window"]
        keys = pairs = 0
        for a, b in zip(ql.tolist(), kl.tolist()):
            c = b - a
            if case["op"] == "tree":       # every node: the context, and its ancestors (some six of them)
                seen = c if W < 0 else min(c, W + case["sinks"])
                keys += seen + a
                pairs += a * (seen + min(a, 6))
            else:
                pos = np.arange(c, b)
                lo = np.maximum(0, pos - W)
                keys += int(b - lo[0] + min(case["sinks"], lo[0]))
                pairs += int((pos - lo + 1 + np.minimum(case["sinks"], lo)).sum())
        return {"bytes": 4.0 * keys * case["hkv"] * case["d"] + 4.0 * total * case["hq"] * case["d"] + 4.0 * total * case["hq"],
                "flops": 4.0 * pairs * case["hq"] * case["d"]}
    if case["op"] == "verify":
        es = 2 if case["dtype"] == "bf16" else 4
        rows = case["n"] * _rows(case)
        return {"bytes": (rows * es + (case["n"] * 4 if case["probs"] else 0)) * case["V"], "flops": 3.0 * rows * case["V"]}
    moved = 2.0 * case["n"]                # drafts of a path that do not lie in their place already
    return {"bytes": moved * case["layers"] * case["hkv"] * case["d"] * 2 * 2 * 2, "flops": 0.0}


# ------------------------------------------------------------------ inputs
def _trees(rng, sizes):
    """Parents, depths and ancestor masks (as Python integers) of random trees, level by level: node 0 is
    the root, the last token that is certain."""
    out = []
    for q in sizes:
        parent, depth, mask = [-1], [0], [1]
        level = [0]
        while len(parent) < q:
            nxt = []
            for p in level:
                for _ in range(rng.choice([0, 1, 2, 2, 4]) if p != level[0] else 3):
                    if len(parent) < q:
                        nxt.append(len(parent))
                        parent.append(p)
                        depth.append(depth[p] + 1)
                        mask.append(mask[p] | 1 << (len(parent) - 1))
            level = nxt
        out.append((parent, depth, mask))
    return out


def _words(masks, width):
    """Masks as rows of `width` 32-bit words."""
    raw = b"".join(m.to_bytes(4 * width, "little") for m in masks)
    return torch.from_numpy(np.frombuffer(raw, dtype=np.int32).reshape(len(masks), width).copy()).to(DEV)


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
    """A cache [(layers,) pool, page, hkv, d], stored token by token or head by head."""
    hkv, d, page = case["hkv"], case["d"], case["page"]
    shape = (pool, hkv, page, d) if case["head_major"] else (pool, page, hkv, d)
    t = fill(((case["layers"],) if "layers" in case else ()) + shape)
    return t.transpose(-2, -3) if case["head_major"] else t


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    s = {"case": case}
    if case["op"] == "verify":
        return _prepare_verify(case, seed, g, rng, s)
    ql, kl = _lengths(case)
    total = int(ql.sum())
    s["table"], pool = _pages(case, kl, g)
    s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)).to(DEV)
    s["kv_len"] = torch.from_numpy(kl.astype(np.int32)).to(DEV)
    s["max_q"] = int(ql.max())
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "norm":
        hq = case["hq"]
        # q, k and v side by side, as a fused projection leaves them
        qkv = normal(total, (hq + 2 * hkv) * d) * 3.0
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        s["q_out"] = torch.zeros((total, hq, d), dtype=torch.bfloat16, device=DEV)
        zeros = lambda shape: torch.zeros(shape, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        s["k_cache"], s["v_cache"] = _pool(case, pool, zeros), _pool(case, pool, zeros)
        s["q_norm"] = torch.rand((d,), generator=g, device=DEV) + 0.5
        s["k_norm"] = torch.rand((d,), generator=g, device=DEV) + 0.5
        j = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
        s["inv_freq"] = 10000.0 ** (-2.0 * j / case["rot"]) if case["rot"] else None
        s["positions"] = None
        if case["tree"]:
            at = [c + x for (_, depth, _), c in zip(_trees(rng, ql.tolist()), (kl - ql).tolist()) for x in depth]
            s["positions"] = torch.tensor(at, dtype=torch.int32, device=DEV)
        return s
    if case["op"] == "keep":
        # an accepted path: its drafts lie where they stay, or behind the slots that the path will fill
        fill = lambda shape: normal(*shape)  # noqa: E731
        s["k_cache"], s["v_cache"] = _pool(case, pool, fill), _pool(case, pool, fill)
        path, count = [], []
        for q in ql.tolist():
            a = min(rng.choice([0, 1, 2, 3, 4, 6]), (q - 1) // 2)
            later = sorted(rng.sample(range(a + 1, q), a)) if a else []
            here = rng.randint(0, a)       # so many stay in place
            keep = [0] + list(range(1, here + 1)) + later[here:]
            path += keep + [-1] * (q - len(keep))
            count.append(a)
        s["path"] = torch.tensor(path, dtype=torch.int32, device=DEV)
        s["count"] = torch.tensor(count, dtype=torch.int32, device=DEV)
        s["new_len"] = torch.zeros(case["n"], dtype=torch.int32, device=DEV)
        return s
    hq = case["hq"]
    spread = torch.empty((total, 1, 1), device=DEV).uniform_(0.5, 4.0, generator=g)
    s["q"] = (normal(total, hq, d) * spread).to(torch.bfloat16)
    fill = lambda shape: normal(*shape)  # noqa: E731
    s["k_cache"], s["v_cache"] = _pool(case, pool, fill), _pool(case, pool, fill)
    s["o"] = torch.zeros((total, hq, d), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((total, hq), dtype=torch.float32, device=DEV)
    if case["op"] == "tree":
        trees = _trees(rng, ql.tolist())
        s["mask"] = _words([m for t in trees for m in t[2]], -(-s["max_q"] // 32))
        at = [c + x for (_, depth, _), c in zip(trees, (kl - ql).tolist()) for x in depth]
        s["positions"] = torch.tensor(at, dtype=torch.int32, device=DEV)
    return s


def _prepare_verify(case, seed, g, rng, s):
    n, V = case["n"], case["V"]
    fixed = random.Random(n * 1000003 + V)     # ragged sizes: part of the case, not of the seed
    sizes = [case["q"]] + [max(1, int(case["q"] * fixed.uniform(0.6, 1.0))) for _ in range(n - 1)]
    cu = np.concatenate([[0], np.cumsum(sizes)])
    total = int(cu[-1])
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    ld = -(-V // 8) * 8
    s["cu"] = torch.from_numpy(cu.astype(np.int32)).to(DEV)
    s["max_q"] = max(sizes)
    s["logits"] = torch.randn((total, ld), generator=g, device=DEV, dtype=dt).mul_(3.0)
    T = [0.0 if rng.random() < 0.2 else rng.uniform(0.4, 1.1) for _ in range(n)]   # some requests are greedy
    s["T"] = torch.tensor(T, device=DEV)
    owner = torch.from_numpy(np.repeat(np.arange(n), sizes)).to(DEV)
    s["u"] = torch.rand((total,), generator=g, device=DEV)
    s["u_next"] = torch.rand((n,), generator=g, device=DEV)
    tokens = torch.randint(0, V, (total,), generator=g, device=DEV, dtype=torch.int32)
    s["parents"] = s["probs"] = None
    if case["tree"]:
        # a node's children are likely tokens of its row, in order, now and then a random one
        trees = _trees(rng, sizes)
        parent = np.concatenate([np.array(t[0]) for t in trees])
        top = s["logits"][:, :V].topk(min(8, V), dim=1).indices.cpu().numpy()
        tok = tokens.cpu().numpy()
        nth = {}
        for i in range(total):
            b = int(np.searchsorted(cu, i, side="right")) - 1
            if parent[i] >= 0:
                p = int(cu[b] + parent[i])
                k = nth.get(p, 0)
                nth[p] = k + 1
                if k < top.shape[1] and rng.random() < 0.8:
                    tok[i] = top[p, k]
        tokens = torch.from_numpy(tok).to(DEV)
        s["parents"] = torch.from_numpy(parent.astype(np.int32)).to(DEV)
    elif total > n:
        # the draft model: the target's logits of the row before, with noise
        row = torch.arange(total, device=DEV)
        before = (row - 1).clamp(min=0)
        q = torch.zeros((total, ld), device=DEV)
        for i in range(0, total, 64):
            k = before[i:i + 64]
            x = s["logits"][k, :V].float()
            x += 0.7 * torch.randn(x.shape, generator=g, device=DEV)
            t = s["T"][owner[i:i + 64]][:, None]
            q[i:i + 64, :V] = (x / t.clamp(min=0.05)).softmax(1)
            noise = torch.rand(x.shape, generator=g, device=DEV).clamp(min=1e-20).log_().neg_()
            tokens[i:i + 64] = (q[i:i + 64, :V] / noise).argmax(1).to(torch.int32)
        if case["probs"]:
            s["probs"] = q
    s["tokens"] = tokens
    s["count"] = torch.zeros(n, dtype=torch.int32, device=DEV)
    s["path"] = torch.zeros(total, dtype=torch.int32, device=DEV)
    s["out"] = torch.zeros(total, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _owner(s):
    """Of every packed token: its sequence, its index there and the slot it has."""
    cu = s["cu"].long()
    tok = torch.arange(int(s["q" if "q" in s else "path"].shape[0]), device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    i = tok - cu[seq]
    if "kv_len" not in s:
        return seq, i, None
    return seq, i, (s["kv_len"].long() - (cu[1:] - cu[:-1]))[seq] + i


def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w


def _rotated(x, pos, w, interleaved):
    """x [t, h, d] in fp32 with its first 2 len(w) dims rotated by pos * w; angles in 64 bits."""
    if w is None:
        return x.to(torch.bfloat16)
    r = 2 * w.numel()
    ang = pos.double()[:, None] * w[None, :]
    c, sn = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * c - b * sn, a * sn + b * c
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y, x[..., r:]], -1).to(torch.bfloat16)


def _plain_norm(s):
    case = s["case"]
    seq, _, at = _owner(s)
    pos = at if s["positions"] is None else s["positions"]
    page = s["table"].long()[seq, at // case["page"]]
    slot = at % case["page"]
    s["k_cache"][page, slot] = _rotated(_normed(s["k"], s["k_norm"]), pos, s["inv_freq"], case["interleaved"])
    s["v_cache"][page, slot] = s["v"]
    s["q_out"].copy_(_rotated(_normed(s["q"], s["q_norm"]), pos, s["inv_freq"], case["interleaved"]))


def _plain_attention(s):
    case = s["case"]
    d, hkv = case["d"], case["hkv"]
    grp = case["hq"] // hkv
    table = s["table"].long().clamp(min=0)
    k = s["k_cache"][table].float().flatten(1, 2)           # [n, keys, hkv, d]
    v = s["v_cache"][table].float().flatten(1, 2)
    cu, kl = s["cu"].long(), s["kv_len"].long()
    ql = cu[1:] - cu[:-1]
    ctx = (kl - ql)[:, None, None]
    i = torch.arange(s["max_q"], device=DEV)
    j = torch.arange(k.shape[1], device=DEV)
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    pos = s["positions"].long()[row] if case["op"] == "tree" else (kl - ql)[:, None] + i
    ok = torch.ones((case["n"], s["max_q"], k.shape[1]), dtype=torch.bool, device=DEV)
    if case["window"] >= 0:
        ok = (j >= (pos - case["window"])[..., None]) | (j < case["sinks"])
    if case["op"] == "tree":
        nth = (j - ctx).clamp(min=0, max=32 * s["mask"].shape[1] - 1).expand_as(ok)
        word = torch.gather(s["mask"][row], 2, nth // 32)
        ok = torch.where(j < ctx, ok, ((word >> (nth % 32).int()) & 1).bool() & (j < kl[:, None, None]))
    else:
        ok = ok & (j <= pos[..., None])
    q = s["q"][row].float().unflatten(2, (hkv, grp))
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


def _plain_verify(s):
    """All rows' statistics in 64 bits (a draw lies next to a token's border now and then), then the nodes in
    order: one is tried where its parent is the node its sequence has come to."""
    case = s["case"]
    n, V = case["n"], case["V"]
    cu = s["cu"].long()
    total = s["path"].shape[0]
    seq, _, _ = _owner(s)
    greedy = s["T"] == 0
    T = torch.where(greedy, torch.ones_like(s["T"]), s["T"]).double()
    lse = torch.empty(total, dtype=torch.float64, device=DEV)
    best = torch.empty(total, dtype=torch.long, device=DEV)
    for i in range(0, total, 256):
        x = s["logits"][i:i + 256, :V].double()
        best[i:i + 256] = x.argmax(1)
        x = x / T[seq[i:i + 256]][:, None]
        m = x.amax(1)
        lse[i:i + 256] = m + (x - m[:, None]).exp().sum(1).log()
    ql = cu[1:] - cu[:-1]
    at = torch.zeros(n, dtype=torch.long, device=DEV)        # the node a sequence has come to
    mass = torch.ones(n, dtype=torch.float64, device=DEV)    # what its rejected children have left
    stop = torch.full((n,), -1, dtype=torch.long, device=DEV)   # the last draft rejected there
    count = torch.zeros(n, dtype=torch.long, device=DEV)
    path = torch.full((total,), -1, dtype=torch.long, device=DEV)
    out = torch.full((total,), -1, dtype=torch.long, device=DEV)
    path[cu[:-1]] = 0
    gone = torch.zeros((n, s["max_q"]), dtype=torch.bool, device=DEV)   # rejected children of the node it is at
    for i in range(1, s["max_q"]):
        row = (cu[:-1] + i).clamp(max=total - 1)
        up = s["parents"][row].long() if s["parents"] is not None else torch.full_like(at, i - 1)
        tried = (i < ql) & (up == at)
        tok = s["tokens"][row].long()
        here = cu[:-1] + at
        p = (s["logits"][here, tok].double() / T - lse[here]).exp()
        twice = (gone & (s["tokens"][(cu[:-1, None] + torch.arange(s["max_q"], device=DEV)).clamp(max=total - 1)].long()
                         == tok[:, None])).any(1)
        p = torch.where(twice, torch.zeros_like(p), p)
        if s["probs"] is not None:
            yes = s["u"][row].double() * s["probs"][row, tok].double() < p
        else:
            yes = s["u"][row].double() * mass < p
        yes = torch.where(greedy, tok == best[here], yes) & tried
        no = tried & ~yes
        mass = torch.where(yes, torch.ones_like(mass), torch.where(no, mass - p, mass))
        stop = torch.where(yes, torch.full_like(stop, -1), torch.where(no, torch.full_like(stop, i), stop))
        gone[:, i] = no
        gone &= ~yes[:, None]
        count = count + yes
        where = (cu[:-1] + count).clamp(max=total - 1)
        path[where] = torch.where(yes, torch.full_like(at, i), path[where])
        before = (cu[:-1] + count - 1).clamp(min=0)
        out[before] = torch.where(yes, tok, out[before])
        at = torch.where(yes, torch.full_like(at, i), at)
    # the token after the path, from what the rejected drafts left
    here = cu[:-1] + at
    w = (s["logits"][here, :V].double() / T[:, None] - lse[here][:, None]).exp()
    if s["probs"] is not None:
        left = (w - s["probs"][cu[:-1] + stop.clamp(min=0), :V].double()).clamp(min=0)
        left = torch.where((stop >= 0)[:, None], left, w)
    else:
        left = w.clone()
        b, i = torch.nonzero(gone, as_tuple=True)
        left[b, s["tokens"][cu[:-1][b] + i].long()] = 0
    w = torch.where(left.sum(1, keepdim=True) > 0, left, w)
    c = w.cumsum(1)
    nxt = (c <= s["u_next"].double()[:, None] * c[:, -1:]).sum(1)
    nxt = torch.where(greedy, best[here], nxt)
    out[cu[:-1] + count] = nxt
    s["count"].copy_(count)
    s["path"].copy_(path)
    s["out"].copy_(out)


def _plain_keep(s):
    case = s["case"]
    cu = s["cu"].long()
    seq, i, _ = _owner(s)
    kept = i <= s["count"].long()[seq]
    seq, i, node = seq[kept], i[kept], s["path"].long()[kept]
    ctx = (s["kv_len"].long() - (cu[1:] - cu[:-1]))[seq]
    page, table = case["page"], s["table"].long()
    to, at = ctx + i, ctx + node
    for c in (s["k_cache"], s["v_cache"]):
        rows = c[:, table[seq, at // page], at % page]
        c[:, table[seq, to // page], to % page] = rows
    s["new_len"].copy_(s["kv_len"].long() - (cu[1:] - cu[:-1]) + s["count"] + 1)


def run(s):
    case = s["case"]
    if own:
        import entropy_bounded_denoising_gb300 as dg
    if case["op"] == "norm":
        if own:
            dg.dg_kv_append_norm(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"],
                                 inv_freq=s["inv_freq"], interleaved=case["interleaved"], q=s["q"], q_out=s["q_out"],
                                 q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, positions=s["positions"])
        else:
            _plain_norm(s)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if case["op"] in ("tree", "sink"):
        if own:
            if "workspace" not in s:       # scratch that a program keeps beside its cache
                need = dg.dg_tree_attention_workspace_bytes(case["n"], s["max_q"], case["hq"], case["hkv"], case["d"])
                s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
            if case["op"] == "tree":
                dg.dg_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["o"], s["table"], s["cu"], s["kv_len"],
                                     s["mask"], s["max_q"], positions=s["positions"], lse=s["lse"],
                                     window=case["window"], sinks=case["sinks"], workspace=s["workspace"])
            else:
                dg.dg_sink_attention(s["q"], s["k_cache"], s["v_cache"], s["o"], s["table"], s["cu"], s["kv_len"],
                                     s["max_q"], window=case["window"], sinks=case["sinks"], lse=s["lse"],
                                     workspace=s["workspace"])
        else:
            _plain_attention(s)
        return {"o": s["o"], "lse": s["lse"]}
    if case["op"] == "verify":
        if own:
            dg.dg_verify_drafts(s["logits"], s["tokens"], s["cu"], s["T"], s["u"], s["u_next"], s["count"], s["path"],
                                s["out"], parents=s["parents"], draft_probs=s["probs"], V=case["V"])
        else:
            _plain_verify(s)
        return {"n_accept": s["count"], "path": s["path"], "tokens": s["out"]}
    if own:
        dg.dg_kv_keep(s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"], s["path"], s["count"], s["new_len"])
    else:
        _plain_keep(s)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "new_len": s["new_len"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_norm(s):
    case = s["case"]
    ql, kl = _lengths(case)
    r = case["rot"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    qo = s["q"].double()
    table = s["table"].cpu().numpy()
    w = torch.tensor([10000.0 ** (-2.0 * j / r) for j in range(r // 2)], dtype=torch.float64, device=DEV) if r else None
    first = torch.arange(r // 2, device=DEV) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else r // 2)
    start = 0
    for b in range(case["n"]):
        rows = slice(start, start + int(ql[b]))
        start += int(ql[b])
        at = np.arange(kl[b] - ql[b], kl[b])
        p = torch.from_numpy(at).to(DEV) if s["positions"] is None else s["positions"][rows]

        def turned(x, weight):
            y = x.double()
            y = y / (y.square().sum(-1, keepdim=True) / case["d"] + 1e-6).sqrt() * weight.double()
            if r:
                turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), p.double()[:, None] * w)[:, None, :]
                z = torch.complex(y[..., first], y[..., second]) * turn
                y[..., first], y[..., second] = z.real, z.imag
            return y

        page = torch.from_numpy(table[b][at // case["page"]].astype(np.int64)).to(DEV)
        slot = torch.from_numpy(at % case["page"]).to(DEV)
        kc[page, slot] = turned(s["k"][rows], s["k_norm"])
        vc[page, slot] = s["v"][rows].double()
        qo[rows] = turned(s["q"][rows], s["q_norm"])
    return {"q": qo, "k_cache": kc, "v_cache": vc}


def _exact_attention(s):
    case = s["case"]
    ql, kl = _lengths(case)
    hq, hkv, d, W = case["hq"], case["hkv"], case["d"], case["window"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    start = 0
    for b in range(case["n"]):
        a, m = int(ql[b]), int(kl[b])
        rows = slice(start, start + a)
        start += a
        where = s["table"][b, :-(-m // case["page"])].long()
        k = s["k_cache"][where].reshape(-1, hkv, d)[:m].double()
        v = s["v_cache"][where].reshape(-1, hkv, d)[:m].double()
        p = s["positions"][rows].long() if case["op"] == "tree" else torch.arange(m - a, m, device=DEV)
        key = torch.arange(m, device=DEV)[None, :]
        out = torch.zeros((a, m), dtype=torch.bool, device=DEV)
        if W >= 0:
            out = (p[:, None] - key > W) & (key >= case["sinks"])
        if case["op"] == "tree":
            words = s["mask"][rows].cpu().numpy().view(np.uint8)
            bits = np.unpackbits(words, axis=1, bitorder="little")[:, :a].astype(bool)
            out[:, m - a:] = torch.from_numpy(~bits).to(DEV)
        else:
            out |= key > p[:, None]
        for h in range(hq):
            x = s["q"][rows, h].double() @ k[:, h * hkv // hq].T / d ** 0.5
            x[out] = -math.inf
            z = torch.logsumexp(x, 1)
            lse[rows, h] = z
            o[rows, h] = (x - z[:, None]).exp() @ v[:, h * hkv // hq]
    return {"o": o, "lse": lse}


def _exact_verify(s):
    case = s["case"]
    V = case["V"]
    cu = s["cu"].tolist()
    T, u, u_next = s["T"].double().tolist(), s["u"].double().tolist(), s["u_next"].double().tolist()
    tokens = s["tokens"].tolist()
    parents = s["parents"].tolist() if s["parents"] is not None else None
    counts, paths, outs = [], [], []
    for b in range(case["n"]):
        lo, q = cu[b], cu[b + 1] - cu[b]
        node, path, out = 0, [0], []
        while True:
            row = s["logits"][lo + node, :V].double().cpu()
            p = torch.softmax(row / T[b], 0) if T[b] else torch.nn.functional.one_hot(row.argmax(), V).double()
            left, moved = p.clone(), False
            for c in range(node + 1, q):
                if (parents[lo + c] if parents else c - 1) != node:
                    continue
                t = tokens[lo + c]
                if T[b] == 0:
                    moved = bool(p[t] == 1)
                elif s["probs"] is not None:
                    moved = u[lo + c] * float(s["probs"][lo + c, t].double()) < float(p[t])
                else:
                    moved = u[lo + c] * float(left.sum()) < float(left[t])
                if moved:
                    node = c
                    path.append(c)
                    out.append(t)
                    break
                if T[b] and s["probs"] is not None:
                    left = torch.clamp(p - s["probs"][lo + c, :V].double().cpu(), min=0)
                elif T[b]:
                    left[t] = 0
            if not moved:
                break
        if float(left.sum()) == 0:
            left = p
        edge = torch.cumsum(left, 0)
        nxt = int(p.argmax()) if T[b] == 0 else int(torch.searchsorted(edge, u_next[b] * float(edge[-1]), right=True))
        counts.append(len(path) - 1)
        paths += path + [-1] * (q - len(path))
        outs += out + [nxt] + [-1] * (q - len(out) - 1)
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"n_accept": whole(counts), "path": whole(paths), "tokens": whole(outs)}


def _exact_keep(s):
    case = s["case"]
    ql, kl = _lengths(case)
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    path, count, table = s["path"].tolist(), s["count"].tolist(), s["table"].tolist()
    start, page = 0, case["page"]
    for b in range(case["n"]):
        ctx = int(kl[b] - ql[b])
        for i in range(count[b] + 1):
            src, dst = ctx + path[start + i], ctx + i
            for new, old in ((kc, s["k_cache"]), (vc, s["v_cache"])):
                new[:, table[b][dst // page], dst % page] = old[:, table[b][src // page], src % page]
        start += int(ql[b])
    new_len = torch.from_numpy((kl - ql + np.array(count) + 1).astype(np.int32)).to(DEV)
    return {"k_cache": kc, "v_cache": vc, "new_len": new_len}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "tree": _exact_attention, "sink": _exact_attention, "verify": _exact_verify,
            "keep": _exact_keep}[case["op"]](s)
