"""Measured cases of a speculative decoding step over the paged KV pool.

Operators (the framework's entry points, each called as a user's program does):
  rope     pa.rope_store_kvcache / pa.rope: per-head norm and rotation of this
           step's q and k, the rotated keys and the values into the pool
  tree     pa.decode_tree: attention of a tree of drafted tokens over the pool
  verify   pa.verify_drafts: which drafted tokens the target keeps, and the
           token that follows them, from given random numbers
  compact  pa.compact_kvcache: the kept tokens' rows moved next to the context

Definitions.

rope: a head x of 128 values, optionally x * rsqrt(mean(x^2) + eps) * weight;
then the first R values are rotated in pairs, (i, i + R/2) or (2i, 2i + 1), by
the angle position * f_i, and scaled by g.  f_i = theta^(-2i/R), g = 1;
"linear": f_i / s; "ntk": theta * s^(R/(R-2)) for theta; "yarn": f_i/s for
pairs of long wavelength, f_i for short ones, a ramp between, g = 0.1 ln s + 1.

tree: context_lens counts all keys of a sequence, its n drafted tokens the
last ones.  Draft i sees the keys before the drafts, and draft j where bit j of
tree_mask[b, i] is set.

verify: node 0 is the token that the drafts continue, node i > 0 a drafted
token with parent parents[b, i] < i.  logits[b, v] are the target's at node v,
draft_probs[b, v] the distribution that v's children were drawn from.  At a
node, with w = p = softmax(logits / T) and s = 1: its children in order, child c
with token x is kept if u_c * q(x) * s < w(x); else w = max(w - s q, 0) and
s = sum w.  Without draft_probs (chosen candidates): kept if u_c * s < w(x), else
w(x) = 0.  From a kept child on the same way; where no child is kept the last
token is argmax w / max(E, 1e-10) (p for w where nothing is left of w).
"""
import math

import torch

own = False

D = 128
EPS = 1e-6


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # The new tokens of a decode step, inside the fused QKV projection, with the norms of q and k.
        {"name": "rope store decode b64", "op": "rope", "tokens": 64, "hq": 32, "hkv": 8, "rotary": 128,
         "interleaved": False, "scaling": "none", "factor": 1.0, "theta": 1e6, "far": 8192, "norm": True, "store": True,
         "block": 256, "pad": 0.0, "fused": True},
        # Part of the head, neighbouring pairs, a padded batch, small blocks.
        {"name": "rope store 333 part of head", "op": "rope", "tokens": 333, "hq": 8, "hkv": 2, "rotary": 64,
         "interleaved": True, "scaling": "linear", "factor": 4.0, "theta": 1e4, "far": 16000, "norm": False,
         "store": True, "block": 16, "pad": 0.15, "fused": False},
        # A whole prefill step, positions of a scaled long context.
        {"name": "rope store prefill 16384", "op": "rope", "tokens": 16384, "hq": 32, "hkv": 8, "rotary": 128,
         "interleaved": False, "scaling": "yarn", "factor": 4.0, "theta": 1e6, "far": 131072, "norm": True,
         "store": True, "block": 256, "pad": 0.0, "fused": True},
        # A few short sequences, a small tree each.
        {"name": "tree tiny b4 x5", "op": "tree", "batch": 4, "drafts": 5, "hq": 16, "hkv": 8, "block": 256,
         "lens": "uniform", "lo": 1, "hi": 600, "shape": "tree", "ragged": False},
        # Decode batches of the benchmark, with drafted tokens: a ragged tree, a chain.
        {"name": "tree qwen3-0.6b b64 x8", "op": "tree", "batch": 64, "drafts": 8, "hq": 16, "hkv": 8, "block": 256,
         "lens": "uniform", "lo": 1, "hi": 4096, "shape": "tree", "ragged": True},
        {"name": "tree qwen3-8b b256 x4 chain", "op": "tree", "batch": 256, "drafts": 4, "hq": 32, "hkv": 8,
         "block": 256, "lens": "lognormal", "lo": 1, "hi": 8192, "shape": "chain", "ragged": False},
        # Large trees over long contexts.
        {"name": "tree long b8 32k x64", "op": "tree", "batch": 8, "drafts": 64, "hq": 32, "hkv": 8, "block": 256,
         "lens": "uniform", "lo": 32768, "hi": 32768, "shape": "tree", "ragged": False},
        # One sequence's chain of drafts, fp32 logits, an odd vocabulary.
        {"name": "verify 1 x5 chain fp32", "op": "verify", "batch": 1, "nodes": 5, "vocab": 32003, "dtype": "fp32",
         "probs": True, "shape": "chain", "temps": False, "ragged": False},
        # A batch's chains over the Qwen3 vocabulary, under the sampling temperatures.
        {"name": "verify 64 x6 chain bf16", "op": "verify", "batch": 64, "nodes": 6, "vocab": 151936, "dtype": "bf16",
         "probs": True, "shape": "chain", "temps": True, "ragged": False},
        # Trees of chosen candidates, of different sizes.
        {"name": "verify 32 x32 tree bf16", "op": "verify", "batch": 32, "nodes": 32, "vocab": 151936, "dtype": "bf16",
         "probs": False, "shape": "tree", "temps": True, "ragged": True},
        # What a verified step leaves to move: one layer's small pool, all layers of a batch.
        {"name": "compact b4 x8 one layer", "op": "compact", "batch": 4, "layers": 1, "nodes": 8, "hkv": 8,
         "block": 16, "lo": 1, "hi": 600},
        {"name": "compact b64 x16 28 layers", "op": "compact", "batch": 64, "layers": 28, "nodes": 16, "hkv": 8,
         "block": 256, "lo": 1, "hi": 600},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "tree", "verify", "compact"])
    block = rng.choice([16, 32, 48, 64, 128, 256, 512])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    if op == "rope":
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "hq": hkv * min(group, 32 // hkv), "hkv": hkv,
                "rotary": rng.choice([32, 64, 96, 128]), "interleaved": rng.random() < 0.5, "scaling": scaling,
                "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]), "theta": rng.choice([1e4, 1e6]),
                "far": _log_int(rng, 64, 1 << 20), "norm": rng.random() < 0.5, "store": rng.random() < 0.7,
                "block": block, "pad": rng.choice([0.0, 0.1, 0.5]), "fused": rng.random() < 0.5}
    if op == "tree":
        hi, drafts = _log_int(rng, 1, 32768), _log_int(rng, 1, 64)
        hq = hkv * min(group, 32 // hkv)
        most = min(256, 262144 // hi, (64 * 32 * 262144) // (hi * drafts * hq))
        return {"op": op, "batch": _log_int(rng, 1, max(1, most)), "drafts": drafts, "hq": hq, "hkv": hkv,
                "block": block, "lens": "uniform", "lo": rng.choice([0, 1, hi]), "hi": hi,
                "shape": rng.choice(["tree", "chain"]), "ragged": rng.random() < 0.5}
    if op == "verify":
        vocab, nodes = _log_int(rng, 500, 200000), _log_int(rng, 2, 40)
        return {"op": op, "batch": _log_int(rng, 1, max(1, min(256, 150_000_000 // (vocab * nodes)))), "nodes": nodes,
                "vocab": vocab, "dtype": rng.choice(["bf16", "fp32"]), "probs": rng.random() < 0.5,
                "shape": rng.choice(["tree", "chain"]), "temps": rng.random() < 0.7, "ragged": rng.random() < 0.5}
    hi = _log_int(rng, 1, 2000)
    layers = _log_int(rng, 1, 40)
    return {"op": op, "batch": _log_int(rng, 1, max(1, min(256, 400_000 // (hi * layers)))), "layers": layers,
            "nodes": _log_int(rng, 2, 64), "hkv": hkv, "block": block, "lo": rng.choice([0, hi]), "hi": hi}


def _lens(case, seed):
    """Keys before the drafts (on the host): the same for every seed up to their order."""
    g = torch.Generator().manual_seed(1000 + case["batch"])
    if case.get("lens") == "lognormal":
        n = torch.exp(torch.randn(case["batch"], generator=g)) * 1024
        n = n.round().clamp(case["lo"], case["hi"]).long()
    else:
        n = torch.randint(case["lo"], case["hi"] + 1, (case["batch"],), generator=g)
    g.manual_seed(seed)
    return n[torch.randperm(case["batch"], generator=g)]


def _counts(case, size, seed):
    """Tokens in each sequence's tree: the same for every seed up to their order."""
    if not case.get("ragged"):
        return torch.full((case["batch"],), size)
    g = torch.Generator().manual_seed(2000 + case["batch"])
    n = torch.randint(1, size + 1, (case["batch"],), generator=g)
    g.manual_seed(seed + 3)
    return n[torch.randperm(case["batch"], generator=g)]


def work(case):
    op = case["op"]
    if op == "rope":
        values = case["tokens"] * (case["hq"] + 2 * case["hkv"]) * D
        return {"bytes": 4 * values + 8 * case["tokens"], "flops": 8 * values}
    if op == "tree":
        # Sequence by sequence, with the tree's own keys; lengths and tree sizes meet in the order of seed 0.
        n = _counts(case, case["drafts"], 0)
        keys = _lens(case, 0) + n
        return {"bytes": 4 * int(keys.sum()) * case["hkv"] * D + 4 * int(n.sum()) * case["hq"] * D,
                "flops": 4 * D * case["hq"] * int((n * keys).sum())}
    if op == "verify":
        # The rows of the nodes that are reached (about four with drawn drafts, two with chosen candidates, as
        # these inputs are), one row of draws, and a row of draft probabilities where one is subtracted.
        reach = min(case["nodes"], 4 if case["probs"] else 2)
        size = 4 if case["dtype"] == "fp32" else 2
        a_seq = case["vocab"] * (reach * size + 4 + (4 if case["probs"] else 0))
        return {"bytes": case["batch"] * a_seq, "flops": case["batch"] * case["vocab"] * 4 * (reach + 1)}
    moved = case["batch"] * min(case["nodes"] - 1, 3)
    return {"bytes": moved * case["layers"] * 4 * case["hkv"] * 2 * D, "flops": 0}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _rand(shape, g):
    return torch.rand(shape, generator=g, device="cuda")


def _pool(shape, g):
    """A pool as earlier steps left it: rows in every slot, a few loud channels."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    x[..., 5] *= 4
    return x


def _tables(lens, block, seed):
    """Scattered block tables (-1 past a sequence's blocks) and the pool size."""
    g = torch.Generator().manual_seed(seed + 1)
    counts = -(-lens // block)
    need = int(counts.sum())
    blocks = max(1, math.ceil(1.1 * need))
    perm = torch.randperm(blocks, generator=g)[:need].to(torch.int32)
    width = max(1, int(counts.max()))
    bt = torch.full((len(lens), width), -1, dtype=torch.int32)
    bt[torch.arange(width)[None, :] < counts[:, None]] = perm
    return bt, blocks


def _parents(batch, n, shape, seed):
    """Parents of the tree's tokens: a chain, or each token under one of the few before it."""
    i = torch.arange(n).expand(batch, n)
    if shape == "chain":
        return (i - 1).to(torch.int32)
    g = torch.Generator().manual_seed(seed + 2)
    back = 1 + (torch.rand(batch, n, generator=g) * torch.minimum(i, torch.full_like(i, 4))).long()
    return (i - back).to(torch.int32)


def _masks(parents):
    """Bit j of [b, i]: j is i or an ancestor of i; int64."""
    batch, n = parents.shape
    m = torch.zeros(batch, n, dtype=torch.int64)
    rows = torch.arange(batch)
    for i in range(n):
        m[:, i] = (m[rows, parents[:, i].long()] if i else 0) | (-1 << 63 if i == 63 else 1 << i)
    return m


def _frequencies(case):
    """f_i in 64 bits, and g."""
    r, theta, s = case["rotary"], case["theta"], case["factor"]
    i = torch.arange(r // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        theta = theta * s ** (r / (r - 2))
    f = theta ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] == "yarn":
        at = lambda turns: r * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / s * ramp, 0.1 * math.log(s) + 1.0
    return f, 1.0


ORIGINAL = 32768  # the context that a yarn-scaled model was trained on


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "rope":
        n, hq, hkv, block = case["tokens"], case["hq"], case["hkv"], case["block"]
        if case["fused"]:  # rows inside the fused QKV projection's output
            qkv = _randn((n, hq + 2 * hkv, D), g).to(torch.bfloat16)
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            q, k, v = (_randn((n, h, D), g).to(torch.bfloat16) for h in (hq, hkv, hkv))
        s = {"op": op, "q": q, "k": k, "v": v, "store": case["store"], "interleaved": case["interleaved"],
             "pos": torch.randint(0, case["far"], (n,), generator=g, device="cuda").to(torch.int32)}
        f, s["g"] = _frequencies(case)
        s["f"] = f.cuda()
        s["wq"], s["wk"] = ((1 + 0.2 * _randn((2, D), g)).to(torch.bfloat16) if case["norm"] else (None, None))
        if case["store"]:
            blocks = -(-n // block) + 7
            s["slots"] = torch.randperm(blocks * block, generator=g, device="cuda")[:n].to(torch.int32)
            s["slots"][_rand(n, g) < case["pad"]] = -1
            s["kc"], s["vc"] = (_pool((blocks, block, hkv, D), g) for _ in range(2))
        if own:  # the frequencies that a serving program keeps
            import paged_kv_cache_store_gb300 as pa
            kind = {"none": None, "yarn": ("yarn", case["factor"], ORIGINAL)}
            s["rope"] = pa.rope_frequencies(case["rotary"], case["theta"], interleaved=case["interleaved"],
                                            scaling=kind.get(case["scaling"], (case["scaling"], case["factor"])))
        return s
    if op == "tree":
        batch, t, hq, hkv, block = case["batch"], case["drafts"], case["hq"], case["hkv"], case["block"]
        n = _counts(case, t, seed)
        ctx = _lens(case, seed) + n
        bt, blocks = _tables(ctx, block, seed)
        s = {"op": op, "q": _randn((batch, t, hq, D), g).to(torch.bfloat16), "bt": bt.cuda(),
             "ctx": ctx.to(torch.int32).cuda(), "n": n.to(torch.int32).cuda(),
             "mask": _masks(_parents(batch, t, case["shape"], seed)).cuda(), "scale": 1.0 / math.sqrt(D)}
        s["kc"], s["vc"] = (_pool((blocks, block, hkv, D), g) for _ in range(2))
        if own:  # the split workspace that a serving program keeps
            import paged_kv_cache_store_gb300 as pa
            s["ws"] = pa.decode_tree_workspace(hq, hkv, D, t, device="cuda")
        return s
    if op == "verify":
        batch, n, vocab = case["batch"], case["nodes"], case["vocab"]
        dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        parents = _parents(batch, n, case["shape"], seed)
        p = parents.cuda().long()
        wide = -(-vocab // 8) * 8
        logits = torch.empty((batch, n, wide), dtype=dtype, device="cuda")[..., :vocab]
        probs = torch.empty((batch, n, wide), device="cuda")[..., :vocab] if case["probs"] else None
        temps = _rand(batch, g) * 0.7 + 0.5 if case["temps"] else torch.ones(batch, device="cuda")
        tokens = torch.zeros((batch, n), dtype=torch.int64, device="cuda")
        for v in range(n):  # target logits, a draft model's near them, and the children that it proposes
            x = _randn((batch, vocab), g) * 2.0
            hot = torch.randint(0, vocab, (batch, 16), generator=g, device="cuda")
            x.scatter_add_(1, hot, 6.0 + 3.0 * _randn((batch, 16), g))
            logits[:, v] = x.to(dtype)
            x = (x + 0.5 * _randn((batch, vocab), g)) / temps[:, None]
            if case["probs"]:  # drawn, each child on its own
                q = torch.softmax(x, -1)
                probs[:, v] = q
                picks = torch.multinomial(q, n, replacement=True, generator=g)
            else:  # the likeliest ones
                picks = x.topk(min(n, vocab), -1).indices
            child = p == v
            child[:, 0] = False
            rank = (child.long().cumsum(1) - 1).clamp(0, picks.shape[1] - 1)
            tokens = torch.where(child, picks.gather(1, rank), tokens)
        return {"op": op, "logits": logits, "tokens": tokens.to(torch.int32), "parents": parents.cuda(),
                "u": _rand((batch, n), g), "noise": _pad_rows(-torch.log1p(-_rand((batch, vocab), g))),
                "temps": temps, "probs": probs, "n": _counts(case, n, seed).to(torch.int32).cuda()}
    batch, layers, t, block = case["batch"], case["layers"], case["nodes"], case["block"]
    ctx = _lens(case, seed) + t
    bt, blocks = _tables(ctx, block, seed)
    parents = _parents(batch, t, "tree", seed)
    h = torch.Generator().manual_seed(seed + 5)
    nodes, counts = torch.full((batch, t), -1, dtype=torch.int32), torch.zeros(batch, dtype=torch.int32)
    for b in range(batch):  # a path from the root, as verification keeps one
        path, v = [0], 0
        for c in range(1, t):
            if int(parents[b, c]) == v and float(torch.rand((), generator=h)) < 0.7:
                path.append(c)
                v = c
        nodes[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
        counts[b] = len(path)
    s = {"op": op, "bt": bt.cuda(), "ctx": ctx.to(torch.int32).cuda(), "nodes": nodes.cuda(), "counts": counts.cuda()}
    s["kc"], s["vc"] = (_pool((layers, blocks, block, case["hkv"], D), g) for _ in range(2))
    return s


def _pad_rows(x):
    """x with rows a multiple of 16 bytes apart."""
    wide = torch.empty((x.shape[0], -(-x.shape[1] // 8) * 8), dtype=x.dtype, device=x.device)[:, :x.shape[1]]
    wide.copy_(x)
    return wide


# --------------------------------------------------------------------------
# The plain forms
# --------------------------------------------------------------------------

def _plain_heads(x, s, weight, cos, sin):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    r = 2 * cos.shape[-1]
    if s["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., r:]), -1).to(torch.bfloat16)


def _plain_rope(s):
    angle = s["pos"].double()[:, None, None] * s["f"]  # far positions need 64 bits
    cos, sin = ((t * s["g"]).float() for t in (torch.cos(angle), torch.sin(angle)))
    q, k = _plain_heads(s["q"], s, s["wq"], cos, sin), _plain_heads(s["k"], s, s["wk"], cos, sin)
    if not s["store"]:
        return {"q": q, "k": k}
    keep = s["slots"] >= 0
    slots = s["slots"][keep].long()
    s["kc"].flatten(0, 1)[slots] = k[keep]
    s["vc"].flatten(0, 1)[slots] = s["v"][keep]
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _plain_tree(s):
    batch, t, hq, _ = s["q"].shape
    block, hkv = s["kc"].shape[1:3]
    width = s["bt"].shape[1] * block
    out = torch.empty_like(s["q"])
    # A few sequences at a time: fp32 rows and scores of all of them would not fit.
    step = max(1, (1 << 32) // (4 * width * (2 * hkv * D + 2 * t * hq)))
    pos = torch.arange(width, device="cuda")
    for i in range(0, batch, step):
        part = slice(i, i + step)
        bt, n = s["bt"][part].long().clamp_min(0), s["n"][part, None].long()
        first = s["ctx"][part, None].long() - n  # keys before the drafts
        k, v = (c[bt].flatten(1, 2).transpose(1, 2).float() for c in (s["kc"], s["vc"]))
        b = len(bt)
        j = pos[None] - first
        bit = (s["mask"][part][:, :, None] >> j.clamp(0, 63)[:, None]) & 1
        sees = (j < 0)[:, None] | ((j < n)[:, None] & (j >= 0)[:, None] & (bit == 1))  # [b, t, width]
        sees = sees & (torch.arange(t, device="cuda")[None] < n)[:, :, None]
        v = v.masked_fill((j >= n)[:, None, :, None], 0.0)
        q = s["q"][part].float().view(b, t, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4)
        x = torch.matmul(q.reshape(b, hkv, -1, D), k.transpose(2, 3)) * s["scale"]
        x = x.view(b, hkv, hq // hkv, t, width).masked_fill(~sees[:, None, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
        l = e.sum(-1, keepdim=True)
        o = torch.matmul(e.flatten(2, 3), v).view(b, hkv, hq // hkv, t, D) / torch.where(l == 0, torch.ones_like(l), l)
        out[part] = o.permute(0, 3, 1, 2, 4).reshape(b, t, hq, D).to(torch.bfloat16)
    return out


def _plain_verify(s):
    # 64 bits: a token is kept or not by a comparison, and drawn by another.
    batch, nodes, vocab = s["logits"].shape
    rows = torch.arange(batch, device="cuda")
    at = lambda c: torch.softmax(s["logits"][:, c].double() / s["temps"].double()[:, None], -1)
    cur = torch.zeros(batch, dtype=torch.int64, device="cuda")
    count = cur + 1
    out_tokens = torch.full((batch, nodes), -1, dtype=torch.int32, device="cuda")
    out_nodes = out_tokens.clone()
    out_nodes[:, 0] = 0
    p = at(0)
    w, total = p, torch.ones(batch, dtype=torch.float64, device="cuda")
    for c in range(1, nodes):  # children come after their parents and in order
        x = s["tokens"][:, c].long()[:, None]
        wx = w.gather(1, x)[:, 0]
        child = (s["parents"][:, c] == cur) & (c < s["n"])
        if s["probs"] is None:
            kept = child & (s["u"][:, c].double() * total < wx)
            rest = w.scatter(1, x, 0.0)
        else:
            q = s["probs"][rows, cur].double()
            kept = child & (s["u"][:, c].double() * q.gather(1, x)[:, 0] * total < wx)
            rest = (w - total[:, None] * q).clamp_min(0.0)
        lost = child & ~kept
        new = at(c)
        p = torch.where(kept[:, None], new, p)
        w = torch.where(kept[:, None], new, torch.where(lost[:, None], rest, w))
        total = torch.where(kept, torch.ones_like(total), torch.where(lost, rest.sum(-1), total))
        cur = torch.where(kept, c, cur)
        out_tokens[rows, count - 1] = torch.where(kept, x[:, 0], -1).to(torch.int32)
        out_nodes[rows, count.clamp_max(nodes - 1)] = torch.where(
            kept, c, out_nodes[rows, count.clamp_max(nodes - 1)].long()).to(torch.int32)
        count = count + kept
    w = torch.where((total > 0)[:, None], w, p)
    last = (w / s["noise"].double().clamp_min(1e-10)).argmax(-1)
    out_tokens[rows, count - 1] = last.to(torch.int32)
    return {"tokens": out_tokens, "nodes": out_nodes, "counts": count.to(torch.int32)}


def _plain_compact(s):
    layers, blocks, block, hkv, _ = s["kc"].shape
    t = s["nodes"].shape[1]
    j = torch.arange(t, device="cuda")
    base = s["ctx"].long()[:, None] - t
    slot = lambda pos: s["bt"].long().gather(1, pos // block) * block + pos % block
    moved = (j[None] < s["counts"][:, None]) & (s["nodes"] != j[None])
    src, dst = slot(base + s["nodes"].long().clamp_min(0))[moved], slot(base + j[None])[moved]
    for cache in (s["kc"], s["vc"]):
        flat = cache.view(layers, blocks * block, hkv, D)
        flat[:, dst] = flat[:, src]
    return {"k_cache": s["kc"], "v_cache": s["vc"]}


def run(s):
    op = s["op"]
    if not own:
        return {"rope": _plain_rope, "tree": _plain_tree, "verify": _plain_verify, "compact": _plain_compact}[op](s)
    import paged_kv_cache_store_gb300 as pa
    if op == "rope":
        if not s["store"]:
            q, k = pa.rope(s["q"], s["k"], s["pos"], s["rope"], s["wq"], s["wk"], EPS)
            return {"q": q, "k": k}
        q = pa.rope_store_kvcache(s["q"], s["k"], s["v"], s["pos"], s["rope"], s["kc"], s["vc"], s["slots"], s["wq"],
                                  s["wk"], EPS)
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    if op == "tree":
        return pa.decode_tree(s["q"], s["kc"], s["vc"], s["bt"], s["ctx"], s["mask"], s["scale"], draft_lens=s["n"],
                              workspace=s["ws"])
    if op == "verify":
        r = pa.verify_drafts(s["logits"], s["tokens"], s["parents"], s["u"], s["noise"], s["temps"],
                             draft_probs=s["probs"], draft_lens=s["n"])
        return {"tokens": r.tokens, "nodes": r.nodes, "counts": r.counts}
    pa.compact_kvcache(s["kc"], s["vc"], s["bt"], s["ctx"], s["nodes"], s["counts"])
    return {"k_cache": s["kc"], "v_cache": s["vc"]}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_heads(x, weight, turn, interleaved):
    """Heads rotated as complex numbers; turn [n, R/2] complex."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.double()
    half = turn.shape[-1]
    if interleaved:
        z = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn[:, None]
        y = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn[:, None]
        y = torch.cat((z.real, z.imag), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        r = case["rotary"]
        f = torch.empty(r // 2, dtype=torch.float64)
        g = 1.0
        for i in range(r // 2):
            wave = case["theta"] ** (2 * i / r)
            if case["scaling"] == "linear":
                wave *= case["factor"]
            elif case["scaling"] == "ntk":
                wave *= (case["factor"] ** (r / (r - 2))) ** (2 * i / r)
            elif case["scaling"] == "yarn":
                g = 1.0 + 0.1 * math.log(case["factor"])
                dim = lambda turns: r * math.log(ORIGINAL / (2 * math.pi * turns)) / math.log(case["theta"]) / 2
                lo, hi = max(0, math.floor(dim(32.0))), min(r - 1, math.ceil(dim(1.0)))
                part = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
                wave = 1.0 / ((1 - part) / wave + part / (wave * case["factor"]))
            f[i] = 1.0 / wave
        turn = torch.polar(torch.full((case["tokens"], r // 2), g, dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * f.cuda())
        q = _exact_heads(s["q"], s["wq"], turn, case["interleaved"])
        k = _exact_heads(s["k"], s["wk"], turn, case["interleaved"])
        if not case["store"]:
            return {"q": q, "k": k}
        kc, vc = s["kc"].double(), s["vc"].double()
        at = torch.nonzero(s["slots"] >= 0)[:, 0]
        slot, block = s["slots"][at].long(), case["block"]
        kc[slot // block, slot % block] = k[at]
        vc[slot // block, slot % block] = s["v"][at].double()
        return {"q": q, "k_cache": kc, "v_cache": vc}
    if op == "tree":
        block, hkv, t = case["block"], case["hkv"], case["drafts"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, (c, n) in enumerate(zip(s["ctx"].tolist(), s["n"].tolist())):
            p = torch.arange(c, device="cuda")
            at, o = s["bt"][b].long()[p // block], p % block
            k, v = (x[at, o].double().transpose(0, 1) for x in (s["kc"], s["vc"]))  # [hkv, c, D]
            hide = torch.zeros((n, c), dtype=torch.bool)
            for i, m in enumerate(s["mask"][b, :n].tolist()):
                hide[i, c - n:] = torch.tensor([not (m >> j) & 1 for j in range(n)])
            hide = hide.cuda()[:, None]
            for h in range(hkv):
                q = s["q"][b, :n, h * (case["hq"] // hkv):(h + 1) * (case["hq"] // hkv)].double()
                x = (q @ k[h].T * s["scale"]).masked_fill(hide, -math.inf)
                out[b, :n, h * (case["hq"] // hkv):(h + 1) * (case["hq"] // hkv)] = torch.softmax(x, -1) @ v[h]
        return out
    if op == "verify":
        batch, nodes = s["tokens"].shape
        tokens = torch.full((batch, nodes), -1, dtype=torch.int32)
        path = torch.full((batch, nodes), -1, dtype=torch.int32)
        counts = torch.zeros(batch, dtype=torch.int32)
        for b in range(batch):
            n, parents, drafted = int(s["n"][b]), s["parents"][b].tolist(), s["tokens"][b].tolist()
            u, kept, v = s["u"][b].tolist(), [0], 0
            while True:
                z = s["logits"][b, v].double() / s["temps"][b].double()
                left = p = torch.exp(z - torch.logsumexp(z, -1))  # a distribution at every step
                following = None
                for c in [c for c in range(1, n) if parents[c] == v]:
                    q = torch.zeros_like(p) if s["probs"] is None else s["probs"][b, v].double()
                    if s["probs"] is None:
                        q[drafted[c]] = 1.0
                    if u[c] * float(q[drafted[c]]) < float(left[drafted[c]]):
                        following = c
                        break
                    rest = torch.relu(left - q) if s["probs"] is not None else left * (1.0 - q)
                    left = rest / rest.sum() if float(rest.sum()) > 0 else torch.zeros_like(rest)
                if following is None:
                    break
                kept.append(following)
                v = following
            left = left if float(left.sum()) > 0 else p
            last = int(torch.argmax(torch.log(left) - torch.log(s["noise"][b].double().clamp_min(1e-10))))
            counts[b] = len(kept)
            path[b, :len(kept)] = torch.tensor(kept)
            tokens[b, :len(kept)] = torch.tensor([drafted[c] for c in kept[1:]] + [last])
        return {"tokens": tokens, "nodes": path, "counts": counts}
    block, t = case["block"], case["nodes"]
    kc, vc = s["kc"].clone(), s["vc"].clone()
    bt = s["bt"].tolist()
    for b, (c, n) in enumerate(zip(s["ctx"].tolist(), s["counts"].tolist())):
        where = [divmod(c - t + i, block) for i in range(t)]
        for j, node in enumerate(s["nodes"][b, :n].tolist()):
            (tb, to), (fb, fo) = where[j], where[node]
            kc[:, bt[b][tb], to], vc[:, bt[b][tb], to] = s["kc"][:, bt[b][fb], fo], s["vc"][:, bt[b][fb], fo]
    return {"k_cache": kc, "v_cache": vc}
