"""What is measured of the long-context operators of the paged KV cache.

Four operators, each in a plain form of elementary torch operations (``own``
false) and through the package's entry points (``own`` true):

* ``shared``   decode attention for sequences that share a prefix by groups;
* ``weights``  decode attention that also accumulates the attention weight
  every cached token received;
* ``evict``    compaction of a cache to a budget by those weights;
* ``rope``     rotary embedding (half or interleaved layout, part of the head,
  scaled frequencies, optional RMSNorm) of new queries and keys, with the K/V
  rows written into their slots.

A case fixes the sizes and, through ``lens_seed``, the lengths; the seed of
``prepare`` fixes the values.
"""
import math

import numpy as np
import torch

own = False

BLOCK, DIM = 16, 128
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
SCALE = 1.0 / math.sqrt(DIM)


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # a few chats under one short system prompt, the 16 / 8-head geometry: latency counts
        dict(name="shared-few", op="shared", dtype="f16", seqs=4, groups=1, hq=16, hkv=8, prefix_lo=1024,
             prefix_hi=1024, suffix_lo=1, suffix_hi=200, lens_seed=1),
        # a batch of questions about one long document, the 32 / 8-head geometry
        dict(name="shared-document", op="shared", dtype="bf16", seqs=32, groups=1, hq=32, hkv=8, prefix_lo=32768,
             prefix_hi=32768, suffix_lo=17, suffix_hi=1000, lens_seed=2),
        # several tenants with prompts of their own, ragged groups, every query tile count from one up
        dict(name="shared-tenants", op="shared", dtype="bf16", seqs=192, groups=3, hq=32, hkv=8, prefix_lo=4096,
             prefix_hi=16384, suffix_lo=1, suffix_hi=700, lens_seed=3),
        # one short sequence whose weights are kept: latency counts
        dict(name="weights-one", op="weights", dtype="f16", seqs=1, hq=16, hkv=8, ctx_lo=777, ctx_hi=777,
             lens_seed=4),
        # an ordinary decode batch
        dict(name="weights-batch", op="weights", dtype="bf16", seqs=32, hq=32, hkv=8, ctx_lo=100, ctx_hi=8192,
             lens_seed=5),
        # few very long contexts, eight query heads to a KV head
        dict(name="weights-long", op="weights", dtype="bf16", seqs=5, hq=32, hkv=4, ctx_lo=40000, ctx_hi=100001,
             lens_seed=6),
        # one short sequence trimmed to half: latency counts
        dict(name="evict-one", op="evict", dtype="f16", seqs=1, hkv=8, ctx_lo=1000, ctx_hi=1000, budget=512,
             recent=64, sinks=4, lens_seed=7),
        # a batch trimmed to a common budget; some sequences are still below it
        dict(name="evict-batch", op="evict", dtype="bf16", seqs=32, hkv=8, ctx_lo=900, ctx_hi=8192, budget=2048,
             recent=256, sinks=4, lens_seed=8),
        # very long contexts, a sharp cut
        dict(name="evict-long", op="evict", dtype="bf16", seqs=4, hkv=8, ctx_lo=60000, ctx_hi=131072, budget=16384,
             recent=1024, sinks=16, lens_seed=9),
        # one decode step at far positions, interleaved layout, three quarters of the head
        dict(name="rope-step", op="rope", dtype="f16", tokens=8, hq=16, hkv=8, rotary=96, layout="interleaved",
             norm=False, scaling="linear", pos_hi=120000, lens_seed=10),
        # one prefill chunk, half layout, scaled by wavelength
        dict(name="rope-chunk", op="rope", dtype="bf16", tokens=512, hq=32, hkv=8, rotary=128, layout="half",
             norm=False, scaling="bands", pos_hi=131072, lens_seed=11),
        # many chunks' tokens at once, with the RMSNorm of queries and keys in front
        dict(name="rope-many", op="rope", dtype="bf16", tokens=16383, hq=32, hkv=8, rotary=128, layout="half",
             norm=True, scaling="yarn", pos_hi=1 << 20, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["shared", "weights", "evict", "rope"])
    case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), lens_seed=rng.randrange(1 << 30))
    if op == "rope":
        hq, hkv = rng.choice([(16, 8), (32, 8), (32, 4), (8, 8), (8, 1)])
        return dict(case, tokens=_log(rng, 1, 16383), hq=hq, hkv=hkv, rotary=rng.choice([128, 128, 96, 64, 32, 2]),
                    layout=rng.choice(["half", "interleaved"]), norm=rng.choice([False, True]),
                    scaling=rng.choice(["none", "linear", "bands", "yarn"]), pos_hi=_log(rng, 16, 1 << 20))
    if op == "shared":
        hq, hkv = rng.choice([(16, 8), (32, 8), (32, 4), (8, 8)])
        seqs, prefix, suffix = _log(rng, 1, 192), _log(rng, 16, 32768) // 16 * 16, _log(rng, 1, 1000)
        while seqs > 1 and seqs * (prefix + suffix) * hkv > 192 * 16000 * 8:
            seqs //= 2
        return dict(case, seqs=seqs, groups=rng.randint(1, min(seqs, 6)), hq=hq, hkv=hkv,
                    prefix_lo=rng.choice([prefix, 16 * (prefix // 64)]), prefix_hi=prefix, suffix_lo=1,
                    suffix_hi=suffix)
    seqs, ctx = _log(rng, 1, 64), _log(rng, 1, 100001)
    while seqs > 1 and seqs * ctx > 300000:
        seqs //= 2
    lo = rng.choice([ctx, max(1, ctx // 20)])
    if op == "weights":
        hq, hkv = rng.choice([(16, 8), (32, 8), (32, 4), (8, 8)])
        return dict(case, seqs=seqs, hq=hq, hkv=hkv, ctx_lo=lo, ctx_hi=ctx)
    budget = min(_log(rng, 1, max(1, ctx)), 16384)
    recent = rng.randint(0, budget // 2)
    return dict(case, seqs=seqs, hkv=rng.choice([8, 8, 4, 1]), ctx_lo=lo, ctx_hi=ctx, budget=budget, recent=recent,
                sinks=rng.randint(0, min(16, budget - recent)))


# ---- lengths (from the case alone) --------------------------------------------

def _groups(case):
    """(group sizes, prefix lengths, context lengths) of a shared case."""
    rng = np.random.default_rng(case["lens_seed"])
    cuts = np.sort(rng.choice(np.arange(1, case["seqs"]), case["groups"] - 1, replace=False)) \
        if case["groups"] > 1 else np.zeros(0, np.int64)
    sizes = np.diff(np.concatenate([[0], cuts, [case["seqs"]]]))
    prefix = rng.integers(case["prefix_lo"] // BLOCK, case["prefix_hi"] // BLOCK + 1, case["groups"]) * BLOCK
    prefix[0] = case["prefix_hi"]
    suffix = rng.integers(case["suffix_lo"], case["suffix_hi"] + 1, case["seqs"])
    return sizes, prefix, np.repeat(prefix, sizes) + suffix


def _lens(case):
    rng = np.random.default_rng(case["lens_seed"])
    lens = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, case["seqs"])
    lens[0] = case["ctx_hi"]
    return lens


def _table(rng, lens, num_blocks, first_block=0):
    """Block table of sequences of the given lengths over a shuffled pool (entries past a length: -1)."""
    pages = -(-lens // BLOCK)
    perm = first_block + rng.permutation(num_blocks - first_block)
    bt = np.full((len(lens), max(1, int(pages.max()))), -1, np.int64)
    at = 0
    for s, n in enumerate(pages):
        bt[s, :n] = perm[at:at + n]
        at += n
    return bt


# ---- inputs --------------------------------------------------------------------

def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _attention_inputs(gen, case, lens, bt, num_blocks, sink_slots):
    """Queries and one layer's pool: unit-normal values, every KV head's queries leaning towards the direction
    of the sequences' first keys, which so take a large part of the weight, as first tokens do."""
    dt, hq, hkv = DTYPES[case["dtype"]], case["hq"], case["hkv"]
    lean = torch.randn((hkv, DIM), generator=gen, device="cuda") * 0.65
    q = torch.randn((len(lens), hkv, hq // hkv, DIM), generator=gen, device="cuda") + lean[:, None]
    k = _randn(gen, (num_blocks, BLOCK, hkv, DIM), dt)
    v = _randn(gen, (num_blocks, BLOCK, hkv, DIM), dt)
    k.view(-1, hkv, DIM)[torch.from_numpy(sink_slots).cuda()] = lean.to(dt)
    return dict(q=q.reshape(len(lens), hq, DIM).to(dt), k=k, v=v,
                bt=torch.from_numpy(bt.astype(np.int32)).cuda(),
                lens=torch.from_numpy(lens.astype(np.int32)).cuda(), max_len=int(lens.max()))


def _frequencies(case):
    """Inverse frequencies (radians per position, float64) and attention factor of a rope case."""
    d, theta, factor, trained = case["rotary"], 1e6, 4.0, 32768.0
    f = theta ** (-np.arange(0, d, 2, dtype=np.float64) / d)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "bands":
        turns = trained * f / (2 * math.pi)
        smooth = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return (1 - smooth) * f / factor + smooth * f, 1.0
    if case["scaling"] == "yarn":
        at = lambda beta: d * math.log(trained / (beta * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), d - 1)
        ramp = np.clip((np.arange(d // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng([seed, case["lens_seed"]])
    op = case["op"]
    state = dict(case=case, op=op)
    if op == "shared":
        sizes, prefix, lens = _groups(case)
        first = np.concatenate([[0], np.cumsum(sizes)])
        head = int((prefix // BLOCK).sum())
        own_pages = -(-lens // BLOCK) - np.repeat(prefix, sizes) // BLOCK
        num_blocks = head + int(own_pages.sum())
        perm = rng.permutation(num_blocks)
        bt = np.full((len(lens), int((-(-lens // BLOCK)).max())), -1, np.int64)
        at = 0
        for g, n in enumerate(prefix // BLOCK):
            bt[first[g]:first[g + 1], :n] = perm[at:at + n]
            at += n
        for s, n in enumerate(own_pages):
            p = -(-int(lens[s]) // BLOCK)
            bt[s, p - n:p] = perm[at:at + n]
            at += n
        state.update(_attention_inputs(gen, case, lens, bt, num_blocks, bt[first[:-1], 0] * BLOCK))
        state.update(sizes=torch.from_numpy(sizes.astype(np.int32)).cuda(),
                     prefix=torch.from_numpy(prefix.astype(np.int32)).cuda())
    elif op == "weights":
        lens = _lens(case)
        num_blocks = int((-(-lens // BLOCK)).sum())
        bt = _table(rng, lens, num_blocks)
        state.update(_attention_inputs(gen, case, lens, bt, num_blocks, bt[:, 0] * BLOCK))
        shape = (len(lens), case["hkv"], int(lens.max()))
        state.update(weights=torch.rand(shape, generator=gen, device="cuda") ** 4 * 8.0,
                     weights_out=torch.zeros(shape, device="cuda"))
    elif op == "evict":
        lens = _lens(case)
        left = np.minimum(lens, case["budget"])
        used = int((-(-lens // BLOCK)).sum())
        num_blocks = used + int((-(-left // BLOCK)).sum())
        dt, hkv = DTYPES[case["dtype"]], case["hkv"]
        perm = rng.permutation(num_blocks)
        bt, dst = _table(rng, lens, used), _table(rng, left, num_blocks, used)
        place = lambda t: np.where(t < 0, -1, perm[t]).astype(np.int32)
        # a few heavy tokens, many of no weight at all, and values that repeat
        w = torch.rand((len(lens), hkv, int(lens.max())), generator=gen, device="cuda") ** 6 * 40.0
        w = torch.where(w < 1.0, torch.floor(w * 4.0) / 4.0, w)
        state.update(k=_randn(gen, (num_blocks, BLOCK, hkv, DIM), dt), v=_randn(gen, (num_blocks, BLOCK, hkv, DIM), dt),
                     bt=torch.from_numpy(place(bt)).cuda(), dst=torch.from_numpy(place(dst)).cuda(),
                     lens=torch.from_numpy(lens.astype(np.int32)).cuda(), max_len=int(lens.max()), weights=w,
                     weights_out=torch.zeros((len(lens), hkv, case["budget"]), device="cuda"))
    else:
        dt, hq, hkv, n = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["tokens"]
        num_blocks = -(-n // BLOCK) + 3
        inv, factor = _frequencies(case)
        if n <= 64:  # a decode step: every token at a position of its own
            pos = rng.integers(0, case["pos_hi"], n)
        else:        # chunks of up to 512 consecutive positions
            pos = (rng.integers(0, max(1, case["pos_hi"] - 511), -(-n // 512))[:, None] + np.arange(512)).ravel()[:n]
        state.update(q=_randn(gen, (n, hq, DIM), dt), new_k=_randn(gen, (n, hkv, DIM), dt),
                     new_v=_randn(gen, (n, hkv, DIM), dt), q_out=torch.zeros((n, hq, DIM), device="cuda", dtype=dt),
                     k=_randn(gen, (num_blocks, BLOCK, hkv, DIM), dt), v=_randn(gen, (num_blocks, BLOCK, hkv, DIM), dt),
                     pos=torch.from_numpy(pos.astype(np.int32)).cuda(),
                     slots=torch.from_numpy(rng.permutation(num_blocks * BLOCK)[:n].astype(np.int64)).cuda(),
                     inv=torch.from_numpy(inv).cuda(), factor=float(factor),
                     qw=(1.0 + 0.2 * torch.randn(DIM, generator=gen, device="cuda")).to(dt) if case["norm"] else None,
                     kw=(1.0 + 0.2 * torch.randn(DIM, generator=gen, device="cuda")).to(dt) if case["norm"] else None)
    return state


# ---- the plain forms -------------------------------------------------------------

def _probabilities(st):
    """softmax(scale q K^T) [S, Hkv, G, L] in fp32 over each sequence's own keys, and its values [S, Hkv, L, 128]."""
    slots = (st["bt"].long().clamp(min=0)[:, :, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(1)
    slots = slots[:, :st["max_len"]]
    hkv = st["k"].shape[2]
    k = st["k"].flatten(0, 1)[slots].float()
    q = st["q"].float().view(len(slots), hkv, -1, DIM)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * SCALE
    del k
    hidden = torch.arange(slots.shape[1], device="cuda") >= st["lens"][:, None]
    s = s.masked_fill_(hidden[:, None, None], -math.inf)
    s = torch.exp(s - s.amax(-1, keepdim=True))
    v = st["v"].flatten(0, 1)[slots].float().permute(0, 2, 1, 3)
    return s / s.sum(-1, keepdim=True), v


def _plain_shared(st):
    p, v = _probabilities(st)
    return torch.matmul(p, v).reshape(st["q"].shape).to(st["q"].dtype)


def _plain_weights(st):
    p, v = _probabilities(st)
    seen = torch.arange(p.shape[-1], device="cuda") < st["lens"][:, None]
    st["weights_out"].copy_(torch.where(seen[:, None], st["weights"] + p.sum(2), st["weights_out"]))
    return torch.matmul(p, v).reshape(st["q"].shape).to(st["q"].dtype), st["weights_out"]


def _plain_evict(st):
    case, w, hkv = st["case"], st["weights"], st["k"].shape[2]
    budget, recent, sinks = case["budget"], case["recent"], case["sinks"]
    S, L = w.shape[0], w.shape[2]
    j, lens = torch.arange(L, device="cuda"), st["lens"].long()[:, None]
    new = torch.minimum(lens, torch.tensor(budget, device="cuda"))
    sure = (j < sinks) | (j >= lens - recent) | (lens <= budget)
    key = torch.where(sure[:, None], math.inf, w)
    key = torch.where((j < lens)[:, None], key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :, :budget]
    live = torch.arange(order.shape[-1], device="cuda") < new
    order = torch.sort(torch.where(live[:, None], order, L), dim=-1).values
    kept = torch.full((S, hkv, budget), -1, device="cuda", dtype=torch.int32)
    kept[:, :, :order.shape[-1]] = torch.where(live[:, None], order, -1).int()
    at = kept.long().clamp(min=0)
    src = torch.gather(st["bt"].long()[:, None].expand(-1, hkv, -1), 2, at // BLOCK) * BLOCK + at % BLOCK
    to = torch.arange(budget, device="cuda").clamp(max=st["dst"].shape[1] * BLOCK - 1)
    to = (st["dst"].long()[:, to // BLOCK] * BLOCK + to % BLOCK)[:, None].expand(-1, hkv, -1)
    heads = torch.arange(hkv, device="cuda")[:, None].expand(S, -1, budget)
    on = kept >= 0
    st["k"].flatten(0, 1)[to[on], heads[on]] = st["k"].flatten(0, 1)[src[on], heads[on]]
    st["v"].flatten(0, 1)[to[on], heads[on]] = st["v"].flatten(0, 1)[src[on], heads[on]]
    st["weights_out"].copy_(torch.where(on, torch.gather(w, 2, at), 0.0))
    return kept, new[:, 0].int(), st["weights_out"], st["k"], st["v"]


def _plain_rotate(st, x, weight):
    half, d = st["case"]["layout"] == "half", st["case"]["rotary"]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = st["pos"].double()[:, None] * st["inv"]
    cos, sin = ((torch.cos(angle) * st["factor"]).float()[:, None], (torch.sin(angle) * st["factor"]).float()[:, None])
    a, b = (y[..., :d // 2], y[..., d // 2:d]) if half else (y[..., 0:d:2], y[..., 1:d:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([a, b], -1) if half else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, y[..., d:]], -1).to(x.dtype)


def _plain_rope(st):
    st["q_out"].copy_(_plain_rotate(st, st["q"], st["qw"]))
    st["k"].flatten(0, 1)[st["slots"]] = _plain_rotate(st, st["new_k"], st["kw"])
    st["v"].flatten(0, 1)[st["slots"]] = st["new_v"]
    return st["q_out"], st["k"], st["v"]


# ---- one pass -----------------------------------------------------------------------

def run(state):
    st, op = state, state["op"]
    if own:
        import paged_kv_gqa_cache_gb300 as pa
        if op == "shared":
            if "workspace" not in st:  # kept by a serving loop, as its other workspaces
                st["workspace"] = pa.alloc_decode_shared_workspace(st["q"].shape[0], len(st["sizes"]),
                                                                   st["q"].shape[1], st["k"].shape[2])
                st["out"] = torch.empty_like(st["q"])
            return pa.paged_attn_decode_shared(st["q"], st["k"], st["v"], st["bt"], st["lens"], st["sizes"],
                                               st["prefix"], SCALE, out=st["out"], workspace=st["workspace"],
                                               max_context_len=st["max_len"])
        if op == "weights":
            if "workspace" not in st:
                st["workspace"] = pa.alloc_decode_weights_workspace(st["q"].shape[0], st["q"].shape[1],
                                                                    st["k"].shape[2], st["max_len"])
                st["out"] = torch.empty_like(st["q"])
            return pa.paged_attn_decode_weights(st["q"], st["k"], st["v"], st["bt"], st["lens"], SCALE,
                                                st["weights"], st["weights_out"], out=st["out"],
                                                workspace=st["workspace"], max_context_len=st["max_len"])
        if op == "evict":
            c = st["case"]
            kept, new = pa.kv_evict(st["k"], st["v"], st["bt"], st["lens"], st["weights"], c["budget"],
                                    recent=c["recent"], sinks=c["sinks"], dst_block_tables=st["dst"],
                                    weights_out=st["weights_out"], max_context_len=st["max_len"])
            return kept, new, st["weights_out"], st["k"], st["v"]
        pa.rope_kv_write(st["q"], st["new_k"], st["new_v"], st["inv"], st["pos"], st["slots"], st["k"], st["v"],
                         interleaved=st["case"]["layout"] == "interleaved", attention_factor=st["factor"],
                         q_norm_weight=st["qw"], k_norm_weight=st["kw"], eps=1e-6, q_out=st["q_out"])
        return st["q_out"], st["k"], st["v"]
    return {"shared": _plain_shared, "weights": _plain_weights, "evict": _plain_evict, "rope": _plain_rope}[op](st)


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op, hkv = case["op"], case["hkv"]
    row = hkv * DIM * 2
    if op == "rope":
        n, rows = case["tokens"], case["hq"] + 2 * hkv
        return {"bytes": n * (2 * rows * DIM * 2 + 12), "flops": n * (case["hq"] + hkv) * 3 * case["rotary"]}
    if op == "shared":
        _, prefix, lens = _groups(case)
        sizes = _groups(case)[0]
        tokens = int(prefix.sum() + lens.sum() - (prefix * sizes).sum())
        return {"bytes": tokens * 2 * row + 2 * case["seqs"] * case["hq"] * DIM * 2,
                "flops": 4 * DIM * case["hq"] * int(lens.sum())}
    lens = _lens(case)
    tokens = int(lens.sum())
    if op == "weights":
        return {"bytes": tokens * (2 * row + 8 * hkv) + 2 * case["seqs"] * case["hq"] * DIM * 2,
                "flops": 4 * DIM * case["hq"] * tokens}
    left = int(np.minimum(lens, case["budget"]).sum())
    return {"bytes": tokens * 4 * hkv + left * (4 * row + 4 * hkv) + case["seqs"] * hkv * case["budget"] * 4,
            "flops": 0}


# ---- the same from the definition, in 64 bits ----------------------------------------

def _exact_attention(st):
    """(out [S, Hq, 128], weights [S, Hkv, L]) in float64, sequence by sequence."""
    S, hq, _ = st["q"].shape
    hkv = st["k"].shape[2]
    out = torch.zeros((S, hq, DIM), dtype=torch.float64, device="cuda")
    got = torch.zeros((S, hkv, st["max_len"]), dtype=torch.float64, device="cuda")
    for s, n in enumerate(st["lens"].tolist()):
        pages = st["bt"][s, :-(-n // BLOCK)].long()
        k, v = st["k"][pages].flatten(0, 1)[:n].double(), st["v"][pages].flatten(0, 1)[:n].double()
        for h in range(hkv):
            rows = slice(h * hq // hkv, (h + 1) * hq // hkv)
            logits = (st["q"][s, rows].double() @ k[:, h].T) / math.sqrt(DIM)
            p = torch.softmax(logits, -1)
            out[s, rows] = p @ v[:, h]
            got[s, h, :n] = p.sum(0)
    return out, got


def _exact_rotate(st, x, weight):
    case = st["case"]
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.double()
    d = case["rotary"]
    z = y.clone()
    for i in range(d // 2):
        a, b = (i, i + d // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
        angle = (st["pos"].double() * st["inv"][i])[:, None]
        c, s = torch.cos(angle) * st["factor"], torch.sin(angle) * st["factor"]
        z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    return z


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "shared":
        return _exact_attention(st)[0]
    if op == "weights":
        out, got = _exact_attention(st)
        for s, n in enumerate(st["lens"].tolist()):
            got[s, :, :n] += st["weights"][s, :, :n].double()
        return out, got
    if op == "rope":
        k, v = st["k"].double(), st["v"].double()
        k.view(-1, *k.shape[2:])[st["slots"]] = _exact_rotate(st, st["new_k"], st["kw"])
        v.view(-1, *v.shape[2:])[st["slots"]] = st["new_v"].double()
        return _exact_rotate(st, st["q"], st["qw"]), k, v
    w, bt, dst = (st[n].cpu().numpy() for n in ("weights", "bt", "dst"))
    k, v = st["k"].double(), st["v"].double()
    hkv, budget = case["hkv"], case["budget"]
    left = np.zeros(w.shape[:2] + (budget,))
    for s, n in enumerate(st["lens"].tolist()):
        for h in range(hkv):
            at = np.arange(n)
            if n > budget:
                middle = np.arange(case["sinks"], n - case["recent"])
                heavy = middle[np.argsort(-w[s, h, middle], kind="stable")[:budget - case["sinks"] - case["recent"]]]
                at = np.concatenate([np.arange(case["sinks"]), np.sort(heavy), np.arange(n - case["recent"], n)])
            left[s, h, :len(at)] = w[s, h, at]
            to = torch.from_numpy(dst[s, np.arange(len(at)) // BLOCK].astype(np.int64)).cuda()
            src = torch.from_numpy(bt[s, at // BLOCK].astype(np.int64)).cuda()
            slot, row = (torch.from_numpy(np.arange(len(at)) % BLOCK).cuda(), torch.from_numpy(at % BLOCK).cuda())
            k[to, slot, h] = st["k"][src, row, h].double()
            v[to, slot, h] = st["v"][src, row, h].double()
    return None, None, torch.from_numpy(left).cuda(), k, v
