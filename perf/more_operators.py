"""What is measured of the operators for tokens whose positions are not one line.

Three operators, each in a plain form of elementary torch operations (``own``
false) and through the package's entry points (``own`` true):

* ``tree``    attention of drafted tokens that form a tree behind each
  sequence's cached context: a token sees the committed context, its ancestors
  in the tree and itself;
* ``accept``  the longest path of such a tree that the model's own choices
  confirm, and the cache of every layer compacted to it in place;
* ``axes``    rotary embedding of new queries and keys whose positions have
  several axes (time, height, width), with the K/V rows written into their slots.

A case fixes the sizes and, through ``lens_seed``, the lengths and the trees'
shapes; the seed of ``prepare`` fixes the values.
"""
import math

import numpy as np
import torch

own = False

BLOCK, DIM = 16, 128
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
SCALE = 1.0 / math.sqrt(DIM)
VOCAB = 151936


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one chat with a handful of drafted tokens, the 16 / 8-head geometry: latency counts
        dict(name="tree-one", op="tree", dtype="f16", seqs=1, hq=16, hkv=8, ctx_lo=777, ctx_hi=777, n_lo=5, n_hi=5,
             shape="random", lens_seed=1),
        # many sequences with short chains of drafts, as extra prediction heads give them
        dict(name="tree-chains", op="tree", dtype="bf16", seqs=192, hq=16, hkv=8, ctx_lo=1, ctx_hi=2900, n_lo=1,
             n_hi=8, shape="chain", lens_seed=2),
        # an ordinary batch with trees from a draft model, the 32 / 8-head geometry
        dict(name="tree-batch", op="tree", dtype="bf16", seqs=32, hq=32, hkv=8, ctx_lo=100, ctx_hi=8192, n_lo=16,
             n_hi=32, shape="random", lens_seed=3),
        # wide trees over longer contexts: two query tiles to a KV head
        dict(name="tree-wide", op="tree", dtype="f16", seqs=8, hq=32, hkv=8, ctx_lo=8000, ctx_hi=32768, n_lo=60,
             n_hi=64, shape="full", lens_seed=4),
        # few very long contexts, eight query heads to a KV head
        dict(name="tree-long", op="tree", dtype="bf16", seqs=5, hq=32, hkv=4, ctx_lo=40000, ctx_hi=100001, n_lo=9,
             n_hi=13, shape="random", lens_seed=5),
        # one chat's drafts judged, 28 layers compacted: latency counts
        dict(name="accept-one", op="accept", dtype="f16", seqs=1, layers=28, hkv=8, ctx_lo=777, ctx_hi=777, n_lo=5,
             n_hi=5, shape="random", keep=0.8, lens_seed=6),
        # an ordinary batch, 36 layers
        dict(name="accept-batch", op="accept", dtype="bf16", seqs=32, layers=36, hkv=8, ctx_lo=30, ctx_hi=500, n_lo=16,
             n_hi=32, shape="random", keep=0.8, lens_seed=7),
        # a large batch of wide trees whose drafts are nearly always right
        dict(name="accept-many", op="accept", dtype="bf16", seqs=192, layers=36, hkv=8, ctx_lo=1, ctx_hi=60, n_lo=33,
             n_hi=64, shape="full", keep=0.95, lens_seed=8),
        # one decode step at far positions: every axis at the same position, as text tokens have them
        dict(name="axes-step", op="axes", dtype="f16", tokens=8, hq=16, hkv=8, sections="16,24,24", woven=False,
             layout="half", norm=False, kind="text", pos_hi=120000, lens_seed=9),
        # the patches of one image between text
        dict(name="axes-image", op="axes", dtype="bf16", tokens=911, hq=32, hkv=8, sections="16,24,24", woven=False,
             layout="half", norm=False, kind="image", pos_hi=32768, lens_seed=10),
        # a video, axes woven pair by pair, with the RMSNorm of queries and keys in front
        dict(name="axes-video", op="axes", dtype="bf16", tokens=16383, hq=32, hkv=8, sections="24,20,20", woven=True,
             layout="half", norm=True, kind="video", pos_hi=131072, lens_seed=11),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "accept", "axes"])
    case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), lens_seed=rng.randrange(1 << 30))
    if op == "axes":
        hq, hkv = rng.choice([(16, 8), (32, 8), (32, 4), (8, 8), (8, 1)])
        rotary, axes = rng.choice([128, 128, 96, 64]), rng.randint(2, 4)
        cuts = sorted(rng.sample(range(1, rotary // 2), axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [rotary // 2])]
        return dict(case, tokens=_log(rng, 1, 16383), hq=hq, hkv=hkv, sections=",".join(map(str, sections)),
                    woven=rng.choice([False, True]), layout=rng.choice(["half", "half", "interleaved"]),
                    norm=rng.choice([False, True]), kind=rng.choice(["text", "image", "video"]),
                    pos_hi=_log(rng, 16, 131072))
    shape = rng.choice(["chain", "random", "full", "forest"])
    if op == "accept":
        seqs, n = _log(rng, 1, 192), _log(rng, 1, 64)
        return dict(case, seqs=seqs, layers=rng.choice([1, 28, 36]), hkv=rng.choice([8, 8, 4, 1]), ctx_lo=n,
                    ctx_hi=n + _log(rng, 1, 60), n_lo=rng.choice([n, 1]), n_hi=n, shape=shape,
                    keep=rng.choice([0.5, 0.8, 0.95]))
    hq, hkv = rng.choice([(16, 8), (32, 8), (32, 4), (8, 8)])
    seqs, ctx, n = _log(rng, 1, 192), _log(rng, 1, 100001), _log(rng, 1, 64)
    while seqs > 1 and seqs * ctx > 160000:
        seqs //= 2
    return dict(case, seqs=seqs, hq=hq, hkv=hkv, ctx_lo=rng.choice([ctx, max(1, ctx // 20)]), ctx_hi=ctx,
                n_lo=rng.choice([n, 1]), n_hi=n, shape=shape)


# ---- lengths, trees and positions (from the case alone) -------------------------

def _lens(case):
    """(tree lengths, context lengths, each at least the tree) of a case."""
    rng = np.random.default_rng(case["lens_seed"])
    n = rng.integers(case["n_lo"], case["n_hi"] + 1, case["seqs"])
    lens = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, case["seqs"])
    n[0], lens[0] = case["n_hi"], case["ctx_hi"]
    return n, np.maximum(lens, n)


def _trees(case):
    """Every sequence's parents, one after the other (-1: no parent)."""
    rng = np.random.default_rng([case["lens_seed"], 1])
    out = []
    for n in _lens(case)[0]:
        i = np.arange(n)
        if case["shape"] == "chain":
            p = i - 1
        elif case["shape"] == "full":      # four children to a token, level by level
            p = np.where(i > 0, (i - 1) // 4, -1)
        else:                              # a few of the latest tokens get children
            p = np.where(i > 0, np.maximum(i - 1 - rng.integers(0, 6, n), 0), -1)
            if case["shape"] == "forest":  # and some tokens stand alone
                p = np.where(rng.random(n) < 0.1, -1, p)
        out.append(p)
    return np.concatenate(out)


def _depths(parents, n):
    """Depth (a token without parent: 1) of every token of one tree."""
    depth = np.ones(n, np.int64)
    for i in range(n):
        if parents[i] >= 0:
            depth[i] = depth[parents[i]] + 1
    return depth


def _table(rng, lens, num_blocks):
    """Block table of sequences of the given lengths over a shuffled pool (entries past a length: -1)."""
    pages = -(-lens // BLOCK)
    perm = rng.permutation(num_blocks)
    bt = np.full((len(lens), int(pages.max())), -1, np.int64)
    at = 0
    for s, n in enumerate(pages):
        bt[s, :n] = perm[at:at + n]
        at += n
    return bt


def _sections(case):
    return [int(n) for n in case["sections"].split(",")]


def _pair_axes(case):
    """The axis of every rotated pair: section after section, or woven (the axes in turn, each as long as it lasts)."""
    left = _sections(case)
    if not case["woven"]:
        return np.repeat(np.arange(len(left)), left)
    out, a = [], 0
    while sum(left):
        if left[a]:
            out.append(a)
            left[a] -= 1
        a = (a + 1) % len(left)
    return np.array(out)


def _positions(case):
    """int [axes, tokens]: text runs with one position on every axis, grids with one per axis."""
    rng = np.random.default_rng([case["lens_seed"], 2])
    axes, n = len(_sections(case)), case["tokens"]
    if case["kind"] == "text" and n <= 64:  # a decode step: a token of each sequence
        return np.repeat(rng.integers(0, case["pos_hi"], n)[None], axes, 0)
    at, parts, left = int(rng.integers(0, max(1, case["pos_hi"] - n))), [], n
    grid = case["kind"] != "text"
    text = int(rng.integers(0, 64)) if grid else n
    while left > 0:
        m = min(text, left)
        parts.append(np.repeat(at + np.arange(m)[None], axes, 0))
        at, left = at + m, left - m
        if left <= 0 or not grid:
            break
        h, w = int(rng.integers(4, 40)), int(rng.integers(4, 40))
        frames = 1 if case["kind"] == "image" else int(rng.integers(2, 17))
        t, y, x = np.meshgrid(np.arange(frames), np.arange(h), np.arange(w), indexing="ij")
        cells = np.stack([t.ravel(), y.ravel(), x.ravel(), (y + x).ravel()])[-axes if axes == 2 else 0:][:axes]
        parts.append(at + cells[:, :left])
        left -= parts[-1].shape[1]
        at += max(frames, h, w)
        text = int(rng.integers(1, 64))
    return np.concatenate(parts, 1)


# ---- inputs --------------------------------------------------------------------

def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _cuda(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a.astype(dtype))).cuda()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng([seed, case["lens_seed"]])
    op, dt, hkv = case["op"], DTYPES[case["dtype"]], case["hkv"]
    state = dict(case=case, op=op)
    if op == "axes":
        n, hq = case["tokens"], case["hq"]
        num_blocks = -(-n // BLOCK) + 3
        pairs = sum(_sections(case))
        inv = 1e6 ** (-np.arange(pairs, dtype=np.float64) / pairs)
        state.update(q=_randn(gen, (n, hq, DIM), dt), new_k=_randn(gen, (n, hkv, DIM), dt),
                     new_v=_randn(gen, (n, hkv, DIM), dt), q_out=torch.zeros((n, hq, DIM), device="cuda", dtype=dt),
                     k=_randn(gen, (num_blocks, BLOCK, hkv, DIM), dt), v=_randn(gen, (num_blocks, BLOCK, hkv, DIM), dt),
                     pos=_cuda(_positions(case), np.int32), pair=_cuda(_pair_axes(case), np.int64),
                     slots=_cuda(rng.permutation(num_blocks * BLOCK)[:n], np.int64), inv=torch.from_numpy(inv).cuda(),
                     qw=(1.0 + 0.2 * torch.randn(DIM, generator=gen, device="cuda")).to(dt) if case["norm"] else None,
                     kw=(1.0 + 0.2 * torch.randn(DIM, generator=gen, device="cuda")).to(dt) if case["norm"] else None)
        return state
    n, lens = _lens(case)
    parents = _trees(case)
    num_blocks = int((-(-lens // BLOCK)).sum())
    bt = _table(rng, lens, num_blocks)
    state.update(bt=_cuda(bt, np.int32), lens=_cuda(lens, np.int32), n=_cuda(n, np.int32),
                 parents=_cuda(parents, np.int32), max_len=int(lens.max()), max_n=int(n.max()))
    if op == "tree":
        # unit-normal values, every KV head's queries leaning towards the direction of the sequences' first keys,
        # which so take a large part of the weight, as first tokens do
        hq, total = case["hq"], int(n.sum())
        lean = torch.randn((hkv, DIM), generator=gen, device="cuda") * 0.65
        q = torch.randn((total, hkv, hq // hkv, DIM), generator=gen, device="cuda") + lean[:, None]
        k = _randn(gen, (num_blocks, BLOCK, hkv, DIM), dt)
        k.view(-1, hkv, DIM)[torch.from_numpy(bt[:, 0] * BLOCK).cuda()] = lean.to(dt)
        state.update(q=q.reshape(total, hq, DIM).to(dt), k=k, v=_randn(gen, (num_blocks, BLOCK, hkv, DIM), dt))
        return state
    # accept: the drafts of one path from each root on are the model's choices, each with probability `keep`;
    # any other token's are so by chance only
    draft, target = rng.integers(0, VOCAB, len(parents)), rng.integers(0, VOCAB, len(parents))
    first = 0
    for m in n:
        p = parents[first:first + m]
        at = 0
        while True:
            below = np.flatnonzero(p == at)
            if len(below) == 0 or rng.random() > case["keep"]:
                break
            child = int(rng.choice(below))
            target[first + at] = draft[first + child]
            at = child
        first += m
    shape = (case["layers"], num_blocks, BLOCK, hkv, DIM)
    state.update(draft=_cuda(draft, np.int64), target=_cuda(target, np.int64))
    for name in ("k", "v"):  # bits of ordinary values (0.0625 .. 2): moved, never computed with
        state[name] = torch.empty(shape, device="cuda", dtype=dt)
        state[name].view(torch.int16).random_(0x2c00 if dt is torch.float16 else 0x3d80, 0x4000, generator=gen)
    return state


# ---- the plain forms -------------------------------------------------------------

def _padded(st):
    """Per sequence, padded to the longest tree: the tokens' rows in the packed inputs [S, N], which of them are
    tokens, their parents (-1 there and past the tree)."""
    n = st["n"].long()
    i = torch.arange(st["max_n"], device="cuda")
    live = i < n[:, None]
    row = ((torch.cumsum(n, 0) - n)[:, None] + i).clamp(max=len(st["parents"]) - 1)
    return row, live, torch.where(live, st["parents"].long()[row], -1)


def _plain_tree(st):
    row, live, parent = _padded(st)
    S, N = row.shape
    hkv, hq = st["k"].shape[2], st["q"].shape[1]
    i = torch.arange(N, device="cuda")
    up = (parent[:, :, None] == i).float() + (i[:, None] == i).float()  # ancestors: powers of parent-or-self
    for _ in range(max(1, (N - 1).bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    lens, n = st["lens"].long(), st["n"].long()
    j = torch.arange(st["max_len"], device="cuda")
    rel = j - (lens - n)[:, None]                                       # [S, L]: place in the tree
    tree = torch.gather(up, 2, rel.clamp(0, N - 1)[:, None].expand(-1, N, -1)) > 0
    seen = (rel < 0)[:, None] | (tree & (rel < n[:, None])[:, None])    # [S, N, L]
    slots = (st["bt"].long().clamp(min=0)[:, :, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(1)
    slots = slots[:, :st["max_len"]]
    k = st["k"].flatten(0, 1)[slots].float()
    q = st["q"][row].float().view(S, N, hkv, hq // hkv, DIM).permute(0, 2, 3, 1, 4).reshape(S, hkv, -1, DIM)
    s = (torch.matmul(q, k.permute(0, 2, 3, 1)) * SCALE).view(S, hkv, -1, N, st["max_len"])
    del k
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    s = torch.exp(s - s.amax(-1, keepdim=True))
    s = (s / s.sum(-1, keepdim=True)).view(S, hkv, -1, st["max_len"])
    v = torch.where((j < lens[:, None])[:, :, None, None], st["v"].flatten(0, 1)[slots].float(), 0.0)
    o = torch.matmul(s, v.permute(0, 2, 1, 3)).view(S, hkv, -1, N, DIM).permute(0, 3, 1, 2, 4).reshape(S, N, hq, DIM)
    return o[live].to(st["q"].dtype)


def _plain_accept(st):
    row, live, parent = _padded(st)
    N = row.shape[1]
    draft, target = st["draft"][row], st["target"][row]
    up = parent.clamp(min=0)
    good = live & ((parent < 0) | (draft == torch.gather(target, 1, up)))
    depth = live.long()
    hop = torch.where(parent < 0, -1, up)
    for _ in range(max(1, (N - 1).bit_length())):  # pointer doubling: all ancestors good, and how many
        more, to = hop >= 0, hop.clamp(min=0)
        good, depth = good & (torch.gather(good, 1, to) | ~more), depth + torch.gather(depth, 1, to) * more
        hop = torch.where(more, torch.gather(hop, 1, to), -1)
    i = torch.arange(N, device="cuda")
    score = torch.where(good, depth * N + (N - 1 - i), -1)
    best = score.amax(1)
    node = torch.where(best >= 0, N - 1 - best % N, 0)
    num = torch.where(best >= 0, best // N, 0)
    path = torch.full_like(row, -1)
    at = node
    for step in range(N):  # from the node up to its root
        to = (num - 1 - step).clamp(min=0)
        on = num > step
        path[torch.arange(len(path), device="cuda"), to] = torch.where(
            on, at, path[torch.arange(len(path), device="cuda"), to])
        at = torch.where(on, torch.gather(parent, 1, at[:, None])[:, 0].clamp(min=0), at)
    start = st["lens"].long() - st["n"].long()
    place = lambda x: (torch.gather(st["bt"].long(), 1, (x // BLOCK).clamp(max=st["bt"].shape[1] - 1)) * BLOCK
                       + x % BLOCK)
    on = path >= 0
    src, dst = place(start[:, None] + path.clamp(min=0))[on], place(start[:, None] + i)[on]
    for name in ("k", "v"):
        flat = st[name].flatten(1, 2)
        flat[:, dst] = flat[:, src]
    nxt = torch.where(num > 0, torch.gather(target, 1, node[:, None])[:, 0], -1)
    return path.int(), num.int(), nxt, (start + num).int(), st["k"], st["v"]


def _plain_rotate(st, x, weight):
    half, d = st["case"]["layout"] == "half", 2 * len(st["pair"])
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = st["pos"].double()[st["pair"]].T * st["inv"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = (y[..., :d // 2], y[..., d // 2:d]) if half else (y[..., 0:d:2], y[..., 1:d:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([a, b], -1) if half else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, y[..., d:]], -1).to(x.dtype)


def _plain_axes(st):
    st["q_out"].copy_(_plain_rotate(st, st["q"], st["qw"]))
    st["k"].flatten(0, 1)[st["slots"]] = _plain_rotate(st, st["new_k"], st["kw"])
    st["v"].flatten(0, 1)[st["slots"]] = st["new_v"]
    return st["q_out"], st["k"], st["v"]


# ---- one pass -----------------------------------------------------------------------

def run(state):
    st, op = state, state["op"]
    if own:
        import paged_kv_gqa_cache_gb300 as pa
        if op == "tree":
            if "workspace" not in st:  # kept by a serving loop, as its other workspaces
                st["workspace"] = pa.alloc_tree_workspace(st["bt"].shape[0], st["q"].shape[1], st["k"].shape[2])
                st["out"] = torch.empty_like(st["q"])
            return pa.paged_attn_tree(st["q"], st["k"], st["v"], st["bt"], st["lens"], st["n"], st["parents"], SCALE,
                                      out=st["out"], workspace=st["workspace"], max_context_len=st["max_len"])
        if op == "accept":
            if "pools" not in st:  # the layers' descriptors, kept with the cache
                st["pools"] = pa.layer_pools(list(zip(st["k"], st["v"])))
            path, num, nxt, lens = pa.tree_accept(st["draft"], st["target"], st["parents"], st["n"], st["lens"],
                                                  st["pools"], st["bt"], max_tree_len=st["max_n"])
            return path, num, nxt, lens, st["k"], st["v"]
        if "axes" not in st:  # fixed by the model's configuration
            st["axes"] = pa.rope_axes(_sections(st["case"]), woven=st["case"]["woven"])
        pa.rope_kv_write_axes(st["q"], st["new_k"], st["new_v"], st["inv"], st["pos"], st["axes"], st["slots"],
                              st["k"], st["v"], interleaved=st["case"]["layout"] == "interleaved",
                              q_norm_weight=st["qw"], k_norm_weight=st["kw"], eps=1e-6, q_out=st["q_out"])
        return st["q_out"], st["k"], st["v"]
    return {"tree": _plain_tree, "accept": _plain_accept, "axes": _plain_axes}[op](st)


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op, hkv = case["op"], case["hkv"]
    row = hkv * DIM * 2
    if op == "axes":
        n, rows = case["tokens"], case["hq"] + 2 * hkv
        return {"bytes": n * (2 * rows * DIM * 2 + 8 + 4 * len(_sections(case))),
                "flops": n * (case["hq"] + hkv) * 6 * sum(_sections(case))}
    n, lens = _lens(case)
    total = int(n.sum())
    trees = np.split(_trees(case), np.cumsum(n)[:-1])
    if op == "tree":
        keys = sum(int((L - m) * m + _depths(p, m).sum()) for p, m, L in zip(trees, n, lens))
        return {"bytes": int(lens.sum()) * 2 * row + total * (2 * case["hq"] * DIM * 2 + 4),
                "flops": 4 * DIM * case["hq"] * keys}
    # which tokens move is the values' doing: a path of the expected length, all of it but the root moved
    moved = sum(sum(case["keep"] ** d for d in range(1, int(_depths(p, m).max()))) for p, m in zip(trees, n))
    return {"bytes": total * 20 + int(moved * case["layers"] * 4 * row), "flops": 0}


# ---- the same from the definition, in 64 bits ----------------------------------------

def _exact_tree(st):
    hq, hkv = st["q"].shape[1], st["k"].shape[2]
    out, first = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"), 0
    for s, (L, n) in enumerate(zip(st["lens"].tolist(), st["n"].tolist())):
        parents = st["parents"][first:first + n].tolist()
        hidden = np.ones((n, L), bool)
        hidden[:, :L - n] = False
        for i in range(n):
            a = i
            while a >= 0:
                hidden[i, L - n + a] = False
                a = parents[a]
        hidden = torch.from_numpy(hidden).cuda()
        pages = st["bt"][s, :-(-L // BLOCK)].long()
        k, v = st["k"][pages].flatten(0, 1)[:L], st["v"][pages].flatten(0, 1)[:L]
        for g in range(hq):
            h = g * hkv // hq
            logits = (st["q"][first:first + n, g].double() @ k[:, h].double().T) / math.sqrt(DIM)
            out[first:first + n, g] = torch.softmax(logits.masked_fill(hidden, -math.inf), -1) @ v[:, h].double()
        first += n
    return out


def _exact_rotate(st, x, weight):
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.double()
    z, d = y.clone(), 2 * len(st["pair"])
    for i, axis in enumerate(st["pair"].tolist()):
        a, b = (i, i + d // 2) if st["case"]["layout"] == "half" else (2 * i, 2 * i + 1)
        angle = (st["pos"][axis].double() * st["inv"][i])[:, None]
        c, s = torch.cos(angle), torch.sin(angle)
        z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    return z


def exact(case, seed):
    if case["op"] == "accept":
        return None  # whole numbers and moved bits: nothing is computed
    st = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(st)
    k, v = st["k"].double(), st["v"].double()
    k.view(-1, *k.shape[2:])[st["slots"]] = _exact_rotate(st, st["new_k"], st["kw"])
    v.view(-1, *v.shape[2:])[st["slots"]] = st["new_v"].double()
    return _exact_rotate(st, st["q"], st["qw"]), k, v
