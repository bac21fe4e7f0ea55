"""Plain 64-bit forms of the operators on trees of drafted tokens, for the tests:
written from the operators' definitions, sharing nothing with the library's kernels."""
import numpy as np
import torch

from longctx_reference import BLOCK, DIM, place, random_pool, TORCH

SHAPES = ("chain", "star", "full", "random", "forest", "roots")


def make_tree(shape, n, rng):
    """Parents (int32 [n], -1: none) of a tree of n tokens."""
    i = np.arange(n)
    if shape == "chain":
        p = i - 1
    elif shape == "star":      # all under the first
        p = np.where(i > 0, 0, -1)
    elif shape == "full":
        p = np.where(i > 0, (i - 1) // 3, -1)
    elif shape == "roots":     # nobody has a parent
        p = np.full(n, -1)
    else:
        p = np.array([-1] + [int(rng.integers(0, k)) for k in range(1, n)])[:n]
        if shape == "forest":
            p = np.where(rng.random(n) < 0.3, -1, p)
    return p.astype(np.int32)


def ancestors(parents):
    """Truth matrix [n, n]: row i has i and all above it."""
    n = len(parents)
    out = np.zeros((n, n), bool)
    for i in range(n):
        a = i
        while a >= 0:
            out[i, a] = True
            a = int(parents[a])
    return out


def make_case(trees, ctx, hq, hkv, dtype, seed, peak=1.0, width=0, device="cuda"):
    """Sequences with these trees (a list of parents) and whole lengths; every slot without a token holds NaN."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=device).manual_seed(seed)
    lens = np.asarray(ctx, np.int64)
    n = np.array([len(t) for t in trees])
    assert (lens >= n).all()
    bt, nb = place(rng, np.maximum(lens, 1), extra=3)
    if width > bt.shape[1]:
        bt = np.concatenate([bt, np.full((len(bt), width - bt.shape[1]), -1, np.int32)], 1)
    kc, vc = random_pool(g, nb, hkv, dtype, device), random_pool(g, nb, hkv, dtype, device)
    live = torch.zeros((nb, BLOCK), dtype=torch.bool)
    for s, L in enumerate(lens):
        pos = np.arange(L)
        live[bt[s, pos // BLOCK], pos % BLOCK] = True
    kc[~live.to(device)] = float("nan")
    vc[~live.to(device)] = float("nan")
    total = int(n.sum())
    q = (torch.randn((total, hq, DIM), generator=g, device=device) * peak).to(TORCH[dtype])
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device=device)
    return dict(q=q, kc=kc, vc=vc, bt=i32(bt), lens=i32(lens), n=i32(n), trees=trees, dtype=dtype, bt_h=bt, lens_h=lens,
                parents=i32(np.concatenate(trees) if total else np.zeros(0)))


def attention(c, scale, skip=()):
    """(out, sum of |p v|, largest scale sum |q_i k_i|) of every row in float64 (rows of `skip`ped sequences: NaN)."""
    q, hq, hkv = c["q"], c["q"].shape[1], c["kc"].shape[2]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    mag, worst, row = torch.zeros_like(out), 0.0, 0
    for s, t in enumerate(c["trees"]):
        n, L = len(t), int(c["lens_h"][s])
        if n and s not in skip:
            pages = torch.as_tensor(c["bt_h"][s][:-(-L // BLOCK)], device=q.device).long()
            k = c["kc"][pages].flatten(0, 1)[:L].double().transpose(0, 1)  # [Hkv, L, 128]
            v = c["vc"][pages].flatten(0, 1)[:L].double().transpose(0, 1)
            seen = torch.ones((n, L), dtype=torch.bool, device=q.device)
            seen[:, L - n:] = torch.as_tensor(ancestors(t), device=q.device)
            x = q[row:row + n].double().view(n, hkv, hq // hkv, DIM).permute(1, 2, 0, 3)  # [Hkv, G, n, 128]
            z = (scale * torch.matmul(x, k[:, None].transpose(2, 3))).masked_fill(~seen, -float("inf"))
            p = torch.softmax(z, -1)
            # a value that a row does not see plays no part, whatever it is
            bad = ~torch.isfinite(v)
            sight = torch.matmul((seen[None, None] * 1.0).expand(hkv, hq // hkv, n, L), (bad * 1.0)[:, None])
            v = torch.where(bad, 0.0, v)
            back = lambda y: y.permute(2, 0, 1, 3).reshape(n, hq, DIM)
            out[row:row + n] = back(torch.where(sight.amax(-1, keepdim=True) > 0, float("nan"),
                                                torch.matmul(p, v[:, None])))
            mag[row:row + n] = back(torch.matmul(p, v[:, None].abs()))
            worst = max(worst, float((scale * torch.matmul(x.abs(), k[:, None].abs().transpose(2, 3))).nan_to_num().max()))
        row += n
    return out, mag, worst


def accept(parents, draft, target):
    """(path, next token) of one tree, from the definition."""
    best, depth_of = None, 0
    ok = []
    for i, p in enumerate(parents):
        p = int(p)
        ok.append(p < 0 or (ok[p] and draft[i] == target[p]))
        if ok[i]:
            path, a = [], i
            while a >= 0:
                path.append(a)
                a = int(parents[a])
            if len(path) > depth_of:
                best, depth_of = path[::-1], len(path)
    return (best, int(target[best[-1]])) if best else ([], -1)


def move(pool, table, start, path):
    """The pool (a numpy array [blocks, 16, ...]) with the path's rows moved, through a copy of the sources."""
    slot = lambda p: (table[p // BLOCK], p % BLOCK)
    rows = [pool[slot(start + a)].copy() for a in path]
    for i, r in enumerate(rows):
        pool[slot(start + i)] = r
