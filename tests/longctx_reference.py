"""Plain 64-bit forms of the long-context operators (numpy, loops over
sequences and heads), for the tests: written from the operators' definitions,
sharing nothing with the library's kernels."""
import numpy as np
import torch

BLOCK, DIM = 16, 128
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
# a rounding to the type is off by at most half a step, relative to the value ...
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
# ... or, below the type's normal range, by half of its smallest value
HALF_TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def rotate(x, positions, inv_freq, factor, interleaved, weight=None, eps=0.0):
    """(rotated rows, per-element sum of the magnitudes that entered it) of x [T, H, 128] in float64."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    out, mag = y.copy(), np.abs(y)
    d = 2 * len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + d // 2)
        angle = positions.astype(np.float64) * f
        c, s = (np.cos(angle) * factor)[:, None], (np.sin(angle) * factor)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        mag[..., a] = mag[..., b] = (np.abs(y[..., a]) + np.abs(y[..., b])) * abs(factor)
    return out, mag


def evict_keep(w, n, budget, recent, sinks):
    """Indices that stay of n tokens with weights w (float64 or float32), ascending."""
    if n <= budget:
        return np.arange(n)
    middle = np.arange(sinks, n - recent)
    rank = np.where(np.isnan(w[middle]), -np.inf, w[middle].astype(np.float64))
    # a NaN lies below every number, -inf among them; lexsort: last key first
    order = np.lexsort((middle, -rank, np.isnan(w[middle])))
    heavy = np.sort(middle[order[:budget - sinks - recent]])
    return np.concatenate([np.arange(sinks), heavy, np.arange(n - recent, n)]).astype(np.int64)


def gather(cache, table_row, n, head):
    """Rows 0 .. n - 1 of one KV head of a pool [blocks, 16, Hkv, 128] through a block-table row."""
    pos = np.arange(n)
    return cache[table_row[pos // BLOCK], pos % BLOCK, head]


def attention(q, k_cache, v_cache, tables, lens, scale):
    """(out [S, Hq, 128], weight per KV head and token [S, Hkv, max], sum of |p v| [S, Hq, 128]) in float64."""
    S, hq, _ = q.shape
    hkv = k_cache.shape[2]
    G = hq // hkv
    out, mag = np.zeros((S, hq, DIM)), np.zeros((S, hq, DIM))
    w = np.zeros((S, hkv, max(int(lens.max()), 1)))
    for s in range(S):
        n = int(lens[s])
        for h in range(hkv):
            k, v = gather(k_cache, tables[s], n, h), gather(v_cache, tables[s], n, h)
            for g in range(G):
                x = scale * (k @ q[s, h * G + g])
                p = np.exp(x - x.max())
                p /= p.sum()
                out[s, h * G + g] = p @ v
                mag[s, h * G + g] = p @ np.abs(v)
                w[s, h, :n] += p
    return out, w, mag


def place(rng, lens, extra=2, first=0):
    """A shuffled block table (int32, -1 past a length) of the given lengths and the pool's block count."""
    pages = [-(-int(n) // BLOCK) for n in lens]
    total = first + sum(pages) + extra
    perm = first + rng.permutation(total - first)
    bt = np.full((len(lens), max(max(pages), 1)), -1, np.int32)
    at = 0
    for s, n in enumerate(pages):
        bt[s, :n] = perm[at:at + n]
        at += n
    return bt, total


def random_pool(gen, blocks, hkv, dtype, device="cuda"):
    return torch.randn((blocks, BLOCK, hkv, DIM), generator=gen, device=device).to(TORCH[dtype])


def bits(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy().copy()


def attention_torch(q, k_cache, v_cache, tables, lens, scale):
    """(out, sum of |p v|, largest scale * sum |q_i k_i|) of the same in float64 on the tensors' own device."""
    S, hq, _ = q.shape
    hkv = k_cache.shape[2]
    G = hq // hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mag, worst = torch.zeros_like(out), 0.0
    for s in range(S):
        n = int(lens[s])
        rows = torch.as_tensor(tables[s][:-(-n // BLOCK)], device=q.device).long()
        k = k_cache[rows].flatten(0, 1)[:n].double().transpose(0, 1)  # [Hkv, n, 128]
        v = v_cache[rows].flatten(0, 1)[:n].double().transpose(0, 1)
        x = q[s].double().view(hkv, G, DIM)
        p = torch.softmax(scale * torch.matmul(x, k.transpose(1, 2)), -1)
        out[s] = torch.matmul(p, v).view(hq, DIM)
        mag[s] = torch.matmul(p, v.abs()).view(hq, DIM)
        worst = max(worst, float(scale * torch.matmul(x.abs(), k.abs().transpose(1, 2)).max()))
    return out, mag, worst
