"""Plain 64-bit forms of the operators for long and shared caches, written out from their definitions, for
the parity tests."""
import math

import torch

from plain_ops import paths


def cache_rows(t, block_table, block_size, b, pos):
    """Rows of sequence b at these positions, [len(pos), Hkv, D]."""
    if block_table is None:
        return t[b, pos]
    return t.reshape(-1, *t.shape[2:])[[int(block_table[b, p // block_size]) * block_size + p % block_size for p in pos]]


def listed_attention(q, k_tree, v_tree, cache_k, cache_v, prefix_len, parents, scale, positions, block_table=None,
                     block_size=16):
    """(out, spread) in float64 on the CPU.  positions(b, n, h): the prefix positions (a list, where one
    may occur twice) that node n sees through KV head h.  spread is sum(p |v|), the size that errors of
    the weights are relative to."""
    B, N, Hq, D = q.shape
    Hkv = k_tree.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64)
    spread = torch.zeros_like(out)
    for b in range(B):
        path = paths(parents[b] if isinstance(parents[0], (list, tuple)) else parents)
        kept = {}
        for n in range(N):
            for h in range(Hkv):
                pos = positions(b, n, h)
                key = (h, tuple(pos))
                if key not in kept:
                    kept[key] = (cache_rows(cache_k, block_table, block_size, b, pos)[:, h].double(),
                                 cache_rows(cache_v, block_table, block_size, b, pos)[:, h].double())
                k = torch.cat([kept[key][0], k_tree[b, path[n], h].double()])
                v = torch.cat([kept[key][1], v_tree[b, path[n], h].double()])
                x = q[b, n, h * G:(h + 1) * G].double() @ k.T * scale
                p = torch.softmax(x, -1)
                out[b, n, h * G:(h + 1) * G] = p @ v
                spread[b, n, h * G:(h + 1) * G] = p @ v.abs()
    return out, spread


def page_positions(pages, page_size, length):
    """The positions that a list of pages names."""
    return [p for j in pages if j >= 0 for p in range(j * page_size, min(length, (j + 1) * page_size))]


def page_bounds(bounds, cache_k, prefix_len, start, block_table, page_size):
    out = bounds.clone()
    for b, L in enumerate(prefix_len.tolist()):
        s = max(0, int(start[b])) if start is not None else 0
        for j in range(s // page_size, -(-L // page_size) if s < L else 0):
            rows = cache_rows(cache_k, block_table, page_size, b, list(range(j * page_size, min(L, (j + 1) * page_size))))
            to = out[int(block_table[b, j])] if block_table is not None else out[b, j]
            to[:, 0], to[:, 1] = rows.amin(0), rows.amax(0)
    return out


def page_scores(q, bounds, prefix_len, page_size, block_table=None, per_node=False):
    """(scores, size): size bounds the sum of the products' magnitudes of any of the set's rows."""
    B, N, Hq, D = q.shape
    Hkv = bounds.shape[-3]
    G = Hq // Hkv
    P = block_table.shape[1] if block_table is not None else bounds.shape[1]
    out = torch.full((B, N if per_node else 1, Hkv, P), -math.inf, dtype=torch.float64)
    size = torch.zeros_like(out)
    for b, L in enumerate(prefix_len.tolist()):
        for j in range(-(-L // page_size)):
            x = (bounds[int(block_table[b, j])] if block_table is not None else bounds[b, j]).double()
            for h in range(Hkv):
                rows = q[b, :, h * G:(h + 1) * G].double()
                up = rows.clamp(min=0) * x[h, 1] + rows.clamp(max=0) * x[h, 0]  # [N, G, D]
                s, m = up.sum(-1), up.abs().sum(-1)
                if per_node:
                    out[b, :, h, j], size[b, :, h, j] = s.amax(1), m.amax(1)
                else:
                    out[b, 0, h, j], size[b, 0, h, j] = s.max(), m.max()
    return out, size


def select_pages(scores, prefix_len, page_size, count, first, last):
    out = torch.full((*scores.shape[:-1], count), -1, dtype=torch.int32)
    for b, L in enumerate(prefix_len.tolist()):
        n = -(-L // page_size)
        for s in range(scores.shape[1]):
            for h in range(scores.shape[2]):
                if n <= count:
                    got = list(range(n))
                else:
                    keep = set(range(first)) | set(range(n - last, n))
                    x = scores[b, s, h].tolist()
                    rank = lambda i: (0 if math.isnan(x[i]) else 1, 0 if math.isnan(x[i]) else -x[i], i)  # noqa: E731
                    rest = sorted((i for i in range(n) if i not in keep), key=rank)[:count - len(keep)]
                    got = sorted(keep | set(rest))
                out[b, s, h, :len(got)] = torch.tensor(got, dtype=torch.int32)
    return out
