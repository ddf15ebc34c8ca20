"""Plain 64-bit forms of the operators around the KV cache, written out from their definitions
(loops over sequences and nodes, numpy), for the parity tests."""
import math

import numpy as np
import torch


def paths(parent):
    """Each node's root path, root first; a node's depth is its path's length - 1."""
    out = []
    for n, p in enumerate(parent):
        out.append([n] if p < 0 else out[p] + [n])
    return out


def window_attention(q, k_tree, v_tree, cache_k, cache_v, prefix_len, parents, scale, window, sinks=0,
                     block_table=None, block_size=16):
    """(out, spread) in float64, CPU tensors.  parents: one parent list, or one per sequence.
    spread is sum(p |v|), the size that errors of the weights are relative to."""
    B, N, Hq, D = q.shape
    Hkv = k_tree.shape[2]
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64)
    spread = torch.zeros_like(out)
    for b in range(B):
        par = parents[b] if isinstance(parents[0], (list, tuple)) else parents
        L = int(prefix_len[b])
        path = paths(par)
        P = [L + len(x) - 1 for x in path]
        keep = [p for p in range(L) if p < sinks or min(P) - p < window]
        see = torch.zeros(N, len(keep) + N, dtype=torch.bool)
        for n in range(N):
            see[n, :len(keep)] = torch.tensor([P[n] - p < window or p < sinks for p in keep], dtype=torch.bool)
            for d, j in enumerate(path[n]):
                see[n, len(keep) + j] = P[n] - (L + d) < window or L + d < sinks
        if block_table is None:
            kp, vp = cache_k[b, keep], cache_v[b, keep]
        else:
            rows = [int(block_table[b, p // block_size]) * block_size + p % block_size for p in keep]
            kp = cache_k.reshape(-1, Hkv, D)[rows]
            vp = cache_v.reshape(-1, Hkv, D)[rows]
        k = torch.cat([kp, k_tree[b]]).double().permute(1, 2, 0)  # [Hkv, D, keys]
        v = torch.cat([vp, v_tree[b]]).double().permute(1, 0, 2)  # [Hkv, keys, D]
        x = q[b].double().view(N, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        s = (x @ k * scale).view(Hkv, N, Hq // Hkv, -1).masked_fill(~see[None, :, None, :], -math.inf)
        p = torch.softmax(s, -1).view(Hkv, -1, s.shape[-1])
        for to, y in ((out, p @ v), (spread, p @ v.abs())):
            to[b] = y.view(Hkv, N, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(N, Hq, D)
    return out, spread


def attention_bound(out, spread, dtype, D, score_size, keys):
    """How far an fp32-accumulating kernel's result may be from `out`, element by element.
    score_size bounds scale * sum |q_i k_i|.
      scores: D products and sums in fp32, each off by 2^-24 of at most score_size, move every
              weight by a relative 2 (D + 2) 2^-24 score_size (its own score and the others' in
              the denominator); the exponential and the scaling add 2^-21
      sums:   `keys` fp32 additions each in numerator and denominator: 2 keys 2^-24
      bf16:   the weights are rounded for the second product, 2^-8 each, and so is the result
    Weights' errors count relative to spread = sum(p |v|), the result's rounding to itself."""
    rel = 2 * (D + 2) * 2.0 ** -24 * score_size + 2.0 ** -21 + 2 * keys * 2.0 ** -24
    if dtype == torch.bfloat16:
        return (2.0 ** -8 * 1.01 + rel) * spread + 2.0 ** -8 * (out.abs() + (2.0 ** -8 * 1.01 + rel) * spread)
    return rel * spread + 2.0 ** -24 * out.abs()


def qk_norm_rope(qkv, Hq, Hkv, q_weight, k_weight, inv_freq, positions, eps, interleaved):
    """(q, k, v) [T, H, D] float64 and the pair sizes |a| + |b| that errors are relative to."""
    D = q_weight.numel()
    half = inv_freq.numel()
    x = qkv.double().reshape(-1, Hq + 2 * Hkv, D)
    y = x.clone()
    size = x.abs().clone()
    w = torch.cat([q_weight.double().expand(Hq, D), k_weight.double().expand(Hkv, D)])
    y[:, :Hq + Hkv] = x[:, :Hq + Hkv] / torch.sqrt((x[:, :Hq + Hkv] ** 2).mean(-1, keepdim=True) + eps) * w
    z = y.clone()
    for t, pos in enumerate(positions.reshape(-1).tolist()):
        for i in range(half):
            c, s = math.cos(pos * float(inv_freq[i])), math.sin(pos * float(inv_freq[i]))
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            a, b = y[t, :Hq + Hkv, ia], y[t, :Hq + Hkv, ib]
            z[t, :Hq + Hkv, ia], z[t, :Hq + Hkv, ib] = a * c - b * s, a * s + b * c
            size[t, :Hq + Hkv, ia] = size[t, :Hq + Hkv, ib] = a.abs() + b.abs()
    size[:, :Hq + Hkv, 2 * half:] = y[:, :Hq + Hkv, 2 * half:].abs()
    return (z[:, :Hq], z[:, Hq:Hq + Hkv], z[:, Hq + Hkv:]), (size[:, :Hq], size[:, Hq:Hq + Hkv])


def rope_bound(out, size, dtype, D):
    """fp32 between load and store: the mean of D squares (D roundings, halved by the root), the
    root and its product, the weight, sine and cosine and the two products and their sum: (D/2 +
    16) 2^-24 of |a| + |b|; then one rounding to bf16, 2^-8 of the result."""
    rel = (D / 2 + 16) * 2.0 ** -24
    last = 2.0 ** -8 * (out.abs() + rel * size) if dtype == torch.bfloat16 else 0.0
    return rel * size + last


def block_tables(length, new_tokens, block_table, free_blocks, head, block_size, num_slots):
    """numpy int arrays in, dict of them out (block_table a copy)."""
    table = block_table.copy()
    slots, positions, start = [], [], [0]
    for b in range(len(length)):
        held = -(-int(length[b]) // block_size)
        total = -(-(int(length[b]) + int(new_tokens[b])) // block_size)
        for j in range(held, total):
            table[b, j] = free_blocks[head]
            head += 1
        for p in range(int(length[b]), int(length[b]) + int(new_tokens[b])):
            slots.append(int(table[b, p // block_size]) * block_size + p % block_size)
            positions.append(p)
        start.append(len(slots))
    pad = [-1] * (num_slots - len(slots))
    return dict(block_table=table, token_start=np.array(start), slots=np.array(slots + pad),
                positions=np.array(positions + pad), free_head=np.array([head]))
