"""Plain fp64 / integer definitions of the serving operators around the verification calls.

Numpy only, written from the definitions: page planning, the K/V store, differential tree attention
and products with 4-bit weights.  Tests compare the library against these.
"""
from __future__ import annotations

import numpy as np

from . import ENOSPACE

EDEVICE = -4


def page_plan(cu_new, kv_len, page_size, held, ring, ring_state, block_table, n_tokens):
    """Requests in order take pages from the ring's head or give surplus pages to its tail.

    Returns (status, held_out, ring_state_out, slot_cap, slot_map); ring and block_table are
    updated in place.  Valid inputs only."""
    P, cap = int(page_size), len(ring)
    head, tail = (int(x) for x in ring_state)
    free = tail - head
    held_out = np.array(held, dtype=np.int32).copy()
    slots = np.full(n_tokens, -1, dtype=np.int64)
    given, status = [], 0
    asked = 0                               # pages asked for so far, by served requests or not
    for r in range(len(kv_len)):
        new = int(cu_new[r + 1]) - int(cu_new[r])
        need = -(-(int(kv_len[r]) + new) // P)
        grow = max(0, need - int(held[r]))
        asked += grow
        if grow and asked > free:
            status = ENOSPACE
            continue
        given += [int(p) for p in block_table[r, need:int(held[r])]]
        for i in range(int(held[r]), need):
            block_table[r, i] = ring[head % cap]
            head += 1
        held_out[r] = need
        for j in range(new):
            t = int(kv_len[r]) + j
            slots[int(cu_new[r]) + j] = int(block_table[r, t // P]) * P + t % P
    for page in given:
        ring[tail % cap] = page
        tail += 1
    return status, held_out, np.array([head, tail], np.int64), held_out * np.int32(P), slots


def kv_store(slot_map, rows, pool):
    """pool[slot] <- row, in place; slots outside the pool are skipped.  Returns a status."""
    status = 0
    for i, s in enumerate(np.asarray(slot_map)):
        if 0 <= s < len(pool):
            pool[s] = rows[i]
        elif s != -1:
            status = EDEVICE
    return status


def ancestors(parent):
    """[n, n] bool: whether node j is node i or an ancestor of it (local parent array)."""
    n = len(parent)
    sees = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            sees[i, j] = True
            j = int(parent[j])
    return sees


def attention_diff(cu_nodes, parent, cache_rows, q, k_tree, v_tree, k_cache, v_cache, scale, lam,
                   norm_w=None, eps=0.0, out_scale=1.0):
    """Differential attention of every tree node.  cache_rows: per request, the cache rows of its
    positions; tensors fp64 [rows][heads][128].  Keys that a node does not see take no part, not
    even when they hold infinities or NaN.  Returns out [n][hq][128] and lse [n][hq][2]."""
    hq, hkv = q.shape[1], k_tree.shape[1]
    out, lse = np.zeros(q.shape), np.zeros((len(q), hq, 2))
    for r in range(len(cu_nodes) - 1):
        a, b = int(cu_nodes[r]), int(cu_nodes[r + 1])
        sees = ancestors(parent[a:b])
        rows = np.asarray(cache_rows[r], dtype=np.int64)
        for i in range(b - a):
            k = np.concatenate([k_cache[rows], k_tree[a:b][sees[i]]])
            v = np.concatenate([v_cache[rows], v_tree[a:b][sees[i]]])
            for h in range(hq):
                kh, vh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
                maps = []
                for m in range(2):
                    z = scale * (kh[:, 64 * m:64 * m + 64] @ q[a + i, h, 64 * m:64 * m + 64])
                    top = z.max()
                    e = np.exp(z - top)
                    lse[a + i, h, m] = top + np.log(e.sum())
                    maps.append((e / e.sum()) @ vh)
                d = maps[0] - float(lam[h]) * maps[1]
                if norm_w is not None:
                    d = d / np.sqrt((d * d).mean() + eps) * norm_w
                out[a + i, h] = d * out_scale
    return out, lse


def w4_weights(wq, scales, zeros, group):
    """fp64 [N][K] weights (q - z) s: byte k / 2 of a row holds k (low half) and k + 1."""
    wq = np.asarray(wq)
    w = np.empty((wq.shape[0], 2 * wq.shape[1]))
    w[:, 0::2], w[:, 1::2] = wq & 15, wq >> 4
    z = 8.0 if zeros is None else np.repeat(np.asarray(zeros, dtype=np.float64), group, axis=1)
    return (w - z) * np.repeat(np.asarray(scales, dtype=np.float64), group, axis=1)


def w4_linear(x, wq, scales, zeros, group, bias=None):
    """fp64 x W^T + bias."""
    y = np.asarray(x, dtype=np.float64) @ w4_weights(wq, scales, zeros, group).T
    return y if bias is None else y + np.asarray(bias, dtype=np.float64)
