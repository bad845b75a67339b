"""CPU oracle of the attention over key spans, in fp64 over the dequantised paged caches.

TEST INFRASTRUCTURE ONLY.  Query row r of a sequence of L tokens, at position pos, sees the keys
max(0, key_begin[r]) <= j < min(L, key_end[r]) (defaults 0 and pos + 1), with logits
s_j = scale q . k_j, then softcap tanh(s_j / softcap), then s_j - slope |pos - j|; rows that see no key are zero.
``decode(rows)`` gives the vectors [N, d] (fp64) that cached rows [N, row bytes] stand for.
"""
from __future__ import annotations

import numpy as np


def attention(query, cache, block_tables, seq_lens, query_start_loc, scale, decode, key_begin=None, key_end=None, softcap=0.0,
              alibi_slopes=None):
    """(out [Nq, Hq, d], size [Nq, Hq]): the outputs, NaN in rows of no sequence, and sum_j w_j |v_j|_2 of each row, what
    errors of the weights are relative to."""
    q = query.detach().cpu().double().numpy() if hasattr(query, "detach") else np.asarray(query, np.float64)
    nq, hq, d = q.shape
    H, num_blocks = cache.shape[3], cache.shape[0]
    G = hq // H
    out, size = np.full((nq, hq, d), np.nan), np.zeros((nq, hq))
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        q0, q1 = int(query_start_loc[b]), int(query_start_loc[b + 1])
        out[q0:q1] = 0.0
        if L == 0 or q1 == q0:
            continue
        j = np.arange(L)
        blk = np.asarray(block_tables[b])[j // 16]
        there = (blk >= 0) & (blk < num_blocks)
        rows = cache[np.where(there, blk, 0), :, j % 16]          # [L, 2, H, bytes]
        pos = L - (q1 - q0) + np.arange(q1 - q0)
        lo = np.maximum(0, np.asarray(key_begin)[q0:q1]) if key_begin is not None else np.zeros_like(pos)
        hi = np.minimum(L, np.asarray(key_end)[q0:q1] if key_end is not None else pos + 1)
        seen = there & (j >= lo[:, None]) & (j < hi[:, None])     # [queries, L]
        some = seen.any(axis=1)
        for h in range(H):
            k, v = (decode(np.ascontiguousarray(rows[:, i, h])) for i in (0, 1))
            for g in range(h * G, (h + 1) * G):
                s = scale * (q[q0:q1, g] @ k.T)
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                if alibi_slopes is not None:
                    s = s - float(alibi_slopes[g]) * np.abs(pos[:, None] - j)
                s = np.where(seen, s, -np.inf)
                w = np.exp(s - np.where(some, s.max(axis=1), 0.0)[:, None])
                w = w / np.where(some, w.sum(axis=1), 1.0)[:, None]
                out[q0:q1, g] = w @ np.where(seen.any(axis=0)[:, None], v, 0.0)
                size[q0:q1, g] = w @ np.linalg.norm(v, axis=1)
    return out, size
