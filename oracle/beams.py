"""Beam search over the 8-bit cache, float64 (test infrastructure only): the next beams, and where their states go.

Restates from the definitions alone:

* candidate (i, v) of an item has key = score_i + ((x_iv - m_i) - log sum_u e^(x_iu - m_i)); the largest keys come first, the
  lowest (i, v) first among equal ones; -infinity is no candidate; a finished beam has the one candidate (i, pad);
* beam j continues parents[j]: a parent's first child keeps its slot, the others take the slots of childless beams, both in
  ascending order, and the parent's n mod P tail rows go there.
"""
from __future__ import annotations

import numpy as np


def select(logits, scores, n_out: int, finished=None, pad: int = 0):
    """logits [beams][vocab], scores [beams] of one item: (keys, tokens, parents) [n_out], -inf and -1 where there are none."""
    K, V = logits.shape
    key = np.full((K, V), -np.inf)
    for i in range(K):
        s, x = float(scores[i]), logits[i].astype(np.float64)
        if np.isnan(s) or s == np.inf or s == -np.inf:
            continue
        if finished is not None and finished[i]:
            key[i, pad] = s
            continue
        if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
            continue
        m = x.max()
        key[i] = s + ((x - m) - np.log(np.exp(x - m).sum()))
    flat = key.reshape(-1)
    # (a larger logit of the same beam has the larger key, also where the difference is lost in the sum's 64 bits)
    order = np.lexsort((np.arange(flat.size), -logits.reshape(-1).astype(np.float64), np.arange(flat.size) // V, -flat))[:n_out]
    order = order[flat[order] > -np.inf]
    out = np.full(n_out, -np.inf), np.full(n_out, -1, np.int32), np.full(n_out, -1, np.int32)
    out[0][:len(order)], out[1][:len(order)], out[2][:len(order)] = flat[order], order % V, order // V
    return out


def places(parents):
    """Per child of one item: (the old beam whose slot it takes, whether its parent's tail rows are copied there)."""
    parents = [int(p) for p in parents]
    spare = [k for k in range(len(parents)) if k not in parents]
    kept, out = set(), []
    for p in parents:
        if p >= 0 and p not in kept:
            kept.add(p)
            out.append((p, False))
        else:
            out.append((spare.pop(0), p >= 0))
    return out


def reorder(parents, table, lens, slots, tail, P: int):
    """One item: new (table, lens, slots); tail [layers][slots][heads][2][P][d] is changed in place."""
    new_table, new_lens, new_slots = np.full_like(table, -1), np.zeros_like(lens), np.zeros_like(slots)
    for j, (p, (k, copy)) in enumerate(zip(parents, places(parents))):
        new_slots[j] = slots[k]
        if p >= 0:
            new_table[j], new_lens[j] = table[p], lens[p]
        if copy:
            r = int(lens[p]) % P
            tail[:, slots[k], :, :, :r] = tail[:, slots[p], :, :, :r]
    return new_table, new_lens, new_slots
