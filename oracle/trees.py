"""Whole prompts and trees of drafted tokens (test infrastructure).

* ``attention_prompt`` -- causal scaled dot-product attention of packed sequences;
* ``tree_path`` -- the nodes from a tree's root to a node;
* ``attention_tree`` -- attention of a tree's nodes over a shared prefix, the sequence's
  committed entries and the nodes' ancestors;
* ``accept_tree`` -- the walk to the lowest-numbered child that holds the sampled token.

A tree is a list of parents: -1 for node 0, the root, and for unused rows.
Everything is evaluated in fp64; arrays are in plain layouts.
"""

from __future__ import annotations

import math

import numpy as np


def _attend(q, k, v):
    """(sum_t w_t v_t, sum_t w_t |v_t|) of queries q [..., D] over k, v [T][D]."""
    s = q @ k.T / math.sqrt(q.shape[-1])
    w = np.exp(s - s.max(axis=-1, keepdims=True))
    w /= w.sum(axis=-1, keepdims=True)
    return w @ v, w @ np.abs(v)


def attention_prompt(q, k, v, starts):
    """q [rows][n_kv][group][D]; k, v [rows][n_kv][D]; sequence s is rows starts[s] ..
    starts[s+1]-1.  (out, spread) of q's shape, zeros outside the sequences."""
    q = np.asarray(q, np.float64)
    out, spread = np.zeros_like(q), np.zeros_like(q)
    for a, b in zip(starts[:-1], starts[1:]):
        for r in range(a, b):
            for j in range(q.shape[1]):
                out[r, j], spread[r, j] = _attend(q[r, j], k[a:r + 1, j], v[a:r + 1, j])
    return out, spread


def tree_path(parents, i):
    """Nodes from the root to node i, both included; [] where row i is unused."""
    if i > 0 and parents[i] < 0:
        return []
    path = [i]
    while path[0] > 0:
        path.insert(0, parents[path[0]])
    return path


def attention_tree(q, shared_k, shared_v, own_k, own_v, pos, parents):
    """q [B][n][n_kv][group][D]; shared_k, shared_v [n_kv][P][D]; own_k, own_v
    [B][n_kv][L][D], node i's entry at pos[b] + i; pos [B] (negative: idle); parents
    [B][n].  (out, spread) of q's shape, zeros for idle sequences and unused rows."""
    q = np.asarray(q, np.float64)
    out, spread = np.zeros_like(q), np.zeros_like(q)
    for b in range(q.shape[0]):
        for i in range(q.shape[1]):
            path = tree_path(parents[b], i)
            if pos[b] < 0 or not path:
                continue
            at = list(range(pos[b])) + [pos[b] + a for a in path]
            for j in range(q.shape[2]):
                k = np.concatenate([shared_k[j], own_k[b, j, at]])
                v = np.concatenate([shared_v[j], own_v[b, j, at]])
                out[b, i, j], spread[b, i, j] = _attend(q[b, i, j], k, v)
    return out, spread


def accept_tree(parents, tokens, sampled):
    """(accepted, bonus, path, committed) of one tree: tokens[i] the draft at node i,
    sampled[i] what decoding samples after it."""
    path = [0]
    while True:
        fits = [c for c in range(1, len(parents)) if parents[c] == path[-1] and tokens[c] == sampled[path[-1]]]
        if not fits:
            break
        path.append(fits[0])
    return len(path) - 1, sampled[path[-1]], path, [sampled[i] for i in path]
