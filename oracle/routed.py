"""CPU reference of the routed operators: rows of one batch that go to different weights.

NumPy, fp64. A slot ``i = t * topk + j`` is choice ``j`` of token ``t``; an id outside ``[0, groups)`` is
no group. Rows are sorted by group, slots ascending within one, the slots of no group last.
"""
from __future__ import annotations

import numpy as np

from .glu import silu, swiglu_split


def route_ref(ids: np.ndarray, groups: int):
    """``(offsets[groups + 1], order[S], slot[tokens, topk])`` by one loop over the slots."""
    flat = np.asarray(ids).reshape(-1)
    bins = [[] for _ in range(groups + 1)]
    for i, e in enumerate(flat.tolist()):
        bins[e if 0 <= e < groups else groups].append(i)
    offsets = np.cumsum([0] + [len(b) for b in bins[:groups]]).astype(np.int32)
    order = np.array([i for b in bins for i in b], dtype=np.int32)
    slot = np.full(flat.size, -1, dtype=np.int32)
    n = int(offsets[-1])
    slot[order[:n]] = np.arange(n, dtype=np.int32)
    return offsets, order, slot.reshape(np.asarray(ids).shape)


def dispatch_ref(x, offsets, order, topk):
    n = int(offsets[-1])
    xs = np.zeros((len(order), x.shape[1]), dtype=x.dtype)
    xs[:n] = x[order[:n] // topk]
    return xs


def combine_ref(ys, slot, weights):
    """``y[t] = sum_j weights[t, j] ys[slot[t, j]]``; a slot of no group adds nothing."""
    y = np.zeros((slot.shape[0], ys.shape[1]))
    for t in range(slot.shape[0]):
        for j in range(slot.shape[1]):
            if slot[t, j] >= 0:
                y[t] += float(weights[t, j]) * np.asarray(ys[slot[t, j]], dtype=np.float64)
    return y


def combine_backward_ref(dy, ys, slot, weights):
    dys = np.zeros(ys.shape)
    dw = np.zeros(slot.shape)
    for t in range(slot.shape[0]):
        for j in range(slot.shape[1]):
            if slot[t, j] >= 0:
                d = np.asarray(dy[t], dtype=np.float64)
                dys[slot[t, j]] = float(weights[t, j]) * d
                dw[t, j] = d @ np.asarray(ys[slot[t, j]], dtype=np.float64)
    return dys, dw


def dispatch_backward_ref(dxs, slot):
    return combine_ref(dxs, slot, np.ones(slot.shape))


def grouped_ref(xs, offsets, w_hats, glu=False):
    """Sorted rows times their groups' weights ``w_hats[e][K, N]``; zeros past the last group."""
    xs = np.asarray(xs, dtype=np.float64)
    N = w_hats[0].shape[1]
    out = np.zeros((xs.shape[0], N // 2 if glu else N))
    for e, w in enumerate(w_hats):
        a, b = int(offsets[e]), int(offsets[e + 1])
        y = xs[a:b] @ np.asarray(w, dtype=np.float64)
        if glu:
            g, u = swiglu_split(y)
            y = silu(g) * u
        out[a:b] = y
    return out


def lora_ref(y, x, lora_a, lora_b, ids, scaling):
    out = np.array(y, dtype=np.float64)
    for m, a in enumerate(np.asarray(ids).tolist()):
        if 0 <= a < len(lora_a):
            t = np.asarray(lora_a[a], dtype=np.float64) @ np.asarray(x[m], dtype=np.float64)
            out[m] += float(scaling[a]) * (np.asarray(lora_b[a], dtype=np.float64) @ t)
    return out
