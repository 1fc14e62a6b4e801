"""Plain 64-bit forms of the paged cache (numpy)."""
from __future__ import annotations

import numpy as np
import torch


def as64(t) -> np.ndarray:
    return t.detach().to("cpu", torch.float64).numpy()


def keys64(pool, table, n: int) -> np.ndarray:
    """The first ``n`` keys of a sequence: pool [pages, rows, F], its row of the page table."""
    size = pool.shape[1]
    ids = table[:-(-n // size)].long()
    return as64(pool[ids.to(pool.device)]).reshape(len(ids) * size, pool.shape[2])[:n]


def ancestors(parents) -> list:
    """Per node the list of its ancestors and itself, from the top."""
    out = []
    for j, p in enumerate(parents):
        out.append((out[p] if p >= 0 else []) + [j])
    return out


def mask_words(lists, n: int) -> np.ndarray:
    """Node lists as 64-bit words."""
    words = -(-n // 64)
    out = np.zeros((len(lists), words), dtype=np.uint64)
    for i, nodes in enumerate(lists):
        for j in nodes:
            out[i, j // 64] |= np.uint64(1 << (j % 64))
    return out.view(np.int64)


def seen(length: int, count: int, i: int, nodes=None) -> np.ndarray:
    """Keys that token i of a row's `count` new ones sees; nodes: its list in a tree."""
    first = length - count
    if i >= count:
        at = []
    elif nodes is None:
        at = range(0, first + i + 1)
    else:
        at = list(range(0, first)) + [first + j for j in sorted(nodes) if j < count and first + j >= 0]
    return np.array(list(at), dtype=np.int64)


def attend64(q, lat, rope, scale: float):
    """q [H, D] over keys lat / rope [T, .]: ctx [H, rank], lse [H]."""
    if len(lat) == 0:
        return np.zeros((q.shape[0], lat.shape[1])), np.full(q.shape[0], -np.inf)
    s = (q @ np.concatenate([lat, rope], 1).T) * scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(1, keepdims=True)
    return (p / total) @ lat, (m + np.log(total))[:, 0]


def rms_norm64(x, w, eps: float) -> np.ndarray:
    with np.errstate(invalid="ignore", divide="ignore"):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def rotate64(x, pos, theta: float) -> np.ndarray:
    """x [n, d] pair-interleaved, pos [n]: the angles' roundings are the operator's."""
    d = x.shape[1]
    j = np.arange(d // 2)
    inv = np.power(np.float64(np.float32(theta)), (-2.0 * j / d).astype(np.float32).astype(np.float64)).astype(np.float32)
    a = (pos[:, None].astype(np.float64) * inv.astype(np.float64)).astype(np.float32).astype(np.float64)
    re, im = x[:, 0::2], x[:, 1::2]
    return np.concatenate([re * np.cos(a) - im * np.sin(a), im * np.cos(a) + re * np.sin(a)], 1)
