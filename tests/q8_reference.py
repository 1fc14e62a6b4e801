"""Plain 64-bit forms of the 8-bit cache, the attention weights and the eviction (numpy)."""
from __future__ import annotations

import numpy as np
import torch

E_MIN, E_MAX = 64, 134


def codes64(codes) -> np.ndarray:
    """Values of e4m3 codes (uint8) in units, from their bits."""
    n = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    mant, ex = n & 7, (n >> 3) & 15
    mag = np.where(ex == 0, mant * 2.0 ** -9, (8.0 + mant) * np.exp2(ex - 10.0))
    v = np.where(n >= 128, -mag, mag)
    return np.where((n & 127) == 127, np.nan, v)


def held64(codes, scales, block: int) -> np.ndarray:
    """``codes`` [T, rank], ``scales`` [blocks] -> values [T, rank]."""
    e = np.clip(np.asarray(scales).astype(np.int64), E_MIN, E_MAX)[np.arange(len(codes)) // block]
    return codes64(codes) * np.exp2(e - 127.0)[:, None]


def nearest_e4m3(x) -> np.ndarray:
    """The e4m3 value nearest to ``x`` (ties to even, saturating at 448)."""
    a = np.minimum(np.abs(x), 448.0)
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.copysign(np.round(a / step) * step, x)


def exponent64(amax: float) -> int:
    """The smallest exponent byte whose unit holds ``amax`` in 448 units."""
    if not np.isfinite(amax):
        return E_MAX
    f, k = np.frexp(amax)                      # amax = 2f * 2^(k-1), 448 = 1.75 * 2^8
    return int(np.clip(E_MIN if amax == 0 else 127 + k - 9 + (f > 0.875), E_MIN, E_MAX))


def near_exponent_border(amax: float, slack: float) -> bool:
    """Whether a relative change of ``slack`` may change the exponent."""
    return amax == 0 or exponent64(amax * (1 + slack)) != exponent64(amax * (1 - slack))


def rms_norm64(x, w, eps: float) -> np.ndarray:
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def scores64(q, keys, scale: float) -> np.ndarray:
    """q [H, D], keys [T, D] -> [H, T]."""
    return (q @ keys.T) * scale


def attend64(q, lat, rope, scale: float, at=None):
    """One query row: q [H, D], lat / rope [visible T, .]; ``at`` lists positions (a multiset).
    Returns ctx [H, rank] and lse [H]."""
    if at is not None:
        lat, rope = lat[at], rope[at]
    H = q.shape[0]
    if len(lat) == 0:
        return np.zeros((H, lat.shape[1])), np.full(H, -np.inf)
    s = scores64(q, np.concatenate([lat, rope], 1), scale)
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(1, keepdims=True)
    return (p / total) @ lat, (m + np.log(total))[:, 0]


def key_weights64(q, lat, rope, lse, w, scale: float, decay: float, n_new: int) -> np.ndarray:
    """One batch row: q [s_q, H, D], the window's lat / rope [T, .], lse [s_q, H], w [T]."""
    T, s_q = len(lat), q.shape[0]
    out = np.where(np.arange(T) < T - n_new, decay * w if decay else 0.0, 0.0)
    keys = np.concatenate([lat, rope], 1)
    for i in range(s_q):
        limit = min(T, T - s_q + 1 + i)
        if limit > 0:
            out[:limit] += np.exp(scores64(q[i], keys[:limit], scale) - lse[i][:, None]).sum(0)
    return out


def evict64(w, n: int, keep: int, sink: int, recent: int):
    """Kept window positions of a row of n tokens with weights w[n] (f32), or None when all stay."""
    if n <= keep:
        return None
    bits = np.asarray(w, dtype=np.float32).view(np.uint32)
    order = np.where(bits >> 31, ~bits, bits ^ np.uint32(0x80000000)).astype(np.int64)
    middle = np.arange(sink, n - recent)
    best = sorted(middle.tolist(), key=lambda p: (-order[p], p))[:keep - sink - recent]
    return np.array(list(range(sink)) + sorted(best) + list(range(n - recent, n)), dtype=np.int32)


def as64(t) -> np.ndarray:
    return t.detach().to("cpu", torch.float64).numpy()
