"""Plain 64-bit definitions of the adapter projection and of the experts' row
operators (numpy and torch on the CPU), with the error bounds that the GPU
tests hold the kernels to."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24      # half a step of fp32, relative
UB16 = 2.0 ** -8      # half a step of bf16, relative


def sort_ref(ids: np.ndarray, G: int):
    """(order, pos, m_sizes) by the definition: a stable sort by expert, the
    dropped slots (outside [0, G)) behind the others."""
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < G), flat, G).astype(np.int64)
    order = np.argsort(key, kind="stable")
    pos = np.empty(flat.size, dtype=np.int64)
    pos[order] = np.arange(flat.size)
    pos[key == G] = -1
    return order, pos.reshape(ids.shape), np.bincount(key, minlength=G + 1)[:G]


def gather_ref(x, pos, xs):
    """xs with the named rows replaced (float64 in, float64 out)."""
    out = xs.copy()
    T, k = pos.shape
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < len(out):
                out[pos[t, j]] = x[t]
    return out


def combine_ref(z, pos, w):
    """(y, bound): y[t] = sum_j w z; the bound counts k fp32 roundings of the
    sum of magnitudes and half a bf16 step of the result."""
    T, k = pos.shape
    y = np.zeros((T, z.shape[1]))
    mag = np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < len(z):
                term = (1.0 if w is None else float(w[t, j])) * z[pos[t, j]]
                y[t] += term
                mag[t] += np.abs(term)
    acc = 2 * k * U32 * mag
    return y, acc + UB16 * (np.abs(y) + acc)


def combine_grad_ref(dy, z, pos, w, dz):
    """(dz, its bound, dw, its bound): one fp32 product and one bf16 rounding
    for dz; width products and additions in fp32 for dw."""
    T, k = pos.shape
    dz = dz.copy()
    bz = np.zeros_like(dz)
    dw = np.zeros((T, k))
    bw = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = pos[t, j]
            if 0 <= p < len(z):
                dz[p] = float(w[t, j]) * dy[t]
                bz[p] = np.abs(dz[p]) * (UB16 * (1 + U32) + U32)
                dw[t, j] = np.dot(dy[t], z[p])
                bw[t, j] = (dy.shape[1] + 8) * U32 * np.dot(np.abs(dy[t]), np.abs(z[p]))
    return dz, bz, dw, bw


def lora_ref(x, q, s, a, b, ids, sc, group):
    """(y, bound) of the projection with adapters, float64 (x [M, K], q [N, K]
    nibbles, s [N, K/group], a [L, R, K], b [L, N, R], sc [L]).

    The bound adds up: half a bf16 step of y; the projection's fp32 sums (per
    group a chain of fp32 additions of x (128 + q) and of -136 sum x, magnitude
    at most |x| 279 s; group + 8 additions in a group, one per group and slice
    across them); the adapter's fp32 sum over K (K + 8 additions), its split
    into two bf16 parts (2^-16), and its fp32 sum over the rank (2 R + 4
    additions)."""
    M, K = x.shape
    N = q.shape[0]
    L, R = a.shape[0], a.shape[1]
    sf = np.repeat(s, group, axis=1)
    y = x @ (sf * (q - 8.0)).T
    acc = (group + K // group + 24) * U32 * (np.abs(x) @ (279.0 * sf).T)
    for l in range(L):
        rows = np.nonzero(ids == l)[0]
        if len(rows):
            h = sc[l] * (x[rows] @ a[l].T)
            hm = abs(sc[l]) * (np.abs(x[rows]) @ np.abs(a[l]).T)
            y[rows] += h @ b[l].T
            eh = (K + 8) * U32 * hm + 2.0 ** -16 * np.abs(h)
            acc[rows] += (eh + (2 * R + 4) * U32 * np.abs(h)) @ np.abs(b[l]).T
    return y, acc + UB16 * (np.abs(y) + acc)


def within(got: np.ndarray, ref: np.ndarray, bound: np.ndarray, what: str):
    assert np.all(np.isfinite(got)), f"{what}: {np.count_nonzero(~np.isfinite(got))} values not finite"
    # 1e-12 of the reference: its own rounding
    over = np.abs(got - ref) - bound - 1e-12 * np.abs(ref)
    i = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over[i] <= 0, \
        f"{what}: {np.count_nonzero(over > 0)} outside, at {i}: {got[i]} against {ref[i]}, bound {bound[i]}"


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()
