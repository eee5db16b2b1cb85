"""Plain 64-bit implementations of the router, the row plan, the few-token expert layer and the adapters, with the
error bounds that the GPU tests hold the kernels to.

A rounding to nearest is off by at most half a step: 2^-8 relative for bf16, 2^-11 for fp16, 2^-24 for fp32. A chain
of n fp32 additions is off by at most n 2^-24 of the sum of its terms' magnitudes (tensor-core sums, which may
truncate instead of rounding, by twice that).
"""
import math

import numpy as np
import torch

BF16, F16, F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def groups(ids, E):
    """ids: nested lists [T][topk]. (group_offsets, row_index, pos) as numpy int32."""
    topk = len(ids[0]) if ids else 1
    flat = [e for row in ids for e in row]
    order = sorted(range(len(flat)), key=lambda i: (flat[i] if 0 <= flat[i] < E else E, i))
    counts = np.zeros(E, np.int64)
    for e in flat:
        if 0 <= e < E:
            counts[e] += 1
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    pos = np.full(len(flat), -1, np.int32)
    for r, i in enumerate(order[:off[-1]]):
        pos[i] = r
    return off, np.array([i // topk for i in order], np.int32), pos.reshape(len(ids), topk)


def route(logits, topk, sigmoid, renorm, scale):
    """logits: fp64 numpy [T, E]. (weights [T, topk], relative bound per weight, ids)."""
    T, E = logits.shape
    w, tol = np.zeros((T, topk)), np.zeros((T, topk))
    ids = np.full((T, topk), -1, np.int64)
    for t in range(T):
        l = [-math.inf if math.isnan(v) else min(v, float(np.finfo(np.float32).max)) for v in logits[t]]
        pick = [e for e in sorted(range(E), key=lambda e: (-l[e], e))[:topk] if l[e] > -math.inf]
        if not pick:
            continue
        m = max(l)
        if sigmoid:
            c = min(m, 0.0) if renorm else 0.0
            p = {e: math.exp(min(l[e], 0.0) - c) / (1 + math.exp(-abs(l[e]))) for e in pick}
            total = sum(p.values()) if renorm else 1.0
            span = max(abs(min(l[e], 0.0) - c) for e in pick)
        else:
            p = {e: math.exp(l[e] - m) for e in (pick if renorm else range(E)) if l[e] > -math.inf}
            total = sum(p.values())
            span = max(m - l[e] for e in pick)
        for j, e in enumerate(pick):
            w[t, j] = scale * p[e] / total
            ids[t, j] = e
        # the argument's rounding, two exponentials and their sum of E / 32 + 5 terms in a row, the divisions
        tol[t] = (2 * min(span, 110.0) + 2 * 3 + E / 32 + 5 + 6) * F32
    return w, tol, ids


def hadamard(b):
    i = np.arange(b)
    return np.array([[(-1) ** bin(x & y).count("1") for y in i] for x in i], np.float64)


def dequant(codes, sf_rows):
    """codes u8 [N, K/2], sf_rows u8 [N, K/32] -> fp64 [N, K]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    return GRID[c] * np.repeat(np.exp2(sf_rows.astype(np.float64) - 127), 32, axis=1)


def rotate(x, b):
    return (x.reshape(-1, b) @ hadamard(b)).reshape(x.shape) if b > 1 else x


def spread(e, b):
    """Error of a rotation's outputs from its inputs' errors: their sum over the block."""
    return np.repeat(e.reshape(-1, b).sum(1), b).reshape(e.shape) if b > 1 else e


def moe_layer(X, weights, off, row_index, pos, layer):
    """X fp64 [T, K]; layer: dict of numpy arrays wq_gu, sf_gu (row-major scales), wq_dn, sf_dn, inv_gu, inv_dn, b, b_dn.
    Returns (out, bound): the bf16 rounding of the output, plus what rounding x' and h' to fp16 (groups of 32 scaled by a
    power of two) and fp32 sums of K and I terms leave, carried through the layer to first order."""
    T, K = X.shape
    E, I2 = layer["wq_gu"].shape[:2]
    I, N = I2 // 2, layer["wq_dn"].shape[1]
    where = {int(p): (t, j) for t, row in enumerate(pos) for j, p in enumerate(row) if p >= 0}
    out, bound = np.zeros((T, N)), np.zeros((T, N))
    n = np.arange(I)
    gate, up = 128 * (n // 64) + n % 64, 128 * (n // 64) + 64 + n % 64

    def fp16_groups(v):
        # half a step of fp16: 2^-11 of the value, or 2^-25 after scaling a group's largest value to 2^-10 or more
        return F16 * np.abs(v) + 2.0 ** -15 * np.repeat(np.abs(v).reshape(len(v), -1, 32).max(2), 32, axis=1)

    for e in range(E):
        rows = [r for r in range(off[e], off[e + 1]) if r in where]
        if not rows:
            continue
        x = X[row_index[rows]] * (layer["inv_gu"][e] if layer["inv_gu"] is not None else 1.0)
        ex = spread(9 * F32 * np.abs(x), layer["b"])
        x = rotate(x, layer["b"])
        ex = ex + fp16_groups(x)
        W = dequant(layer["wq_gu"][e], layer["sf_gu"][e])
        gu = x @ W.T
        egu = ex @ np.abs(W).T + 2 * (K / 16 + 8) * F32 * (np.abs(x) @ np.abs(W).T)
        g, u, eg, eu = gu[:, gate], gu[:, up], egu[:, gate], egu[:, up]
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-g))
        h = g * s * u
        eh = 1.1 * np.abs(u) * eg + np.abs(g * s) * eu + 1.1 * eg * eu + 16 * F32 * np.abs(h)
        inv = layer["inv_dn"][e] if layer["inv_dn"] is not None else 1.0
        h, eh = h * inv, spread(eh * inv + 9 * F32 * np.abs(h * inv), layer["b_dn"])
        h = rotate(h, layer["b_dn"])
        eh = eh + fp16_groups(h)
        W = dequant(layer["wq_dn"][e], layer["sf_dn"][e])
        y, ey = h @ W.T, eh @ np.abs(W).T + 2 * (I / 16 + 64) * F32 * (np.abs(h) @ np.abs(W).T)
        for i, r in enumerate(rows):
            t, j = where[r]
            out[t] += weights[t, j] * y[i]
            bound[t] += abs(weights[t, j]) * (ey[i] + 64 * F32 * np.abs(y[i]))
    return out, bound * (1 + BF16) + BF16 * np.abs(out) + 2.0 ** -133


def lora(Y, X, A, B, scale, off, row_index, rounding):
    """fp64 tensors; rounding: half a step of the output type. Returns (out, bound): fp32 sums, X A^T in bf16 for bf16 outputs
    (half a step of it, 2^-8 of each of its values) and in all of fp32's bits otherwise, the output's rounding."""
    out, bound = Y.clone(), torch.zeros_like(Y)
    K, r = X.shape[1], A.shape[1]
    for a in range(A.shape[0]):
        rows = row_index[off[a]:off[a + 1]].long()
        if not len(rows):
            continue
        x, s = X[rows], (scale[a] if scale is not None else 1.0)
        v, mag = x @ A[a].T, x.abs() @ A[a].abs().T
        ev = 2 * (K / 16 + 16) * F32 * mag + (BF16 * v.abs() if rounding == BF16 else 0.0)
        out[rows] += s * (v @ B[a].T)
        bound[rows] += abs(s) * (ev @ B[a].abs().T + 2 * (r + 8) * F32 * (v.abs() @ B[a].abs().T))
    return out, bound * (1 + rounding) + rounding * out.abs() + 2 * F32 * Y.abs() + 2.0 ** -133
