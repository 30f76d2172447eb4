"""Plain fp64 CPU oracle of the stand-alone operators around the experts.

TEST INFRASTRUCTURE ONLY, like ``oracle.moe_oracle``: the definitions written
out with numpy in fp64, sharing no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def rms_norm(v, weight, eps, offset):
    v = np.asarray(v, np.float64)
    return v / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps) * (offset + np.asarray(weight, np.float64))


def combine_rows(rows, inv_pos, pair_weights):
    """sum_j pair_weights[t, j] * rows[inv_pos[t, j]]; positions outside the rows add nothing."""
    out = np.zeros((inv_pos.shape[0], rows.shape[1]))
    for t in range(inv_pos.shape[0]):
        for j in range(inv_pos.shape[1]):
            p = int(inv_pos[t, j])
            if 0 <= p < rows.shape[0]:
                out[t] += float(pair_weights[t, j]) * rows[p]
    return out


def block_norm(residual, branch, w_pre=None, w_post=None, gate=None, gate_sigmoid=False, residual_scale=1.0,
               branch_scale=1.0, eps=1e-6, offset=0.0, inv_pos=None, pair_weights=None):
    """(r', h) of the norms around a block; h is None without w_pre. gate broadcasts against [T, K]."""
    stream = 0.0 if residual is None else residual_scale * np.asarray(residual, np.float64)
    if branch is not None:
        b = np.asarray(branch, np.float64)
        if inv_pos is not None:
            b = combine_rows(b, inv_pos, pair_weights)
        if w_post is not None:
            b = rms_norm(b, w_post, eps, offset)
        if gate is not None:
            g = np.asarray(gate, np.float64)
            b = b * (1.0 / (1.0 + np.exp(-g)) if gate_sigmoid else g)
        stream = stream + branch_scale * b
    return stream, None if w_pre is None else rms_norm(stream, w_pre, eps, offset)


def quantize_rows(x, src_rows=None):
    """(codes, scales) of every selected row: 127 x / max|x| to the nearest whole
    number, halves to even; a missing row is empty, a row with a NaN or an
    infinity has scale NaN."""
    x = np.asarray(x, np.float64)
    src = np.arange(x.shape[0]) if src_rows is None else np.asarray(src_rows)
    codes = np.zeros((len(src), x.shape[1]), np.int8)
    scales = np.zeros(len(src), np.float64)
    for i, s in enumerate(src):
        if s < 0 or s >= x.shape[0]:
            continue
        if not np.all(np.isfinite(x[s])):
            scales[i] = np.nan
            continue
        top = np.max(np.abs(x[s]))
        if top > 0:
            codes[i] = np.rint(127.0 * x[s] / top).astype(np.int8)
            scales[i] = top / 127.0
    return codes, scales


def group_ranges(offsets, rows, experts):
    """[begin, end) of every expert: the offsets' running maximum clamped to [0, rows]."""
    if offsets is None:
        return [(0, rows)]
    o = np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, rows))
    return [(int(o[e]), int(o[e + 1])) for e in range(experts)]


def grouped_matmul(x, w, offsets=None, row_scales=None, channel_scales=None):
    """(y, covered): y [R, N] fp64 and the rows that belong to an expert."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    y = np.zeros((x.shape[0], w.shape[1]))
    covered = np.zeros(x.shape[0], bool)
    for e, (a, b) in enumerate(group_ranges(offsets, x.shape[0], w.shape[0])):
        y[a:b] = x[a:b] @ w[e].T
        if channel_scales is not None:
            y[a:b] *= np.asarray(row_scales, np.float64)[a:b, None] * np.asarray(channel_scales, np.float64)[e][None, :]
        covered[a:b] = True
    return y, covered
