"""Plain float64 definitions of the operators around the caches: RMSNorm and its gradient, rotary
positions and their frequencies, the cache append, MLA attention with a window and sinks.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

from __future__ import annotations

import math

import numpy as np

from .dsa_oracle import E4M3_MAX, sparse_mla_token


def rmsnorm(x, weight, eps, residual=None):
    """(y, h, rstd): h = x + residual, y = h * rstd * weight, rstd = (mean(h^2) + eps)^-1/2 per row."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * np.asarray(weight, np.float64), h, rstd


def row_scales(v, group=0):
    """amax / 448, at least the smallest fp32, over each row (group 0) or each `group` columns of it; 1 where the
    maximum is 0."""
    v = np.abs(np.asarray(v, np.float64))
    if group:
        amax = np.stack([v[:, c:c + group].max(axis=1) for c in range(0, v.shape[1], group)], axis=1)
    else:
        amax = v.max(axis=1)
    return np.where(amax > 0, np.maximum(amax / E4M3_MAX, 2.0 ** -149), 1.0)


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None):
    """(dh, dw): the vector-Jacobian product of y(h, weight) with dy, plus dresidual on h."""
    dy, h, rstd = (np.asarray(a, np.float64) for a in (dy, h, rstd))
    g = dy * np.asarray(weight, np.float64)
    r = rstd[:, None]
    dh = r * (g - h * r * r * (g * h).mean(axis=1, keepdims=True))
    return dh + (0.0 if dresidual is None else np.asarray(dresidual, np.float64)), (dy * h * r).sum(axis=0)


def rope_frequencies(rot_dim, theta, scaling="plain", factor=1.0, original_ctx=0.0, beta_fast=32.0, beta_slow=1.0):
    """(freqs [rot_dim / 2], mscale): radians per position of each pair."""
    def dim_of(turns):
        return rot_dim * math.log(original_ctx / (2 * math.pi * turns)) / (2 * math.log(theta))

    if scaling == "ntk":
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    freqs, mscale = [], 1.0
    for i in range(rot_dim // 2):
        f = theta ** (-2 * i / rot_dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            low, high = max(math.floor(dim_of(beta_fast)), 0), min(math.ceil(dim_of(beta_slow)), rot_dim - 1)
            ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            f = f / factor * ramp + f * (1 - ramp)
            mscale = 0.1 * math.log(factor) + 1
        freqs.append(f)
    return np.array(freqs), mscale


def rope(x, positions, freqs, rot_offset, rot_dim, half, mscale=1.0, transpose=False):
    """x [rows, heads, dim] with the pairs of dims [rot_offset, rot_offset + rot_dim) turned."""
    out = np.array(x, np.float64)
    for i in range(rot_dim // 2):
        a, b = (i, i + rot_dim // 2) if half else (2 * i, 2 * i + 1)
        a, b = a + rot_offset, b + rot_offset
        angle = np.asarray(positions, np.float64)[:, None] * freqs[i]
        c, s = mscale * np.cos(angle), mscale * np.sin(angle) * (-1.0 if transpose else 1.0)
        u, v = out[:, :, a].copy(), out[:, :, b].copy()
        out[:, :, a], out[:, :, b] = u * c - v * s, u * s + v * c
    return out


def cache_rows(kv, kv_weight, eps, key, positions, freqs, half, key_half, key_rot_offset, mscale=1.0):
    """(latent rows [n, 576], indexer keys [n, d_I], both unrounded) that the append writes."""
    n, _, _ = rmsnorm(kv[:, :512], kv_weight, eps)
    r = rope(np.asarray(kv)[:, None, 512:], positions, freqs, 0, 64, half, mscale)[:, 0]
    k = rope(np.asarray(key)[:, None, :], positions, freqs, key_rot_offset, 64, key_half, mscale)[:, 0]
    return np.concatenate([n, r], axis=1), k


def window_positions(length, window, sinks):
    """Positions that the query at position length - 1 sees, ascending."""
    return np.array([s for s in range(length) if s > length - 1 - window or s < sinks], np.int64)


def window_mla_token(q, latent, length, window, sinks, sm_scale):
    """(out [H, 512], lse [H]) of the query at position length - 1; zeros and -inf with no key."""
    sel = window_positions(length, window, sinks)
    if len(sel) == 0:
        return np.zeros((q.shape[0], 512)), np.full(q.shape[0], -np.inf)
    return sparse_mla_token(q, latent, sel, sm_scale)
