"""Plain 64-bit forms of the rotation, the 4-bit cache, its attention and the token log probabilities."""
from __future__ import annotations

import numpy as np

from sparse_attention_decode_pages_gb300 import workloads as wl

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16(x):
    """float64 values rounded to bf16 (through float32; the inputs of the tests are bf16 already)."""
    return wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(np.asarray(x, np.float32))).astype(np.float64)


# ---------------------------------------------------------------- rotation

def rope_table(n_pos, rot, theta=10000.0):
    """float32 [n_pos][2][rot / 2]."""
    if rot == 0:
        return np.zeros((n_pos, 2, 0), np.float32)
    ang = np.arange(n_pos)[:, None] * theta ** (-np.arange(0, rot, 2) / rot)
    return np.stack([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def norm_rope(x, weight, table, positions, eps, interleaved):
    """x [rows][heads][D] (float64), one position a row: the rotated rows and, for tolerances, the sums of
    the magnitudes that each output is made of."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    rot = 2 * table.shape[2]
    y, mag = x.copy(), np.abs(x)
    for row, p in enumerate(positions):
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = float(table[p, 0, i]), float(table[p, 1, i])
            y[row, :, a] = x[row, :, a] * c - x[row, :, b] * s
            y[row, :, b] = x[row, :, b] * c + x[row, :, a] * s
            mag[row, :, a] = mag[row, :, b] = np.abs(x[row, :, a]) + np.abs(x[row, :, b])
    return y, mag


# ---------------------------------------------------------------- the 4-bit format

def e4m3_values():
    """The values of the 127 non-negative e4m3 bytes (0x7f is NaN)."""
    b = np.arange(128)
    e, f = b >> 3, b & 7
    v = np.where(e > 0, (8 + f) * 2.0 ** (e - 10.0), f * 2.0 ** -9)
    return v[:127]


def _nearest_even(v, grid):
    """Index of the nearest grid value to each v >= 0, ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - v, v - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def kv4_quantise(x, exp):
    """Codes (0..15) and scale bytes of x [..][D] (float64 bf16 values)."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // 16, 16) / 2.0 ** exp
    mag = np.where(np.isnan(g), 0.0, np.abs(g))
    grid = e4m3_values()
    scale = _nearest_even(np.minimum(mag.max(-1) / 6, grid[-1]), grid)
    s = grid[scale][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        a = np.where(s > 0, mag / s, 0.0)
    codes = _nearest_even(np.minimum(a, 6.0), E2M1) + 8 * np.where(np.isnan(g), False, np.signbit(g))
    return codes.reshape(x.shape).astype(np.uint8), scale.astype(np.uint8)


def kv4_values(codes, scale, exp):
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.append(e4m3_values(), np.nan)[scale & 127] * 2.0 ** exp
    return (v.reshape(*scale.shape, 16) * s[..., None]).reshape(codes.shape)


def kv4_pack(codes, scale):
    """A tile's bytes [ps * D * 9 / 16] from codes [ps][D] and scale bytes [ps][D / 16]."""
    return np.concatenate([(codes[:, 0::2] | codes[:, 1::2] << 4).reshape(-1), scale.reshape(-1)])


def kv4_unpack(tile, ps, D):
    c = tile[: ps * D // 2].reshape(ps, D // 2)
    return np.stack([c & 15, c >> 4], -1).reshape(ps, D), tile[ps * D // 2:].reshape(ps, D // 16)


# ---------------------------------------------------------------- attention

def attention(q, k, v, scale, visible):
    """One query row q [D] over k, v [n][D]: o, lse, and what the tolerances are made of: sum p |v| and
    the largest scale * sum |q| |k|."""
    if not visible.any():
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0
    k, v = k[visible], v[visible]
    z = scale * (k @ q)
    m = z.max()
    p = np.exp(z - m)
    total = p.sum()
    return p @ v / total, m + np.log(total), p @ np.abs(v) / total, abs(scale) * (np.abs(k) @ np.abs(q)).max()


# ---------------------------------------------------------------- log probabilities

def logprobs(x, targets, inv_t, top_k):
    """x [rows][n] float64 logits."""
    rows = len(x)
    lse, ent, lp = np.zeros(rows), np.zeros(rows), np.zeros(rows)
    ids, tops = np.full((rows, top_k), -1, np.int64), np.full((rows, top_k), -np.inf)
    for r in range(rows):
        z = x[r] * inv_t
        live = z > -np.inf
        t = targets[r]
        if np.isnan(z).any():
            lse[r] = ent[r] = np.nan
            lp[r] = np.nan if t >= 0 else 0.0
        elif not live.any():
            lse[r], ent[r], lp[r] = -np.inf, 0.0, (-np.inf if t >= 0 else 0.0)
        else:
            m = z[live].max()
            lse[r] = m + np.log(np.exp(z[live] - m).sum())
            p = np.exp(z[live] - lse[r])
            ent[r] = -(p * (z[live] - lse[r])).sum()
            lp[r] = z[t] - lse[r] if t >= 0 else 0.0
        order = sorted((i for i in range(len(z)) if z[i] > -np.inf), key=lambda i: (-x[r, i], i))[:top_k]
        ids[r, : len(order)] = order
        tops[r, : len(order)] = z[order] - lse[r]
    return lp, ent, lse, ids, tops
