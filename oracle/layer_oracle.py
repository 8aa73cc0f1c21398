"""Plain CPU oracle of the feed-forward layer with experts and of the fp8 linear layers.

TEST INFRASTRUCTURE ONLY, like ``awq_oracle``: slow, readable restatements of the formulas, in float64 where a result is
a rounded number and in float32, operation by operation, where it is defined bit for bit (e4m3 codes and their scales).
16-bit values travel as float32.  The prepared layout is written here from its definition.
"""

from __future__ import annotations

import numpy as np

from .awq_oracle import AWQ_ORDER, unpack

f32 = np.float32


# ---- router and plan

def route(logits, top_k: int, normalize: bool):
    """(weights float64 [T, top_k], ids [T, top_k]): the largest first, of equals the lowest expert; no NaN, no +inf."""
    x = np.asarray(logits, np.float64)
    ids = np.argsort(-x, axis=1, kind="stable")[:, :top_k]
    top = x.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        p = np.where(np.isneginf(top), 0.0, np.exp(x - np.where(np.isneginf(top), 0.0, top)))
        chosen = np.take_along_axis(p, ids, 1)
        total = (chosen if normalize else p).sum(axis=1, keepdims=True)
        weights = np.where(total > 0, chosen / total, 0.0)
    return weights, ids.astype(np.int32)


def plan(ids, experts: int):
    """(offsets, order, place): positions of each expert's choices, in order; -1 where a choice has no expert."""
    ids = np.asarray(ids).reshape(-1)
    order = np.full(len(ids), -1, np.int32)
    place = np.full(len(ids), -1, np.int32)
    offsets = np.zeros(experts + 1, np.int32)
    row = 0
    for e in range(experts):
        offsets[e] = row
        for i in np.flatnonzero(ids == e):
            order[row], place[i] = i, row
            row += 1
    offsets[experts] = row
    return offsets, order, place


# ---- weights

def dequantize(qweight, qzeros, scales):
    """float64 [K, N] of one layer: (q - z) s, exact; scales float32 [K / 128, N]."""
    q = unpack(qweight).astype(np.int32)
    z = np.full((scales.shape[0], q.shape[1]), 8, np.int32) if qzeros is None else unpack(qzeros).astype(np.int32)
    rep = np.repeat(np.arange(scales.shape[0]), 128)
    return (q - z[rep]).astype(np.float64) * scales[rep].astype(np.float64)


def prepack(qweight, qzeros, scale_bits, gated: bool) -> np.ndarray:
    """uint8 [experts, tiles, K / 128, 17024]: byte by byte what the prepared layout says."""
    E, K, nw = qweight.shape
    N, groups = nw * 8, K // 128
    half = N // 2
    tiles = -(-half // 128) if gated else -(-N // 256)
    out = np.zeros((E, tiles, groups, 17024), np.uint8)
    for e in range(E):
        q = unpack(qweight[e]).astype(np.uint8)
        z = np.full((groups, N), 8, np.uint8) if qzeros is None else unpack(qzeros[e]).astype(np.uint8)
        for j in range(tiles):
            for c in range(256):
                if gated:
                    n = 128 * j + c % 128
                    n = n + half * (c // 128) if n < half else N
                else:
                    n = 256 * j + c
                if n >= N:
                    continue
                for g in range(groups):
                    unit = out[e, j, g]
                    codes = q[128 * g:128 * g + 128, n]
                    for chunk in range(4):
                        at = (c // 128) * 8192 + chunk * 2048 + ((c % 128) ^ (2 * chunk)) * 16
                        for w in range(4):
                            word = 0
                            for i in range(8):
                                word |= int(codes[32 * chunk + 8 * w + AWQ_ORDER[i]]) << (4 * i)
                            p = w ^ (chunk // 2)
                            unit[at + 4 * p:at + 4 * p + 4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
                    unit[16384 + c // 2] |= int(z[g, n]) << (4 * (c % 2))
                    unit[16512 + 2 * c:16512 + 2 * c + 2] = np.frombuffer(np.uint16(scale_bits[e, g, n]).tobytes(), np.uint8)
    return out


# ---- the products

def silu(v):
    v = np.asarray(v, np.float64)
    return v / (1.0 + np.exp(-v))


def grouped(x, weights, offsets, src):
    """float64 [R, N] and the sum of the terms' magnitudes: row r of expert e is x[src[r]] W_e (zeros for src < 0)."""
    R = len(src)
    N = weights[0].shape[1]
    y, mag = np.zeros((R, N)), np.zeros((R, N))
    for e in range(len(weights)):
        for r in range(offsets[e], offsets[e + 1]):
            if src[r] >= 0:
                row = x[src[r]].astype(np.float64)
                y[r] = row @ weights[e].astype(np.float64)
                mag[r] = np.abs(row) @ np.abs(weights[e].astype(np.float64))
    return y, mag


# ---- e4m3

def e4m3_values() -> np.ndarray:
    """The 256 codes' values (NaN for 0x7F and 0xFF), from sign, exponent (bias 7) and 3 bits of mantissa."""
    out = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        if c & 127 == 127:
            v = np.nan
        out[c] = -v if c & 128 else v
    return out


def e4m3_codes(v) -> np.ndarray:
    """Codes nearest to float32 v (|v| <= 464), of two equally near the one with an even mantissa; the sign is kept."""
    table = e4m3_values()[:127]
    a = np.abs(np.asarray(v, np.float64))
    above = np.clip(np.searchsorted(table, a), 0, 126)
    below = np.maximum(above - 1, 0)
    up, down = table[above] - a, a - table[below]
    code = np.where((up < down) | ((up == down) & (above % 2 == 0)) | (a >= 448.0), above, below)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def fp8_quant(x):
    """(codes uint8 [M, K], scales float32 [ceil(K / 128), M]) of float32 x [M, K]."""
    M, K = x.shape
    groups = -(-K // 128)
    codes, scales = np.zeros((M, K), np.uint8), np.zeros((groups, M), f32)
    for g in range(groups):
        part = x[:, 128 * g:128 * g + 128].astype(f32)
        with np.errstate(invalid="ignore", divide="ignore"):
            s = np.max(np.abs(part), axis=1) / f32(448)
            s[~np.isfinite(part).all(axis=1)] = np.nan
            ok = np.isfinite(s) & (s > 0)
            q = part / np.where(ok, s, f32(1))[:, None]
            codes[:, 128 * g:128 * g + 128] = np.where(ok[:, None], e4m3_codes(np.where(ok[:, None], q, 0)), 0)
        scales[g] = s
    return codes, scales


def fp8_gemm(xq, s_x, wq, s_w):
    """float64 [M, N] and the terms' magnitudes, from codes and scales."""
    table = e4m3_values()
    M, K = xq.shape
    N = wq.shape[0]
    y, mag = np.zeros((M, N)), np.zeros((M, N))
    block = np.arange(N) // 128
    for g in range(-(-K // 128)):
        a, w = table[xq[:, 128 * g:128 * g + 128]], table[wq[:, 128 * g:128 * g + 128]]
        s = s_x[g].astype(np.float64)[:, None] * s_w[block, g].astype(np.float64)[None]
        y += (a @ w.T) * s
        mag += (np.abs(a) @ np.abs(w).T) * np.abs(s)
    return y, mag
