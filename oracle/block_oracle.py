"""Plain CPU oracle of the operators between the linear layers of a decoder block.

TEST INFRASTRUCTURE ONLY, like ``awq_oracle``: slow, readable restatements of the formulas, in float64 where a
result is a rounded number and in float32, operation by operation, where the result is defined bit for bit
(codes, scales, rotations).  Two 16-bit types travel as their float32 values; ``round16`` rounds to them.

The cache layout is written here from its definition, as explicit byte and bit positions.
"""

from __future__ import annotations

import numpy as np

from .awq_oracle import AWQ_ORDER, bf16_round, bf16_to_float

f32 = np.float32


def round16(x, bf16: bool) -> np.ndarray:
    """float32 -> the nearest fp16 or bf16 value, as float32."""
    x = np.asarray(x, dtype=f32)
    return bf16_to_float(bf16_round(x)).astype(f32) if bf16 else x.astype(np.float16).astype(f32)


# ---- norm

def rmsnorm(x, residual, weight, eps: float):
    """(y, h) in float64: h = x + residual, y = h w / sqrt(mean(h^2) + eps)."""
    h = x.astype(np.float64) + (0.0 if residual is None else residual.astype(np.float64))
    return h * weight.astype(np.float64) / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps), h


def rmsnorm_codes(x, residual, weight, eps: float):
    """(codes int8, scale float64): codes from t = h w in float32, one rounding for each operation."""
    h = x.astype(f32) if residual is None else x.astype(f32) + residual.astype(f32)
    t = h * weight.astype(f32)
    step = np.max(np.abs(t), axis=1, keepdims=True) / f32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        codes = np.where(step > 0, np.clip(np.rint(t / step), -128, 127), 0)
    _, h64 = rmsnorm(x, residual, weight, eps)
    rstd = 1.0 / np.sqrt(np.mean(h64 * h64, axis=1) + eps)
    return codes.astype(np.int8), step[:, 0].astype(np.float64) * rstd


# ---- rotation

def rope_table(positions: int, rot: int, base: float = 10000.0) -> np.ndarray:
    """float32 [positions, rot]: rot / 2 cosines, then rot / 2 sines, of position * base^(-2i / rot)."""
    angle = np.arange(positions, dtype=np.float64)[:, None] * base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(f32)


def rope(x, row, interleaved: bool) -> np.ndarray:
    """One head (float32 [D]) turned by one table row (float32 [rot]), operation by operation in float32."""
    out, half = x.astype(f32).copy(), len(row) // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = row[i], row[half + i]
        out[a] = f32(f32(x[a] * c) - f32(x[b] * s))
        out[b] = f32(f32(x[b] * c) + f32(x[a] * s))
    return out


# ---- the 4-bit cache

UNIT = 16


def kv4_unit_bytes(dim: int) -> int:
    return 16 * dim + 128


def kv4_quantize(x):
    """(codes uint8, scale, zero float16) over the last axis of float32 x."""
    x = x.astype(f32)
    low, high = x.min(axis=-1), x.max(axis=-1)
    scale = np.minimum((high - low) / f32(15), f32(65504)).astype(np.float16)
    zero = np.clip(low, f32(-65504), f32(65504)).astype(np.float16)
    s, z = scale.astype(f32)[..., None], zero.astype(f32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        codes = np.where(s > 0, np.clip(np.rint((x - z) / s), 0, 15), 0)
    return codes.astype(np.uint8), scale, zero


def kv4_place(dim: int, token: int, channel: int, value: bool) -> tuple[int, int]:
    """(byte of the unit, bit shift in the byte) of one code."""
    if not value:
        nibble = AWQ_ORDER.index(channel % 8)
        return token * (dim // 2) + channel // 8 * 4 + nibble // 2, 4 * (nibble % 2)
    wide = dim // 8
    half = (((token // 8) * 8 + channel // wide) * 4 + token % 8 // 2) * (wide // 4) + channel % wide // 4
    return 8 * dim + 4 * half + 2 * (token % 2) + channel % 4 // 2, 4 * (channel % 2)


def _places(dim: int, value: bool):
    at = np.array([[kv4_place(dim, t, c, value) for c in range(dim)] for t in range(UNIT)])
    return at[..., 0], at[..., 1]


def kv4_write(cache, slot: int, head: int, kcode, ks, kz, vcode, vs, vz) -> None:
    """One token of one head into a cache uint8 [pages, kv_heads, page_size / 16, unit]."""
    pages, _, units, unit = cache.shape
    dim = (unit - 128) // 16
    page, rest = divmod(slot, units * UNIT)
    u = cache[page, head, rest // UNIT]
    t = rest % UNIT
    for value, codes in ((False, kcode), (True, vcode)):
        for c in range(dim):
            byte, shift = kv4_place(dim, t, c, value)
            u[byte] = (int(u[byte]) & (0xF0 >> shift)) | (int(codes[c]) << shift)
    u[16 * dim + 8 * t: 16 * dim + 8 * t + 8] = np.array([ks, kz, vs, vz], dtype=np.float16).view(np.uint8)


def kv4_pack(kcode, vcode, meta) -> np.ndarray:
    """A whole cache from codes [pages, kv_heads, page_size, D] and meta float16 [pages, kv_heads, page_size, 4]."""
    pages, heads, size, dim = kcode.shape
    cache = np.zeros((pages, heads, size // UNIT, kv4_unit_bytes(dim)), dtype=np.uint8)
    for value, codes in ((False, kcode), (True, vcode)):
        byte, shift = _places(dim, value)
        codes = codes.reshape(pages, heads, size // UNIT, UNIT, dim)
        for s in (0, 4):  # every byte has one low and one high nibble
            t, c = np.nonzero(shift == s)
            cache[..., byte[t, c]] |= codes[..., t, c] << s
    cache[..., 16 * dim:] = np.ascontiguousarray(
        meta.reshape(pages, heads, size // UNIT, UNIT * 4)).view(np.uint8).reshape(pages, heads, size // UNIT, 128)
    return cache


def kv4_read(cache, slots, head: int):
    """(key code, key scale, key zero, value code, value scale, value zero) of `slots` (int array) of one head."""
    pages, _, units, unit = cache.shape
    dim = (unit - 128) // 16
    slots = np.asarray(slots, dtype=np.int64)
    u = cache[slots // (units * UNIT), head, slots % (units * UNIT) // UNIT]
    t = slots % UNIT
    out = []
    meta = np.ascontiguousarray(u[:, 16 * dim:]).view(np.float16).reshape(-1, UNIT, 4)[np.arange(len(slots)), t]
    for value in (False, True):
        byte, shift = _places(dim, value)
        code = u[np.arange(len(slots))[:, None], byte[t]] >> shift[t] & 15
        out += [code, meta[:, 2 * value].astype(f32), meta[:, 2 * value + 1].astype(f32)]
    return tuple(out)


def kv4_dequant(code, scale, zero) -> np.ndarray:
    """zero + code * scale in float32, each operation rounded once."""
    return zero[:, None] + code.astype(f32) * scale[:, None]


def kv4_attention(q, cache, block_table, kv_len, q_start, scale: float, window: int = 0):
    """(out, lse, mag, reach) in float64 for q float32 [T, heads, D].

    mag[row, d] = sum_j p_j (u scale + |zero|) and reach[row] = |scale| max_j sum_d |q_d| (u scale + |zero|) are
    the sizes that rounding errors of the value product and of the scores are relative to.
    """
    T, heads, dim = q.shape
    kv_heads, size = cache.shape[1], cache.shape[2] * UNIT
    per = heads // kv_heads
    out, mag = np.zeros((T, heads, dim)), np.zeros((T, heads, dim))
    lse, reach = np.full((T, heads), -np.inf), np.zeros((T, heads))
    for b, length in enumerate(kv_len):
        length, begin, end = int(length), int(q_start[b]), int(q_start[b + 1])
        if length <= 0 or end <= begin:
            continue
        at = np.arange(length)
        slots = block_table[b][at // size].astype(np.int64) * size + at % size
        for kvh in range(kv_heads):
            ku, ks, kz, vu, vs, vz = (x.astype(np.float64) for x in kv4_read(cache, slots, kvh))
            k, v = kz[:, None] + ku * ks[:, None], vz[:, None] + vu * vs[:, None]
            kmag, vmag = np.abs(kz)[:, None] + ku * np.abs(ks)[:, None], np.abs(vz)[:, None] + vu * np.abs(vs)[:, None]
            rows = q[begin:end, kvh * per:(kvh + 1) * per].astype(np.float64)  # [n, per, D]
            pos = length - (end - begin) + np.arange(end - begin)
            seen = at[None] <= pos[:, None]
            if window > 0:
                seen &= at[None] > pos[:, None] - window
            s = np.where(seen[:, None], scale * (rows @ k.T), -np.inf)
            some = seen.any(axis=1)
            if not some.any():
                continue
            s, top = s[some], s[some].max(axis=2, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(axis=2, keepdims=True)
            sel, hs = begin + np.nonzero(some)[0], slice(kvh * per, (kvh + 1) * per)
            out[sel, hs] = (p / total) @ v
            mag[sel, hs] = (p / total) @ vmag
            lse[sel, hs] = (top + np.log(total))[..., 0]
            size_of = np.where(seen[some][:, None], np.abs(scale) * (np.abs(rows[some]) @ kmag.T), 0.0)
            reach[sel, hs] = size_of.max(axis=2)
    return out, lse, mag, reach
