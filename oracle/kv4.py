"""The 4-bit paged cache's format and the rotary rotation, element by element in 64
bits -- TEST INFRASTRUCTURE, NOT PRODUCT CODE.

Layout, per page and KV head: units of 32 keys, each [K codes 16 d bytes][V codes
16 d][K pairs][V pairs] (pairs: scale then min, 16 bits each).  With J = min(d / 32, 4):
K word ((32 c + key) * 4 + t) * J + j holds dims 32 (J c + j) + 8 t + n, n = 0..7, in
nibble n; V word ((((key / 8) * d / 32 / J + c) * 8 + g) * 4 + key % 8 / 2) * J + j holds
dims 32 (J c + j) + 4 g + n, n = 0..3, in nibble n + 4 (key % 2).
"""
from __future__ import annotations

import numpy as np
import torch


def unit_bytes(d: int, group: int) -> int:
    return 32 * d + 2 * 32 * (d // group) * 4


def k_nibble(d: int, key: int, dim: int) -> int:
    """Nibble of a unit (two per byte, the low one first) that holds K[key, dim]."""
    J = min(d // 32, 4)
    block, t, n = dim // 32, dim % 32 // 8, dim % 8
    c, j = divmod(block, J)
    return 8 * (((32 * c + key) * 4 + t) * J + j) + n


def v_nibble(d: int, key: int, dim: int) -> int:
    J = min(d // 32, 4)
    block, g, n = dim // 32, dim % 32 // 4, dim % 4
    c, j = divmod(block, J)
    word = ((((key // 8) * (d // 32 // J) + c) * 8 + g) * 4 + key % 8 // 2) * J + j
    return 32 * d + 8 * word + 4 * (key % 2) + n


_MAPS: dict = {}


def _maps(d: int):
    """Nibble indices [32, d] of K and V in a unit."""
    if d not in _MAPS:
        _MAPS[d] = tuple(np.array([[f(d, r, x) for x in range(d)] for r in range(32)]) for f in (k_nibble, v_nibble))
    return _MAPS[d]


def bits16(x: torch.Tensor) -> np.ndarray:
    """Bit patterns of bf16 / fp16 values."""
    return x.contiguous().view(torch.int16).numpy().view(np.uint16)


def from_bits16(u: np.ndarray, dtype) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(u).view(np.int16).copy()).view(dtype)


def quantise(x: torch.Tensor, group: int):
    """Codes [..., d] (uint8) and pairs [..., d / group, 2] (x's type) of finite 16-bit rows x."""
    dt = x.dtype
    f = x.double().numpy()
    f = f.reshape(*f.shape[:-1], f.shape[-1] // group, group)
    mn, mx = f.min(-1, keepdims=True), f.max(-1, keepdims=True)
    s = torch.from_numpy((mx - mn) / 15).float().to(dt)
    s = torch.where(s.float() < 2.0 ** -100, torch.zeros_like(s), s)
    sd = s.double().numpy()
    code = np.where(sd > 0, np.minimum(np.rint((f - mn) / np.where(sd > 0, sd, 1.0)), 15), 0)
    pairs = torch.cat([s, torch.from_numpy(mn).to(dt)], -1)
    return code.reshape(*x.shape).astype(np.uint8), pairs


def values(codes: np.ndarray, pairs: torch.Tensor, group: int) -> np.ndarray:
    """min + scale * code in fp64."""
    p = pairs.double().numpy()
    c = codes.reshape(*codes.shape[:-1], codes.shape[-1] // group, group).astype(np.float64)
    return (p[..., 1:] + p[..., :1] * c).reshape(codes.shape)


def write(page: np.ndarray, first: int, kv, group: int) -> None:
    """Store rows first.. of one (page, head) (uint8 [page bytes]); kv = ((K codes, K pairs), (V codes, V pairs))."""
    n, d = kv[0][0].shape
    ng, ub = d // group, unit_bytes(d, group)
    for which in (0, 1):
        codes, pairs = kv[which]
        pb = bits16(pairs).reshape(n, ng, 2)
        for i in range(n):
            unit = page[(first + i) // 32 * ub:((first + i) // 32 + 1) * ub]
            r = (first + i) % 32
            at = _maps(d)[which][r]
            low = at % 2 == 0
            unit[at[low] // 2] = (unit[at[low] // 2] & 0xF0) | codes[i][low]
            unit[at[~low] // 2] = (unit[at[~low] // 2] & 0x0F) | (codes[i][~low] << 4)
            par = unit[32 * d + which * 128 * ng:][:128 * ng].view(np.uint16).reshape(32, ng, 2)
            par[r] = pb[i]


def read(page: np.ndarray, first: int, n: int, d: int, group: int, dtype):
    """((K codes, K pairs), (V codes, V pairs)) of n rows of one (page, head)."""
    ng, ub = d // group, unit_bytes(d, group)
    out = []
    for which in (0, 1):
        codes = np.zeros((n, d), np.uint8)
        pb = np.zeros((n, ng, 2), np.uint16)
        for i in range(n):
            unit = page[(first + i) // 32 * ub:((first + i) // 32 + 1) * ub]
            r = (first + i) % 32
            at = _maps(d)[which][r]
            codes[i] = (unit[at // 2] >> (4 * (at % 2))) & 15
            pb[i] = unit[32 * d + which * 128 * ng:][:128 * ng].view(np.uint16).reshape(32, ng, 2)[r]
        out.append((codes, from_bits16(pb, dtype).reshape(n, ng, 2)))
    return tuple(out)


def rotate(x, cos_sin, pos, interleaved: bool):
    """Rows x [n, h, d] turned by cos_sin [max_positions, R] at pos [n] (fp64), and the sum of the magnitudes
    of the two products of each element (0 where nothing turns)."""
    x = np.asarray(x, np.float64)
    R = cos_sin.shape[1]
    c, s = cos_sin[pos, None, :R // 2].astype(np.float64), cos_sin[pos, None, R // 2:].astype(np.float64)
    y, size = x.copy(), np.zeros_like(x)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = abs(x[..., a] * c) + abs(x[..., b] * s)
    size[..., b] = abs(x[..., b] * c) + abs(x[..., a] * s)
    return y, size
