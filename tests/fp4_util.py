"""4-bit rows in plain torch, for the tests: the definition in include/sgemm.h step
by step, FP32 where it says FP32, and what the rows stand for in 64 bits."""
from __future__ import annotations

import torch

from dense_fp32_matrix_09_gb300 import sgemm

BLOCK = {sgemm.FP4_MX: 32, sgemm.FP4_NV: 16}
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def blocks_of(fmt, K):
    return -(-K // BLOCK[fmt])


def words_of(fmt, K):
    return -(-blocks_of(fmt, K) // 4)


def scale_index(fmt, rows, K):
    """Byte of row i, block b in the tiles (rows x blocks)."""
    i, b, words = torch.arange(rows)[:, None], torch.arange(blocks_of(fmt, K))[None, :], words_of(fmt, K)
    return ((i // 128) * words + b // 4) * 512 + (i % 32) * 16 + (i // 32) % 4 * 4 + b % 4


def tiled(fmt, scales, K, fill=0):
    """Scale bytes (rows x blocks) in tiles; rows behind the last filled with `fill`, blocks with 0."""
    rows, words = scales.shape[0], words_of(fmt, K)
    out = torch.full((-(-rows // 128), words, 32, 4, 4), fill, dtype=torch.uint8)
    full = torch.full((out.shape[0] * 128, words * 4), fill, dtype=torch.uint8)
    full[:rows] = 0
    full[:rows, :scales.shape[1]] = scales
    out[:] = full.view(-1, 4, 32, words, 4).permute(0, 3, 2, 1, 4)
    return out.reshape(-1)


def scale_values(fmt, scales):
    """Scale bytes in 64 bits."""
    if fmt == sgemm.FP4_MX:
        v = torch.exp2(scales.double() - 127)
        return torch.where(scales == 255, torch.full_like(v, float("nan")), v)
    return scales.view(torch.float8_e4m3fn).double()


def code_values(codes):
    v = GRID[(codes & 7).long()]
    return torch.where(codes >= 8, -v, v)


def unpack(Q, K):
    """Codes (rows x K) of packed rows."""
    b = Q[:, :(K + 1) // 2]
    return torch.stack((b & 15, b >> 4), dim=2).reshape(Q.shape[0], -1)[:, :K]


def pack(codes):
    if codes.shape[1] % 2:
        codes = torch.cat((codes, torch.zeros_like(codes[:, :1])), dim=1)
    return codes[:, ::2] | codes[:, 1::2] << 4


def values(fmt, codes, scales, row):
    """What rows stand for, in 64 bits."""
    K = codes.shape[1]
    x = code_values(codes) * scale_values(fmt, scales).repeat_interleave(BLOCK[fmt], dim=1)[:, :K]
    return x if row is None else x * row.double()[:, None]


def nearest_codes(x):
    """Codes of FP32 values: the nearest, a tie to the even code, 6 at most."""
    x = x.double()
    borders = (GRID[1:] + GRID[:-1]) / 2
    below, above = torch.bucketize(x.abs(), borders), torch.bucketize(x.abs(), borders, right=True)
    index = torch.where(below % 2 == 0, below, above)
    return (index + 8 * torch.signbit(x).long()).to(torch.uint8)


def quantize(fmt, v):
    """(codes, scale bytes, m) of FP32 rows by the definition; m the rows' largest magnitudes.
    Row scales: NV m / 2688 (see row_scales)."""
    v = v.float()
    M, K = v.shape
    n = BLOCK[fmt]
    full = torch.zeros(M, blocks_of(fmt, K) * n)
    full[:, :K] = v
    full = full.view(M, -1, n)
    top = full.abs().amax(dim=2)
    top = torch.where(full.isnan().any(dim=2), torch.full_like(top, float("nan")), top)
    m = top.amax(dim=1)
    m = torch.where(top.isnan().any(dim=1), torch.full_like(m, float("nan")), m)
    if fmt == sgemm.FP4_MX:
        number = torch.isfinite(top)
        _, e = torch.frexp(torch.where(number & (top > 0), top, torch.ones_like(top)).double())  # f in [0.5, 1)
        e = torch.where(top > 0, (e - 3).clamp(min=-127), torch.full_like(e, -127))
        byte = torch.where(number, e + 127, torch.full_like(e, 255))
        q = torch.where(number[:, :, None], full.double() / torch.exp2(e.double())[:, :, None], torch.zeros(1, dtype=torch.float64))
        codes = nearest_codes(q)
        codes[~number[:, :, None].expand_as(codes)] &= 0
        return codes.view(M, -1)[:, :K], byte.to(torch.uint8), m
    some = torch.isfinite(m) & (m >= 2688 * 2.0 ** -126)
    safe = torch.where(some, m, torch.ones_like(m))
    near, up = torch.tensor(448.0) / safe, torch.tensor(2688.0) / safe
    full = torch.where(some[:, None, None], full, torch.zeros(1))
    top = torch.where(some[:, None], top, torch.zeros(1))
    byte = (top * near[:, None]).to(torch.float8_e4m3fn)
    s = byte.float()
    f = torch.where(s > 0, up[:, None] / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(s))
    codes = nearest_codes(full * f[:, :, None])
    codes[(f == 0)[:, :, None].expand_as(codes)] &= 0
    return codes.view(M, -1)[:, :K], byte.view(torch.uint8), m


def row_scales(m):
    """NV: m / 2688 in FP32; 0 for rows too small, NaN for rows that are not finite."""
    r = m / torch.tensor(2688.0)
    r = torch.where(m < 2688 * 2.0 ** -126, torch.zeros_like(r), r)
    return torch.where(torch.isfinite(m), r, torch.full_like(r, float("nan")))


def random_rows(fmt, rows, K, gen, scales=(0.5, 1.0, 2.0)):
    """(codes, scale bytes, row): every code, scales and row scales powers of two near 1,
    so that sums of products are exact in FP32."""
    codes = torch.randint(0, 16, (rows, K), generator=gen, dtype=torch.uint8)
    s = torch.tensor(scales)[torch.randint(0, len(scales), (rows, blocks_of(fmt, K)), generator=gen)]
    byte = (torch.log2(s).round().to(torch.int32) + 127).to(torch.uint8) if fmt == sgemm.FP4_MX else \
        s.to(torch.float8_e4m3fn).view(torch.uint8)
    row = torch.tensor([0.5, 1.0, 2.0])[torch.randint(0, 3, (rows,), generator=gen)]
    return codes, byte, row
