"""Plain MX4 arithmetic for the tests, from the format's definition, in 64-bit
floats and integers on the tensor's own device.  Shares no code with the
library."""
import numpy as np
import torch

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def blocks_of(n):
    return -(-n // 32)


def power(e):
    """2.0 ** e in 64 bits, e an integer tensor."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def random16(blocks, seed):
    """The 32 sixteen-bit numbers of every block (Philox4x32-10, host)."""
    m, h = np.uint64(0xFFFFFFFF), np.uint64(32)
    n = np.arange(4 * blocks, dtype=np.uint64)
    c = [n & m, n >> h, np.zeros_like(n), np.zeros_like(n)]
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> h) ^ c[1] ^ np.uint64(k0), q & m, (p >> h) ^ c[3] ^ np.uint64(k1), p & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    out = np.stack([v for w in c for v in (w & np.uint64(0xFFFF), w >> np.uint64(16))], -1)
    return torch.from_numpy(out.reshape(blocks, 32).astype(np.int64))


def quantize(x, seed=None):
    """(codes [rows, blocks, 32] of 0..15, scale bytes [rows, blocks]) of a
    matrix in blocks along its rows; int64 tensors."""
    rows, cols = x.shape
    nb = blocks_of(cols)
    v = torch.zeros(rows, nb * 32, dtype=torch.float64, device=x.device)
    v[:, :cols] = x.double()
    v = v.view(rows, nb, 32)
    sign = torch.signbit(v)
    a = v.abs()
    bad = ~torch.isfinite(a).all(-1)
    a = torch.where(bad.unsqueeze(-1), 0.0, a)
    top = a.amax(-1)
    _, e = torch.frexp(top)
    s = torch.where(top > 0, e.to(torch.int64) - 1 - 2 + 127, 0).clamp(min=0)
    a = a / power(s - 127).unsqueeze(-1)  # exact: below 8
    grid = torch.tensor(MAGNITUDES + (8.0,), dtype=torch.float64, device=x.device)
    at = torch.bucketize(a, grid, right=True) - 1
    low, high = grid[at], grid[at + 1]
    if seed is None:
        mid = (low + high) / 2
        up = (a > mid) | ((a == mid) & (at % 2 == 1))
    else:
        r = random16(rows * nb, seed).to(x.device).view(rows, nb, 32)
        up = torch.floor((a - low) / (high - low) * 65536).to(torch.int64) + r >= 65536
    code = torch.minimum(at + up.to(torch.int64), torch.tensor(7, device=x.device))
    code = code + 8 * sign.to(torch.int64)
    return torch.where(bad.unsqueeze(-1), 0, code), torch.where(bad, 255, s)


def values(code, s, cols):
    """The 64-bit values of codes and scale bytes, [rows, cols]."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=torch.float64, device=code.device)
    unit = torch.where(s == 255, float("nan"), power(s.clamp(max=254) - 127))
    return (table[code] * unit.unsqueeze(-1)).flatten(-2)[:, :cols]


def rounded(x, seed=None):
    return values(*quantize(x, seed), x.shape[1])


def unpack(m):
    """(codes, scale bytes) of an MX4 matrix of the package, as quantize gives them."""
    nb = blocks_of(m.cols)
    b = m.codes[:, :16 * nb].to(torch.int64)
    return torch.stack([b & 15, b >> 4], -1).view(m.rows, nb, 32), m.scales[:, :nb].to(torch.int64)


def read(m):
    return values(*unpack(m), m.cols)


def pack(code, s, pitch=None, scale_pitch=None):
    """uint8 (codes, scales) tensors of a matrix, rows `pitch` / `scale_pitch` bytes apart."""
    rows, nb = s.shape
    flat = code.reshape(rows, nb * 32)
    c = torch.zeros(rows, pitch or 16 * nb, dtype=torch.uint8, device=s.device)
    c[:, :16 * nb] = (flat[:, 0::2] | (flat[:, 1::2] << 4)).to(torch.uint8)
    out = torch.zeros(rows, scale_pitch or nb, dtype=torch.uint8, device=s.device)
    out[:, :nb] = s.to(torch.uint8)
    return c, out
