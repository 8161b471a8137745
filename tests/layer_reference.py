"""Plain arithmetic of the 8-bit checkpoints, the norm and the embedding for the
tests, from their definitions, in 64-bit floats on the tensor's own device.
Shares no code with the library."""
import torch

U = 2.0 ** -24  # half a step of binary32, relative


def half_step(dtype):
    """Half a step of a type, relative, and half its smallest step."""
    info = torch.finfo(dtype)
    return info.eps / 2, info.smallest_normal * info.eps / 2


def power(e):
    """2.0 ** e in 64 bits, e an integer tensor (the device's pow need not be exact)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def grid8():
    """The magnitudes of E4M3 by their code, 0 .. 126."""
    return [i / 512 for i in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]


def quantize8(x):
    """(codes [rows, 32 blocks], scale bytes [rows, blocks]) of x's rows; int64."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    v = torch.zeros(rows, nb * 32, dtype=torch.float64, device=x.device)
    v[:, :cols] = x.double()
    v = v.view(rows, nb, 32)
    sign = torch.signbit(v).long()
    a = v.abs()
    bad = ~torch.isfinite(a).all(-1)
    a = torch.where(bad.unsqueeze(-1), 0.0, a)
    top = a.amax(-1)
    s = torch.full(top.shape, 3, dtype=torch.int64, device=x.device)
    for k in range(4, 247):  # the smallest that holds the largest element
        s = torch.where(top > 448 * 2.0 ** (k - 1 - 127), k, s)
    a = a / power(s - 127).unsqueeze(-1)
    grid = torch.tensor(grid8() + [480.0], dtype=torch.float64, device=x.device)
    at = torch.bucketize(a, grid, right=True) - 1
    at = at.clamp(max=126)  # over 448 (the largest scale only): 448
    low, high = grid[at], grid[at + 1]
    up = (a - low > high - a) | ((a - low == high - a) & (at % 2 == 1))
    code = (at + up.long()).clamp(max=126) + 128 * sign
    code = torch.where(bad.unsqueeze(-1), 0, code)
    return code.flatten(-2), torch.where(bad, 255, s)


def values8(codes, scales, cols):
    """The values of MX8 bytes, in 64 bits."""
    half = grid8() + [float("nan")]
    table = torch.tensor(half + [-v for v in half], dtype=torch.float64, device=codes.device)
    s = scales.long()
    unit = torch.where(s == 255, float("nan"), power(s - 127))
    v = table[codes.long()][:, :32 * s.shape[1]].view(s.shape[0], s.shape[1], 32) * unit.unsqueeze(-1)
    return v.flatten(-2)[:, :cols]


def norm(h, weight, eps):
    """(y, rstd) of rows of h."""
    h = h.double()
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    return h * rstd.unsqueeze(1) * weight.double(), rstd


def norm_backward(dy, h, weight, rstd, dh=None):
    """(dx, dw, bounds of their binary32 roundings but the last): a sum of n
    terms is off by at most U times the terms' magnitudes for every addition on
    a term's way, and each term takes three roundings here.  A row's sum: 32 in
    a thread, or one in 256 of a longer row's terms, and 12 that join threads
    and round the terms; dw's: less than one a row."""
    dy, h, w, r = dy.double(), h.double(), weight.double(), rstd.double().unsqueeze(1)
    n, rows = h.shape[1], h.shape[0]
    chain = min(n, 32 + n // 256) + 12
    xh, g = h * r, dy * w
    c = (g * xh).mean(1, keepdim=True)
    size = (g * xh).abs().mean(1, keepdim=True)
    dx = r * (g - xh * c)
    off = r * (3 * U * g.abs() + xh.abs() * (chain * U * size + 6 * U * c.abs()))
    if dh is not None:
        dx = dx + dh.double()
        off = off + 2 * U * dx.abs()
    dw = (dy * xh).sum(0)
    return dx, dw, off, (rows + 8) * U * (dy * xh).abs().sum(0)


def embedding_backward(dy, tokens, vocab, scale):
    """(dtable, the bound of its binary32 roundings but the last)."""
    here = (tokens >= 0) & (tokens < vocab)
    out = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device=dy.device)
    size, count = torch.zeros_like(out), torch.zeros(vocab, dtype=torch.float64, device=dy.device)
    for t in torch.nonzero(here).squeeze(1).tolist():
        v = int(tokens[t])
        out[v] += dy[t].double()
        size[v] += dy[t].double().abs()
        count[v] += 1
    return out * scale, (count.unsqueeze(1) + 2) * U * size * abs(scale)


def assert_near(got, want, off, what):
    """got rounds want, which was computed with an error of at most `off`."""
    half, least = half_step(got.dtype)
    bound = off + half * (want.abs() + off) + least
    far = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), what
    worst = (far - bound).max().item() if far.numel() else 0.0
    assert worst <= 0, f"{what}: {worst} beyond the bound (largest difference {far.max().item()})"
