"""GPU tests of the embedding lookup and of its table's gradient against the
formulas in 64 bits."""
import pytest
import torch

import layer_reference as ref
import mx4_reference as ref4
from test_gpu_mx8 import DTYPES, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


def tokens_of(n, vocab, seed, kind="spread", dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "spread":
        t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    elif kind == "few":
        t = torch.randint(0, min(3, vocab), (n,), generator=g, device="cuda") * (vocab // 3)
        t = t.clamp(max=vocab - 1)
    elif kind == "one":
        t = torch.full((n,), vocab - 1, dtype=torch.int64, device="cuda")
    elif kind == "outside":
        t = torch.randint(-2, vocab + 2, (n,), generator=g, device="cuda")
    else:  # nothing but padding
        t = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    return t.to(dtype)


def want_rows(values, tokens, scale):
    here = (tokens >= 0) & (tokens < values.shape[0])
    rows = values[torch.where(here, tokens, 0).long()].double() if values.shape[0] else 0
    return torch.where(here.unsqueeze(1), rows, 0.0) * scale


SHAPES = [(1, 1, 1), (1, 1000, 768), (5, 3, 33), (300, 100, 771), (17, 50000, 64), (1003, 32001, 260), (64, 257, 4097)]


@pytest.mark.parametrize("kind", ["spread", "outside"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_lookup(z, shape, dtype, kind):
    n, vocab, cols = shape
    table = normal(vocab, cols, dtype, 1)
    for scale in (1.0, 27.7):
        for size in (torch.int32, torch.int64):
            t = tokens_of(n, vocab, 2, kind, size)
            got = z.embedding(t, table, scale)
            want = want_rows(table, t, float(torch.tensor(scale, dtype=torch.float32)))
            ref.assert_near(got, want, ref.U * want.abs() + 2.0 ** -149, "lookup")
            if scale == 1.0:
                assert torch.equal(got.double(), want)


@pytest.mark.parametrize("out", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_lookup_in_a_gathered_table(z, shape, out):
    n, vocab, cols = shape
    table = normal(vocab, cols, "f32", 1, 0.02)
    table[vocab // 2] = 0
    m = z.mx4_quantize(table)
    t = tokens_of(n, vocab, 2, "outside")
    got = z.embedding(t, m, 27.7, dtype=DTYPES[out])
    want = want_rows(ref4.read(m), t, float(torch.tensor(27.7, dtype=torch.float32)))
    ref.assert_near(got, want, ref.U * want.abs(), "lookup in MX4")
    assert z.embedding(t, m).dtype == torch.bfloat16


def test_lookup_types_strides_and_rows_that_are_not_numbers(z):
    vocab, cols, n = 50, 300, 40
    space = normal(vocab, 317, "f16", 1)
    space[7, 12] = float("nan")
    space[8, 12] = float("inf")
    t = tokens_of(n, vocab, 3)
    t[3], t[4], t[5] = 7, 8, 7
    for off in (0, 1, 8):
        table = space[:, off:off + cols]
        for dt in DTYPES.values():
            big = torch.full((n, cols + 5), 3.0, dtype=dt, device="cuda")
            got = z.embedding(t, table, 2.0, out=big[:, :cols])
            want = (table.float() * 2)[t].to(dt)
            assert torch.equal(torch.nan_to_num(got.float(), nan=9e4), torch.nan_to_num(want.float(), nan=9e4))
            assert (big[:, cols:] == 3).all()
    m = z.mx4_quantize(space[:, :cols].contiguous())
    got = z.embedding(torch.tensor([7, 9, -1], device="cuda"), m)
    assert torch.isnan(got[0, :32]).all() and torch.isfinite(got[1:]).all() and not got[2].any()


def test_tokens_far_outside_are_padding(z):
    """Also where their low bits alone would be a row's number."""
    table = normal(100, 64, "bf16", 1)
    far = [-1, -(1 << 63), (1 << 63) - 1, (1 << 32) + 3, -(1 << 32) + 3, 100, 1 << 31, 5]
    t = torch.tensor(far, device="cuda")
    got = z.embedding(t, table)
    assert not got[:-1].any() and torch.equal(got[-1], table[5])
    dy = normal(len(far), 64, "bf16", 2)
    grad = z.embedding_backward(dy, t, 100)
    assert torch.equal(grad[5], dy[-1]) and not grad[:5].any() and not grad[6:].any()
    t = torch.tensor([-(1 << 31), (1 << 31) - 1, -1, 7], dtype=torch.int32, device="cuda")
    assert not z.embedding(t, table)[:3].any()
    assert torch.equal(z.embedding_backward(dy[:4].contiguous(), t, 100)[7], dy[3])


BACK = [(1, 1, 1, "one"), (1, 1000, 768, "spread"), (5, 3, 33, "spread"), (300, 100, 771, "outside"), (700, 50, 64, "few"),
        (513, 4, 300, "one"), (100, 5003, 40, "padding"), (1003, 32001, 260, "spread"), (2049, 70000, 24, "outside"),
        (3000, 300, 520, "few"), (4097, 1 << 17, 8, "spread")]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", BACK)
def test_backward(z, shape, dtype):
    n, vocab, cols, kind = shape
    dy, t = normal(n, cols, dtype, 1, 0.1), tokens_of(n, vocab, 2, kind)
    for scale in (1.0, 27.7):
        got = z.embedding_backward(dy, t, vocab, scale)
        want, off = ref.embedding_backward(dy, t, vocab, float(torch.tensor(scale, dtype=torch.float32)))
        assert got.dtype == dy.dtype
        ref.assert_near(got, want, off, "dtable")
    assert torch.equal(z.embedding_backward(dy, t.int(), vocab, 27.7), got)


@pytest.mark.parametrize("n,vocab", [(20000, 40000), (50000, 1000), (140001, 300), (300000, 100000)])
def test_backward_of_many_tokens(z, n, vocab):
    """Whole numbers, whose sums binary32 holds exactly in any order."""
    g = torch.Generator(device="cuda").manual_seed(5)
    dy = torch.randint(-8, 9, (n, 40), generator=g, device="cuda").float()
    t = tokens_of(n, vocab, 6, "outside")
    t[n // 3: n // 2] = 5  # one token over and over
    want = torch.zeros(vocab + 4, 40, dtype=torch.float64, device="cuda").index_add_(0, t + 2, dy.double())[2:-2]
    assert torch.equal(z.embedding_backward(dy, t, vocab).double(), want)


def test_backward_gives_the_same_bits_every_time(z):
    dy, t = normal(9000, 700, "bf16", 1), tokens_of(9000, 500, 2)
    t[1000:5000] = 77
    first = z.embedding_backward(dy, t, 500, 0.37)
    for _ in range(3):
        assert torch.equal(z.embedding_backward(dy, t, 500, 0.37), first)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n", [1, 16, 17, 31, 32, 33, 500, 511, 512, 513, 800])
@pytest.mark.parametrize("vocab,cols", [(1, 8), (1, 2100), (3, 260), (40, 771), (5000, 40), (9, 50000)])
def test_backward_of_few_tokens(z, vocab, cols, n, accumulate):
    """Tokens of one, some and many positions among up to 512, and a few more.
    Whole numbers, as above."""
    g = torch.Generator(device="cuda").manual_seed(n)
    dy = torch.randint(-8, 9, (n, cols), generator=g, device="cuda").float()
    for kind in ("outside", "few", "one"):
        t = tokens_of(n, vocab, 6, kind)
        if kind == "outside" and n > 40:
            t[3:n // 2:2] = vocab - 1  # one token over and over between others
        held = torch.full((vocab, cols), 3.0, device="cuda")
        inside = (t >= 0) & (t < vocab)
        want = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, t[inside], dy[inside].double())
        got = z.embedding_backward(dy, t, vocab, 1.0, out=held, accumulate=accumulate)
        assert torch.equal(got.double(), want + 3 if accumulate else want), kind


@pytest.mark.parametrize("out", list(DTYPES))
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_backward_into_a_gradient_buffer(z, dtype, out):
    """Other types, rows apart, a view off a vector's boundary; whole or added to."""
    n, vocab, cols = 333, 90, 100
    t = tokens_of(n, vocab, 2)
    t[t == 17] = 18  # no token 17
    for off, pad in ((0, 0), (1, 3), (8, 4)):
        dy = normal(n, cols + pad, dtype, 1, 0.1)[:, :cols]
        flat = normal(1, off + vocab * (cols + pad) + 8, out, 4)[0]
        before = flat.clone()
        view = flat[off:off + vocab * (cols + pad)].view(vocab, cols + pad)[:, :cols]
        held = view.clone()
        want, bound = ref.embedding_backward(dy, t, vocab, 0.5)
        assert z.embedding_backward(dy, t, vocab, 0.5, out=view, accumulate=True) is view
        total = want + held.double()
        ref.assert_near(view, total, bound + ref.U * total.abs(), "added")
        assert torch.equal(view[17], held[17])
        z.embedding_backward(dy, t, vocab, 0.5, out=view)
        ref.assert_near(view, want, bound, "whole")
        assert not view[17].any()
        rest = torch.ones_like(flat, dtype=torch.bool)
        rest[off:off + vocab * (cols + pad)].view(vocab, cols + pad)[:, :cols] = False
        assert torch.equal(flat[rest], before[rest])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [1, 3, 5, 8, 40, 257, 771])
def test_both_are_the_same_at_every_offset(z, cols, dtype):
    """The table, dy and the results at every offset of a 16-byte word, rows end
    to end and apart: the bits of the same call on aligned rows; what is beside
    the results stays."""
    from test_gpu_rms_norm import _laid
    n, vocab, up = 150, 70, -(-cols // 8) * 8
    table, dy, t = normal(vocab, cols, dtype, 1), normal(n, cols, dtype, 2), tokens_of(n, vocab, 3, "outside")
    t[t == 11] = 12
    t[20:90] = 5
    want = z.embedding(t, _laid(table, 0, up)[0], 1.5)
    grad = z.embedding_backward(_laid(dy, 0, up)[0], t, vocab, 1.5, out=_laid(table, 0, up)[0])
    added = z.embedding_backward(_laid(dy, 0, up)[0], t, vocab, 1.5, out=_laid(table, 0, up)[0], accumulate=True)
    for off in range(8):
        for pitch in (cols, cols + 1 + off % 4):
            out, space = _laid(dy, (off + 3) % 8, pitch)
            into, other = _laid(table, off, pitch)
            assert torch.equal(z.embedding(t, _laid(table, off, pitch)[0], 1.5, out=out), want)
            z.embedding_backward(_laid(dy, (off + 5) % 8, pitch)[0], t, vocab, 1.5, out=into, accumulate=True)
            assert torch.equal(into, added), (off, pitch)
            z.embedding_backward(_laid(dy, (off + 5) % 8, pitch)[0], t, vocab, 1.5, out=into)
            assert torch.equal(into, grad), (off, pitch)
            for view, memory in ((out, space), (into, other)):
                rest = torch.ones(memory.shape[0], dtype=torch.bool, device="cuda")
                rest.as_strided(view.shape, view.stride(), storage_offset=view.storage_offset()).fill_(False)
                assert (memory[rest] == 7.0).all()


def test_backward_is_the_lookups_gradient_by_differences(z):
    """The lookup is linear in the table: with whole numbers its differences are
    the gradient, exactly."""
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randint(-9, 10, (30, 50), generator=g, device="cuda").float()
    dy = torch.randint(-9, 10, (200, 50), generator=g, device="cuda").float()
    t = tokens_of(200, 30, 3, "outside")
    grad = z.embedding_backward(dy, t, 30, 2.0)
    loss = lambda table: (z.embedding(t, table, 2.0).double() * dy.double()).sum()  # noqa: E731
    for v, c in ((0, 0), (13, 49), (29, 7)):
        moved = table.clone()
        moved[v, c] += 1
        assert float(loss(moved) - loss(table)) == float(grad[v, c])


def test_backward_of_rows_that_are_not_numbers(z):
    dy, t = normal(50, 64, "bf16", 1), torch.arange(50, device="cuda") % 10
    dy[23, 5] = float("nan")
    got = z.embedding_backward(dy, t, 20)
    assert torch.isnan(got[3, 5])
    got[3, 5] = 0
    assert torch.isfinite(got).all()


def test_empty(z):
    dy = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    table = normal(9, 64, "bf16", 1)
    assert tuple(z.embedding(none, table).shape) == (0, 64)
    out = table.clone()
    assert torch.equal(z.embedding_backward(dy, none, 9, out=out, accumulate=True), table)
    assert not z.embedding_backward(dy, none, 9, out=out).any()
    t = torch.tensor([0, -1], device="cuda")
    assert not z.embedding(t, table[:0]).any()
    assert tuple(z.embedding_backward(normal(2, 64, "bf16", 1), t, 0).shape) == (0, 64)


def test_past_32_bit_offsets(z):
    vocab, cols = 70001, 1 << 15
    table = torch.zeros(vocab, cols, dtype=torch.bfloat16, device="cuda")
    last = normal(3, cols, "bf16", 3)
    table[-3:] = last
    t = torch.tensor([vocab - 1, 0, vocab - 3, vocab - 1], device="cuda")
    got = z.embedding(t, table)
    assert torch.equal(got[[0, 2, 3]], last[[2, 0, 2]]) and not got[1].any()
    dy = normal(4, cols, "bf16", 4)
    grad = z.embedding_backward(dy, t, vocab, out=table)
    assert torch.equal(grad[0], dy[1]) and torch.equal(grad[-3], dy[2]) and not grad[1:-3].any() and not grad[-2].any()
    want = dy[0].double() + dy[3].double()
    ref.assert_near(grad[-1], want, ref.U * want.abs(), "the last row")
    del table, grad
    n = 70001
    dy = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
    dy[-3:] = last
    t = torch.arange(n, device="cuda") % 5
    grad = z.embedding_backward(dy, t, 5)
    for k in range(3):
        assert torch.equal(grad[(n - 3 + k) % 5], last[k])
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    t[-1] = 1
    assert torch.equal(z.embedding(t, last[:2].contiguous(), out=dy)[-1], last[1])


def test_wrappers_refuse_what_does_not_fit(z):
    table, t = normal(9, 64, "bf16", 1), torch.zeros(4, dtype=torch.int64, device="cuda")
    dy = normal(4, 64, "bf16", 2)
    for call in (lambda: z.embedding(t.float(), table), lambda: z.embedding(t.view(2, 2), table),
                 lambda: z.embedding(t.short(), table), lambda: z.embedding(t.cpu(), table),
                 lambda: z.embedding(torch.zeros(8, dtype=torch.int64, device="cuda")[::2], table),
                 lambda: z.embedding(t, table.double()), lambda: z.embedding(t, table.t()),
                 lambda: z.embedding(t, table, out=table[:3]), lambda: z.embedding_backward(dy, t[:3], 9),
                 lambda: z.embedding_backward(dy, t, 9, out=table[:8]), lambda: z.embedding_backward(dy, t, 9, accumulate=True),
                 lambda: z.embedding_backward(dy.double(), t, 9)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: z.embedding_backward(dy, t, -1), lambda: z.embedding(t, table, float("nan")), lambda: z.embedding_backward(dy, t, 9, float("inf")),
                 lambda: z.embedding_backward(dy[:1].expand(4, 64), t, 9)):
        with pytest.raises(z.ZeroError):
            call()
