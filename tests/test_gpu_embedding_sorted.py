"""GPU tests of the table gradient of batches that are sorted first -- by one
cluster (513 to 65536 tokens) or by radix passes (more) -- then summed in
segments and joined: three and more launches that share a workspace, the second
of which starts before the first is over."""
import threading

import pytest
import torch

from test_gpu_embedding import tokens_of
from test_gpu_mx8 import DTYPES, normal
from test_gpu_rms_norm import _laid

pytestmark = pytest.mark.gpu
V = 900
LENGTHS = [900, 20000, 66000]


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


def whole(rows, cols, dtype, seed):
    """Whole numbers, whose sums binary32 holds exactly in any order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-8, 9, (rows, cols), generator=g, device="cuda").to(DTYPES[dtype])


def crossing(n, vocab, seed):
    """Tokens in and outside the table, one that fills several segments and more."""
    t = tokens_of(n, vocab, seed, "outside")
    t[n // 7: n // 2] = vocab // 2
    t[n - 40:] = vocab - 1
    return t


def want_of(dy, tokens, vocab, scale=1.0):
    inside = (tokens >= 0) & (tokens < vocab)
    out = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device="cuda")
    return out.index_add_(0, tokens[inside].long(), dy[inside].double()) * scale


def _operands(n, seed=1, cols=96):
    return dict(dy=normal(n, cols, "bf16", seed), t=crossing(n, V, seed), held=normal(V, cols, "bf16", seed + 9))


CALLS = {
    "whole": lambda z, o, **kw: z.embedding_backward(o["dy"], o["t"], V, 1.5, **kw),
    "added": lambda z, o, **kw: z.embedding_backward(o["dy"], o["t"], V, 1.5, out=o["held"].clone(), accumulate=True, **kw),
}
calls = pytest.mark.parametrize("name", list(CALLS))
lengths = pytest.mark.parametrize("n", LENGTHS)


@calls
@lengths
def test_captured_and_replayed(z, n, name):
    """Two graphs of one call, one after the other and both at once."""
    o, other = _operands(n), _operands(n, 50)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        CALLS[name](z, o)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = CALLS[name](z, o)
        graphs.append((g, out, torch.cuda.Stream()))
    for new in (o, other):
        want = CALLS[name](z, new).clone()
        for k in o:
            o[k].copy_(new[k])
        torch.cuda.synchronize()
        for at_once in (False, True):
            for _ in range(3):
                for g, out, stream in graphs:
                    if at_once:
                        with torch.cuda.stream(stream):
                            g.replay()
                    else:
                        g.replay()
            torch.cuda.synchronize()
            for _, out, _ in graphs:
                assert torch.equal(out, want)
                out.zero_()
            torch.cuda.synchronize()


@calls
@lengths
def test_two_streams_at_once(z, n, name):
    both = _operands(n), _operands(n, 50)
    want = [CALLS[name](z, o) for o in both]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for k, o in enumerate(both):
            with torch.cuda.stream(streams[k]):
                got[k].append(CALLS[name](z, o))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(r, want[k]) for r in got[k])


@calls
@lengths
def test_another_stream_while_work_is_pending_on_the_current_one(z, n, name):
    """Blocks freed on the current stream are still read there by work in its
    queue: the workspace of the call on another stream is none of them."""
    o = _operands(n)
    want = CALLS[name](z, o).clone()
    side = torch.cuda.Stream()
    sizes = [1 << k for k in range(12, 25)]
    torch.cuda.synchronize()
    freed = [torch.full((k,), 7, dtype=torch.uint8, device="cuda") for k in sizes]
    copies = [torch.empty_like(t) for t in freed]
    held = o["held"].clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some 10 ms
    for c, t in zip(copies, freed):
        c.copy_(t)
    del freed, t
    kw = dict(out=held, accumulate=True) if name == "added" else {}
    out = z.embedding_backward(o["dy"], o["t"], V, 1.5, stream=side, **kw)
    kept = [torch.full((k,), 9, dtype=torch.uint8, device="cuda") for k in sizes]
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all((c == 7).all() for c in copies) and all((c == 9).all() for c in kept)


@calls
@lengths
def test_from_two_threads(z, n, name):
    both = _operands(n), _operands(n, 50)
    want = [CALLS[name](z, o) for o in both]
    torch.cuda.synchronize()
    wrong = []

    def work(k, o):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                r = CALLS[name](z, o)
                torch.cuda.current_stream().synchronize()
                if not torch.equal(r, want[k]):
                    wrong.append(k)

    threads = [threading.Thread(target=work, args=(k, o)) for k, o in enumerate(both)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@calls
@lengths
def test_right_after_its_operands_are_written(z, n, name):
    """Every operand is written by the launch before the call and spoilt by the
    one after it; so is the table by the call before."""
    o, new = _operands(n), _operands(n, 50)
    want = CALLS[name](z, new)
    for _ in range(5):
        CALLS[name](z, o)
        for k in o:
            o[k].copy_(new[k])
        got = CALLS[name](z, o)
        for v in o.values():
            v.zero_()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        fresh = _operands(n)
        for k in o:
            o[k].copy_(fresh[k])


@pytest.mark.parametrize("n", [700, 66000])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [1, 5, 40, 257, 771])
def test_the_same_at_every_offset(z, cols, dtype, n):
    """dy and the table at every offset of a 16-byte word, rows end to end and
    apart: the bits of the same call on aligned rows; what is beside them stays."""
    vocab, up = 70, -(-cols // 8) * 8
    table, dy, t = normal(vocab, cols, dtype, 1), normal(n, cols, dtype, 2), crossing(n, vocab, 3)
    t[t == 11] = 12
    grad = z.embedding_backward(_laid(dy, 0, up)[0], t, vocab, 1.5, out=_laid(table, 0, up)[0])
    added = z.embedding_backward(_laid(dy, 0, up)[0], t, vocab, 1.5, out=_laid(table, 0, up)[0], accumulate=True)
    assert not grad[11].any() and torch.equal(added[11], table[11])
    for off in range(8):
        for pitch in (cols, cols + 1 + off % 4):
            into, memory = _laid(table, off, pitch)
            source = _laid(dy, (off + 5) % 8, pitch)[0]
            z.embedding_backward(source, t, vocab, 1.5, out=into, accumulate=True)
            assert torch.equal(into, added), (off, pitch)
            z.embedding_backward(source, t, vocab, 1.5, out=into)
            assert torch.equal(into, grad), (off, pitch)
            rest = torch.ones(memory.shape[0], dtype=torch.bool, device="cuda")
            rest.as_strided(into.shape, into.stride(), storage_offset=into.storage_offset()).fill_(False)
            assert (memory[rest] == 7.0).all()


@pytest.mark.parametrize("n", [1500, 66000])
@pytest.mark.parametrize("out", list(DTYPES))
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_into_a_gradient_buffer(z, dtype, out, n):
    """dy and the table of all types, rows apart, a view off a vector's boundary;
    whole or added to: one rounding of the exact sum."""
    vocab, cols = 90, 100
    t = crossing(n, vocab, 2)
    t[t == 17] = 18  # no token 17
    for off, pad in ((0, 0), (1, 3), (8, 4)):
        dy = whole(n, cols + pad, dtype, 1)[:, :cols]
        flat = whole(1, off + vocab * (cols + pad) + 8, out, 4)[0]
        before = flat.clone()
        view = flat[off:off + vocab * (cols + pad)].view(vocab, cols + pad)[:, :cols]
        held, want = view.double(), want_of(dy, t, vocab, 0.5)
        assert z.embedding_backward(dy, t, vocab, 0.5, out=view, accumulate=True) is view
        assert torch.equal(view, (want + held).to(DTYPES[out]))
        z.embedding_backward(dy, t.int(), vocab, 0.5, out=view)
        assert torch.equal(view, want.to(DTYPES[out]))
        rest = torch.ones_like(flat, dtype=torch.bool)
        rest[off:off + vocab * (cols + pad)].view(vocab, cols + pad)[:, :cols] = False
        assert torch.equal(flat[rest], before[rest])


# 17 to 28 bits of a token: two to four passes of the cluster, one to four of the radix sort
@pytest.mark.parametrize("n", [513, 1025, 2049, 9000, 65536, 65537])
@pytest.mark.parametrize("vocab,cols,dtype", [(1, 24, "f32"), (255, 24, "f32"), (256, 8, "f32"), (1 << 17, 24, "f32"), ((1 << 18) - 1, 8, "f32"),
                                              (1 << 18, 8, "bf16"), ((1 << 18) + 3, 24, "f32"), ((1 << 24) + 1, 2, "f16"),
                                              ((1 << 27) + 5, 1, "bf16")])
def test_large_vocabularies(z, vocab, cols, dtype, n):
    dy, t = whole(n, cols, dtype, n), tokens_of(n, vocab, 2, "outside")
    t[n // 3:n // 2] = vocab - 1
    t[3], t[4], t[5] = 0, vocab, vocab - 1
    t[-1] = min(1 << 17, vocab - 1)  # one bit alone
    want = want_of(dy, t, vocab)
    assert torch.equal(z.embedding_backward(dy, t, vocab).double(), want.to(DTYPES[dtype]).double())
    if cols > 1:  # added to what is there, without its first row
        table = torch.ones(vocab, cols, dtype=DTYPES[dtype], device="cuda")
        z.embedding_backward(dy, t, vocab, out=table, accumulate=True)
        assert torch.equal(table.double(), (want + 1).to(DTYPES[dtype]).double())


@lengths
def test_rows_that_are_not_numbers(z, n):
    dy, t = normal(n, 64, "bf16", 1), torch.arange(n, device="cuda") % 10
    clean = z.embedding_backward(dy, t, 20)
    dy[23, 5], dy[n - 1, 7] = float("nan"), float("inf")
    got = z.embedding_backward(dy, t, 20)
    assert torch.isnan(got[3, 5]) and torch.isinf(got[(n - 1) % 10, 7])
    got[3, 5], got[(n - 1) % 10, 7] = clean[3, 5], clean[(n - 1) % 10, 7]
    assert torch.equal(got, clean)


@lengths
def test_differences_of_the_lookup(z, n):
    """The lookup is linear in the table: with whole numbers its differences are
    the gradient, exactly."""
    table, dy, t = whole(30, 50, "f32", 1), whole(n, 50, "f32", 2), crossing(n, 30, 3)
    grad = z.embedding_backward(dy, t, 30, 2.0)
    loss = lambda table: (z.embedding(t, table, 2.0).double() * dy.double()).sum()  # noqa: E731
    for v, c in ((0, 0), (13, 49), (15, 1), (29, 7)):
        moved = table.clone()
        moved[v, c] += 1
        assert float(loss(moved) - loss(table)) == float(grad[v, c])


@pytest.mark.parametrize("kind", ["one", "padding", "few"])
@lengths
def test_one_token_or_none(z, n, kind):
    dy = whole(n, 40, "f32", 1)
    for vocab in (1, 3, 700):
        t = tokens_of(n, vocab, 2, kind)
        want = want_of(dy, t, vocab)
        assert torch.equal(z.embedding_backward(dy, t, vocab).double(), want)
        held = torch.full((vocab, 40), 3.0, device="cuda")
        z.embedding_backward(dy, t, vocab, out=held, accumulate=True)
        assert torch.equal(held.double(), want + 3)
