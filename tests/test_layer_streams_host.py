"""CPU tests of the memory that the wrappers around a layer's products take and
keep when they are given a ``stream``, as test_mx4_streams_host.py has them of
the MX4 ones: a stand-in for torch notes on which stream every block is taken."""
import pytest
import torch

import zero_sharded_optimizer_sm_b200 as z
from test_mx4_streams_host import CURRENT, SIDE, Block, ExternalStream, Stream, World


class Vector(Block):
    def stride(self):
        return (1,)


class LayerWorld(World):
    def __init__(self, monkeypatch):
        super().__init__(monkeypatch)
        for name in ("float16", "float32", "int32", "int64"):
            setattr(z._T, name, getattr(torch, name))
        z._T.empty = lambda shape, dtype=None, device=None: \
            (Vector if not isinstance(shape, tuple) or len(shape) == 1 else Block)(self, shape if isinstance(shape, tuple) else (shape,), dtype)
        for name in ("zero_mx8_quantize", "zero_mx8_dequantize", "zero_mx4_linear_backward_mx8", "zero_rms_norm",
                     "zero_rms_norm_backward", "zero_embedding", "zero_embedding_backward"):
            monkeypatch.setattr(z, name, self.call)

    def vector(self, n, dtype=torch.bfloat16):
        return Vector(self, (n,), dtype)

    def mx8(self, rows, cols):
        nb = -(-cols // 32)
        return z.MX8(self.matrix(rows, 32 * nb, torch.uint8), self.matrix(rows, nb, torch.uint8), rows, cols)

    def tokens(self, n):
        return self.vector(n, torch.int64)


CALLS = {  # the call, and how many blocks it takes: results, workspace
    "quantize": (lambda w, **kw: z.mx8_quantize(w.matrix(40, 96), **kw), 1, 0),
    "dequantize": (lambda w, **kw: z.mx8_dequantize(w.mx8(40, 96), **kw), 1, 0),
    "linear backward": (lambda w, **kw: z.mx4_linear_backward(w.matrix(40, 50), w.mx8(40, 96), w.mx4(50, 96), **kw), 2, 1),
    "norm": (lambda w, **kw: z.rms_norm(w.matrix(40, 96), w.vector(96), residual=w.matrix(40, 96), y8=True, h8=True, **kw), 5, 0),
    "norm, y alone": (lambda w, **kw: z.rms_norm(w.matrix(40, 96), w.vector(96), rstd=False, **kw), 1, 0),
    "norm backward": (lambda w, **kw: z.rms_norm_backward(w.matrix(40, 96), w.mx8(40, 96), w.vector(96),
                                                          w.vector(40, torch.float32), dh=w.matrix(40, 96), **kw), 2, 1),
    "embedding": (lambda w, **kw: z.embedding(w.tokens(40), w.matrix(70, 96), **kw), 1, 0),
    "embedding of MX4": (lambda w, **kw: z.embedding(w.tokens(40), w.mx4(70, 96), **kw), 1, 0),
    "embedding backward": (lambda w, **kw: z.embedding_backward(w.matrix(40, 96), w.tokens(40), 70, **kw), 1, 1),
}


def _blocks_of(results):
    results = results if isinstance(results, tuple) else (results,)
    return [r._space if isinstance(r, z._MX) else r for r in results if r is not None]


def _run(world, name, **kw):
    call, n_results, n_spaces = CALLS[name]
    out = _blocks_of(call(world, **kw))
    new = world.blocks[-(n_results + n_spaces):]  # the operands are made first
    assert len(out) == n_results and all(any(b is o for b in new) for o in out)
    return new, out


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("given", ["object", "handle"])
def test_blocks_come_from_the_stream_that_uses_them(monkeypatch, name, given):
    world = LayerWorld(monkeypatch)
    new, results = _run(world, name, stream=Stream(SIDE) if given == "object" else SIDE)
    assert world.calls == [SIDE]
    assert [b.taken_on for b in new] == [SIDE] * len(new)
    for b in results:  # the caller's own stream will use them next
        assert CURRENT in b.recorded
    assert world.now.cuda_stream == CURRENT


@pytest.mark.parametrize("name", list(CALLS))
def test_the_current_stream_takes_its_own_blocks(monkeypatch, name):
    world = LayerWorld(monkeypatch)
    new, _ = _run(world, name, stream=CURRENT)
    assert world.calls == [CURRENT]
    assert [b.taken_on for b in new] == [CURRENT] * len(new)
    assert all(not b.recorded for b in world.blocks)


OUTS = {
    "quantize": lambda w: dict(out=w.mx8(40, 96)),
    "dequantize": lambda w: dict(out=w.matrix(40, 96)),
    "linear backward": lambda w: dict(dx=w.matrix(40, 96), dw=w.matrix(50, 96)),
    "norm, y alone": lambda w: dict(y=w.matrix(40, 96), h=w.matrix(40, 96), y8=w.mx8(40, 96), h8=w.mx8(40, 96)),
    "norm backward": lambda w: dict(dx=w.matrix(40, 96), dw=w.vector(96)),
    "embedding": lambda w: dict(out=w.matrix(40, 96)),
    "embedding backward": lambda w: dict(out=w.matrix(70, 96)),
}


@pytest.mark.parametrize("name", list(CALLS) + [f"{n}; results given" for n in OUTS])
def test_operands_may_be_freed_after_the_call(monkeypatch, name):
    """What the call was given is kept until the work on that stream has run,
    but for a stream that torch does not own."""
    name, _, given = name.partition("; results")
    for stream, kept in ((Stream(SIDE), True), (SIDE, False), (ExternalStream(SIDE), False)):
        world = LayerWorld(monkeypatch)
        kw = OUTS[name](world) if given else {}
        CALLS[name][0](world, stream=stream, **kw)
        theirs = [b for b in world.blocks if b.taken_on == CURRENT]
        assert theirs and all((SIDE in b.recorded) == kept for b in theirs)
