"""CPU tests of the MX4 wrappers' memory when they are given a ``stream``: a
stand-in for torch notes which stream is current at every allocation, stand-ins
for the library's calls which stream they were given.

A block of the caching allocator may be used at once on the stream that was
current when it was handed out, and only there: on another one nothing orders
the new use after work that is still pending in a block freed a moment ago."""
import contextlib
import ctypes
import types

import pytest
import torch

import zero_sharded_optimizer_sm_b200 as z

DEVICE = torch.device("cuda", 0)
CURRENT, SIDE = 0x1000, 0x2000  # stream handles
SIZES = {torch.bfloat16: 2, torch.float16: 2, torch.float32: 4, torch.uint8: 1}


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream


class ExternalStream(Stream):
    pass


class Block:
    """A device tensor's place: the stream that was current when it was
    handed out, and the streams it was recorded on."""

    def __init__(self, world, shape, dtype):
        self.world, self.shape, self.dtype, self.device, self.is_cuda = world, tuple(shape), dtype, DEVICE, True
        self.taken_on, self.recorded, self.at = world.now.cuda_stream, [], world.next
        world.next += 1 << 30
        world.blocks.append(self)

    def data_ptr(self):
        return self.at

    def stride(self):
        return (self.shape[1], 1)

    def new_empty(self, shape):
        return Block(self.world, shape, self.dtype)

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


class World:
    def __init__(self, monkeypatch):
        self.now, self.next, self.blocks, self.calls = Stream(CURRENT), 1 << 40, [], []

        @contextlib.contextmanager
        def stream(s):
            was, self.now = self.now, s
            try:
                yield
            finally:
                self.now = was

        cuda = types.SimpleNamespace(stream=stream, Stream=Stream, ExternalStream=ExternalStream,
                                     current_device=lambda: 0, current_stream=lambda device=None: self.now,
                                     default_stream=lambda device=None: Stream(0))
        fake = types.SimpleNamespace(
            cuda=cuda, uint8=torch.uint8, bfloat16=torch.bfloat16, device=torch.device,
            empty=lambda shape, dtype=None, device=None: Block(self, shape if isinstance(shape, tuple) else (shape,), dtype))
        codes = {torch.bfloat16: z.ZERO_DTYPE_BF16, torch.float16: z.ZERO_DTYPE_F16, torch.float32: z.ZERO_DTYPE_F32}
        monkeypatch.setattr(z, "_T", fake)
        monkeypatch.setattr(z, "_RAW_STREAM", lambda index: self.now.cuda_stream)
        monkeypatch.setattr(z, "_DTYPE_CODES", codes)
        for name in ("quantize", "transpose", "dequantize", "matmul", "linear", "linear_backward"):
            monkeypatch.setattr(z, f"zero_mx4_{name}", self.call)

    def call(self, *args):
        self.calls.append(args[-1])
        return z.ZERO_OK

    def matrix(self, rows, cols, dtype=torch.bfloat16):
        return Block(self, (rows, cols), dtype)

    def mx4(self, rows, cols, scale_pitch=None):
        nb = -(-cols // 32)
        return z.MX4(self.matrix(rows, 16 * nb, torch.uint8), self.matrix(rows, scale_pitch or nb, torch.uint8), rows, cols)


CALLS = {  # the call, and how many blocks it takes: results, workspace
    "quantize": (lambda w, **kw: z.mx4_quantize(w.matrix(40, 96), **kw), 1, 0),
    "quantize columns": (lambda w, **kw: z.mx4_quantize(w.matrix(40, 96), transpose=True, **kw), 1, 0),
    "quantize both": (lambda w, **kw: z.mx4_quantize_both(w.matrix(40, 96), **kw), 2, 0),
    "transpose": (lambda w, **kw: z.mx4_transpose(w.mx4(40, 96), **kw), 1, 0),
    "dequantize": (lambda w, **kw: z.mx4_dequantize(w.mx4(40, 96), **kw), 1, 0),
    "matmul": (lambda w, **kw: z.mx4_matmul(w.mx4(40, 96, 16), w.mx4(50, 96, 16), **kw), 1, 0),
    "matmul with a workspace": (lambda w, **kw: z.mx4_matmul(w.mx4(40, 96), w.mx4(50, 96), **kw), 1, 1),
    "linear, one token": (lambda w, **kw: z.mx4_linear(w.matrix(1, 96), w.mx4(50, 96, 16), **kw), 1, 0),
    "linear": (lambda w, **kw: z.mx4_linear(w.matrix(40, 96), w.mx4(50, 96), **kw), 1, 1),
    "backward": (lambda w, **kw: z.mx4_linear_backward(w.matrix(40, 50), w.matrix(40, 96), w.mx4(50, 96), **kw), 2, 1),
}


def _blocks_of(results):
    results = results if isinstance(results, tuple) else (results,)
    return [r._space if isinstance(r, z.MX4) else r for r in results]


def _run(world, name, **kw):
    call, n_results, n_spaces = CALLS[name]
    out = _blocks_of(call(world, **kw))
    new = world.blocks[-(n_results + n_spaces):]  # the operands are made first
    assert len(out) == n_results and all(any(b is o for b in new) for o in out)
    return new, out


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("given", ["object", "handle"])
def test_blocks_come_from_the_stream_that_uses_them(monkeypatch, name, given):
    world = World(monkeypatch)
    new, results = _run(world, name, stream=Stream(SIDE) if given == "object" else SIDE)
    assert world.calls == [SIDE]
    assert [b.taken_on for b in new] == [SIDE] * len(new)
    for b in results:  # the caller's own stream will use them next
        assert CURRENT in b.recorded
    assert world.now.cuda_stream == CURRENT


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("given", [None, CURRENT])
def test_the_current_stream_takes_its_own_blocks(monkeypatch, name, given):
    world = World(monkeypatch)
    new, _ = _run(world, name, **({} if given is None else {"stream": given}))
    assert world.calls == [CURRENT]
    assert [b.taken_on for b in new] == [CURRENT] * len(new)
    assert all(not b.recorded for b in world.blocks)


OUTS = {
    "quantize": lambda w: dict(out=w.mx4(40, 96)),
    "quantize both": lambda w: dict(out=w.mx4(40, 96), out_t=w.mx4(96, 40)),
    "transpose": lambda w: dict(out=w.mx4(96, 40)),
    "dequantize": lambda w: dict(out=w.matrix(40, 96)),
    "matmul": lambda w: dict(out=w.matrix(40, 50)),
    "linear": lambda w: dict(out=w.matrix(40, 50)),
    "backward": lambda w: dict(dx=w.matrix(40, 96), dw=w.matrix(50, 96)),
}


@pytest.mark.parametrize("name", list(CALLS) + [f"{n}, results given" for n in OUTS])
def test_operands_may_be_freed_after_the_call(monkeypatch, name):
    """What the call was given -- an operand of the caller's that is freed at
    once, a result's place -- is kept until the work on that stream has run.
    Not for a stream that torch does not own: it may be destroyed before the
    operand is freed, when torch would put an event on it."""
    name, _, given = name.partition(", results")
    for stream, kept in ((Stream(SIDE), True), (SIDE, False), (ExternalStream(SIDE), False)):
        world = World(monkeypatch)
        kw = OUTS[name](world) if given else {}
        CALLS[name][0](world, stream=stream, **kw)
        theirs = [b for b in world.blocks if b.taken_on == CURRENT]
        assert theirs and all((SIDE in b.recorded) == kept for b in theirs)


def test_an_mx4_matrix_of_the_librarys_own_memory_is_kept(monkeypatch):
    world = World(monkeypatch)
    m = z.mx4_quantize(world.matrix(40, 96))
    z.mx4_dequantize(m, stream=Stream(SIDE))
    assert SIDE in m._space.recorded


@pytest.mark.parametrize("handle", [0, 1])
def test_handles_of_the_default_stream(monkeypatch, handle):
    """0 and the legacy stream's handle 1 are torch's default stream."""
    world = World(monkeypatch)
    new, _ = _run(world, "linear", stream=handle)
    assert world.calls == [handle] and [b.taken_on for b in new] == [0, 0]


def test_workspace_sizes_are_the_librarys(monkeypatch):
    """(The stand-ins reach the library's own workspace queries.)"""
    world, n = World(monkeypatch), ctypes.c_int64()
    w = world.mx4(50, 96)
    assert z.zero_mx4_linear_workspace(40, w._c, n) == 0
    new, _ = _run(world, "linear")
    assert new[-1].shape == (n.value,)
