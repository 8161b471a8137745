"""GPU tests of the operators around a layer's products as they are used:
together in a training step, in captured graphs, on other streams and from
several threads."""
import threading

import pytest
import torch

import layer_reference as ref
from test_gpu_mx8 import DTYPES, normal

pytestmark = pytest.mark.gpu
V, T, C, O = 900, 300, 256, 512


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


def _operands(z, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    o = dict(x=normal(T, C, "bf16", seed), r=normal(T, C, "bf16", seed + 1), dy=normal(T, C, "bf16", seed + 2, 0.1),
             dz=normal(T, O, "bf16", seed + 3, 0.1), w=1 + normal(1, C, "bf16", seed + 4, 0.1)[0],
             tokens=torch.randint(-1, V, (T,), generator=g, device="cuda"), table=normal(V, C, "bf16", seed + 5, 0.02),
             lin=z.mx4_quantize(normal(O, C, "bf16", seed + 6, 0.02)))
    o["x8"] = z.mx8_quantize(o["x"])
    o["rstd"] = ref.norm(o["x"], o["w"], 1e-6)[1].float()
    return o


CALLS = {
    "mx8_quantize": lambda z, o, **kw: z.mx8_quantize(o["x"], **kw),
    "mx8_dequantize": lambda z, o, **kw: z.mx8_dequantize(o["x8"], **kw),
    "linear backward": lambda z, o, **kw: z.mx4_linear_backward(o["dz"], o["x8"], o["lin"], **kw),
    "rms_norm": lambda z, o, **kw: z.rms_norm(o["x"], o["w"], residual=o["r"], y8=True, h8=True, **kw),
    "rms_norm_backward": lambda z, o, **kw: z.rms_norm_backward(o["dy"], o["x8"], o["w"], o["rstd"], dh=o["r"], **kw),
    "embedding": lambda z, o, **kw: z.embedding(o["tokens"], o["table"], 2.0, **kw),
    "embedding_backward": lambda z, o, **kw: z.embedding_backward(o["dy"], o["tokens"], V, 2.0, **kw),
}


def _tensors(results):
    results = results if isinstance(results, tuple) else (results,)
    return [t for r in results
            for t in ((r,) if isinstance(r, torch.Tensor) else (r.codes, r.scales[:, :-(-r.cols // 32)]))]


def _clone(results):
    return [t.clone() for t in _tensors(results)]


def _same(got, want):
    return all(torch.equal(a.view(torch.uint8) if a.dtype != torch.uint8 else a, b.view(torch.uint8) if b.dtype != torch.uint8 else b)
               for a, b in zip(got, want)) and len(got) == len(want)


@pytest.mark.parametrize("name", list(CALLS))
def test_captured_and_replayed(z, name):
    """The replay works on what the operands hold by then, and two graphs of the
    same call share nothing."""
    o, other = _operands(z), _operands(z, 50)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        CALLS[name](z, o)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = CALLS[name](z, o)
        graphs.append((g, out))
    for new in (o, other):
        want = _clone(CALLS[name](z, new))
        for k, v in new.items():
            if isinstance(v, torch.Tensor):
                o[k].copy_(v)
            elif v is not o[k]:
                o[k].codes.copy_(v.codes)
                o[k].scales.copy_(v.scales)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert _same(_tensors(out), want)


@pytest.mark.parametrize("name", list(CALLS))
def test_two_streams_at_once(z, name):
    a, b = _operands(z), _operands(z, 50)
    want = [_clone(CALLS[name](z, o)) for o in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for k, o in enumerate((a, b)):
            with torch.cuda.stream(streams[k]):
                got[k].append(CALLS[name](z, o))
    torch.cuda.synchronize()
    for k in range(2):
        for r in got[k]:
            assert _same(_tensors(r), want[k])


@pytest.mark.parametrize("name", list(CALLS))
def test_another_stream_while_work_is_pending_on_the_current_one(z, name):
    """Blocks freed on the current stream are still read there by work in its
    queue; the call on another stream gets none of them, and its operands and
    results stay its own when they are freed at once."""
    o = _operands(z)
    want = _clone(CALLS[name](z, o))
    side = torch.cuda.Stream()
    sizes = sorted({t.numel() * t.element_size() for t in _tensors(CALLS[name](z, o))} | {4096, 1 << 16, 1 << 18, 1 << 20, 1 << 21})
    torch.cuda.synchronize()
    freed = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    copies = [torch.empty_like(t) for t in freed]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some 10 ms
    for c, t in zip(copies, freed):
        c.copy_(t)
    del freed, t
    out = CALLS[name](z, o, stream=side)
    kept = []
    for n in sizes:  # what is taken on the current stream now must not be the call's workspace or results
        kept.append(torch.full((n,), 9, dtype=torch.uint8, device="cuda"))
    side.synchronize()
    torch.cuda.synchronize()
    assert _same(_tensors(out), want)
    assert all((c == 7).all() for c in copies)


@pytest.mark.parametrize("name", list(CALLS))
def test_from_two_threads(z, name):
    a, b = _operands(z), _operands(z, 50)
    want = [_clone(CALLS[name](z, o)) for o in (a, b)]
    torch.cuda.synchronize()
    wrong = []

    def work(k, o):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                r = CALLS[name](z, o)
                torch.cuda.current_stream().synchronize()
                if not _same(_tensors(r), want[k]):
                    wrong.append(k)

    threads = [threading.Thread(target=work, args=(k, o)) for k, o in enumerate((a, b))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("name", list(CALLS))
def test_right_after_its_operands_are_written(z, name):
    """Every operand is written by the launch just before the call."""
    o, new = _operands(z), _operands(z, 50)
    want = _clone(CALLS[name](z, new))
    for k, v in new.items():
        if isinstance(v, torch.Tensor):
            o[k].copy_(v)
        elif v is not o[k]:
            o[k].codes.copy_(v.codes)
            o[k].scales.copy_(v.scales)
    got = CALLS[name](z, o)
    for v in o.values():  # and spoilt right after it
        if isinstance(v, torch.Tensor):
            v.zero_()
    torch.cuda.synchronize()
    assert _same(_tensors(got), want)


def test_a_training_step_with_kept_activations(z):
    """Two ranks: embedding, norm, a 4-bit linear layer; of the activations only
    8-bit checkpoints and the norm's rstd are kept; the gradients are written
    into the ranks' gradient buffers, which step_resident reduces.  Every part
    against the formulas in 64 bits, and the step against Adam's own result for
    the mean of those gradients."""
    n_ranks, vocab, tokens, cols, outs = 2, 96, 70, 64, 128
    numel = [vocab * cols, cols, outs * cols]
    opt = z.ZeroOptimizer(numel, [0, 1, 2], n_ranks, z.ZERO_STAGE_2)
    at = opt.offsets()
    master = torch.zeros(opt.psi_pad, device="cuda")
    master[at[0]:at[0] + numel[0]] = normal(vocab, cols, "f32", 1).flatten()
    master[at[1]:at[1] + numel[1]] = 1 + normal(1, cols, "f32", 2, 0.1)[0]
    master[at[2]:at[2] + numel[2]] = normal(outs, cols, "f32", 3, 0.1).flatten()
    opt.load_master(master)
    grads = []
    for rank in range(n_ranks):
        p = opt.view(z.ZERO_VIEW_PARAM, rank).view(torch.bfloat16)
        table, gain, w = (p[at[k]:at[k] + numel[k]] for k in range(3))
        table, w4 = table.view(vocab, cols), z.mx4_quantize(w.view(outs, cols))
        t = torch.randint(-1, vocab, (tokens,), generator=torch.Generator(device="cuda").manual_seed(rank), device="cuda")
        # forward: x and the residual stream r, then the layer
        x, r = z.embedding(t, table, 8.0), normal(tokens, cols, "bf16", 20 + rank)
        n = z.rms_norm(x, gain, residual=r, y8=True, h8=True)
        out = z.mx4_linear(n.y, w4)
        kept = n.y8, n.h8, n.rstd
        del x, n
        # backward
        g = torch.full((opt.psi_pad,), 0, dtype=torch.int16, device="cuda")
        g16 = g.view(torch.bfloat16)
        dtable, dgain, dw = (g16[at[k]:at[k] + numel[k]] for k in range(3))
        dout, dh = normal(tokens, outs, "bf16", 30 + rank, 0.1), normal(tokens, cols, "bf16", 40 + rank, 0.1)
        dn, _ = z.mx4_linear_backward(dout, kept[0], w4, dw=dw.view(outs, cols))
        dx, _ = z.rms_norm_backward(dn, kept[1], gain, kept[2], dh=dh, dw=dgain)
        z.embedding_backward(dx, t, vocab, 8.0, out=dtable.view(vocab, cols))
        grads.append(g)
        # the formulas, on what each part was given
        h = (z.embedding(t, table, 8.0).float() + r.float()).bfloat16()
        y, rstd = ref.norm(h, gain, 1e-6)
        assert ((kept[2].double() - rstd).abs() <= 30 * ref.U * rstd).all()
        assert torch.equal(out, z.mx4_linear(z.rms_norm(h, gain).y, w4))
        want = z.mx4_linear_backward(dout, z.mx8_dequantize(kept[0]), w4)
        assert torch.equal(dn, want[0]) and torch.equal(dw.view(outs, cols), want[1])
        want_dx, want_dgain, off_dx, off_dgain = ref.norm_backward(dn, z.mx8_dequantize(kept[1]), gain, kept[2], dh)
        ref.assert_near(dx, want_dx, off_dx, "dx")
        ref.assert_near(dgain, want_dgain, off_dgain, "dgain")
        want_table, off = ref.embedding_backward(dx, t, vocab, 8.0)
        ref.assert_near(dtable.view(vocab, cols), want_table, off, "dtable")
    opt.step_resident(grads)
    mean = (sum(g.view(torch.bfloat16).float() for g in grads) * 0.5).bfloat16()
    assert torch.equal(opt.view(z.ZERO_VIEW_GRAD_SHARD).view(torch.bfloat16)[:opt.psi_pad], mean)
    new = opt.view(z.ZERO_VIEW_MASTER)[:opt.psi_pad]
    moved = mean.float() != 0  # Adam's first step: the rate times the gradient's sign
    # (the gradient's own magnitude against eps = 1e-8, and the master's rounding)
    want = master - 1e-3 * mean.float() / (mean.float().abs() + 1e-8)
    assert ((new - want).abs() <= 1e-3 * 1e-5 + master.abs() * 2.0 ** -23)[moved].all()
    assert torch.equal(new[~moved], master[~moved])


def test_the_workspace_is_all_that_is_written(z):
    """The bytes around each call's workspace and results stay."""
    o = _operands(z)
    stream = torch.cuda.current_stream().cuda_stream
    import ctypes
    need = ctypes.c_int64()
    for cols, aligned in ((C, True), (C - 3, False)):
        dy, x = o["dy"][:, :cols].contiguous(), o["x"][:, :cols].contiguous()
        w = o["w"][:cols].contiguous()
        want_dx, want_dw = z.rms_norm_backward(dy, x, w, o["rstd"])
        assert z.zero_rms_norm_backward_workspace(T, cols, need) == 0
        space = torch.full((need.value + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        dx, dw = torch.full((T + 2, cols), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((cols + 16,), 3.0, dtype=torch.bfloat16, device="cuda")
        args = lambda at, n: (dy.data_ptr(), 0, T, cols, cols, x.data_ptr(), cols, None, w.data_ptr(), 0, o["rstd"].data_ptr(),  # noqa: E731
                              None, 0, dx[1:].data_ptr(), cols, dw[8:].data_ptr(), 0, at, n, stream)
        assert z.zero_rms_norm_backward(*args(space.data_ptr() + 256, need.value - 1)) == z.ZERO_EINVAL
        assert z.zero_rms_norm_backward(*args(space.data_ptr() + 256, need.value)) == 0
        assert torch.equal(dx[1:-1], want_dx) and torch.equal(dw[8:-8], want_dw)
        assert (dx[0] == 3).all() and (dx[-1] == 3).all() and (dw[:8] == 3).all() and (dw[-8:] == 3).all()
        assert (space[:256] == 0xA5).all() and (space[256 + need.value:] == 0xA5).all()
        dy, tokens = dy.repeat(3, 1), o["tokens"].repeat(3)  # (few tokens need none)
        want = z.embedding_backward(dy, tokens, V, 2.0)
        assert z.zero_embedding_backward_workspace(3 * T, V, cols, need) == 0 and need.value > 0
        space = torch.full((need.value + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.full((V + 2, cols), 3.0, dtype=torch.bfloat16, device="cuda")
        args = lambda at, n: (dy.data_ptr(), 0, 3 * T, cols, cols, tokens.data_ptr(), 8, V, 2.0, out[1:].data_ptr(), 0, cols, 0,  # noqa: E731
                              at, n, stream)
        assert z.zero_embedding_backward(*args(space.data_ptr() + 256, need.value - 1)) == z.ZERO_EINVAL
        assert z.zero_embedding_backward(*args(space.data_ptr() + 256, need.value)) == 0
        assert torch.equal(out[1:-1], want) and (out[0] == 3).all() and (out[-1] == 3).all()
        assert (space[:256] == 0xA5).all() and (space[256 + need.value:] == 0xA5).all()
