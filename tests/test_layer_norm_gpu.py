"""Layer norm and its gradients against their fp64 definitions (needs a B200).

Bounds (oracle/block_ops.py): the result's rounding and fp32 sums' chains of additions.
"""
import pytest
import torch

from joint_audio_video_flash_b200 import build, ltxattn
from oracle import block_ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    ltxattn.load()


def inputs(rows, cols, groups, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + rows + cols)
    x = (torch.randn(rows, cols, generator=g) * 2 + 0.5).to(dtype)
    dy = torch.randn(rows, cols, generator=g).to(dtype)
    shape = (cols,) if groups == 1 else (groups, cols)
    w = None if groups == 0 else (1 + 0.2 * torch.randn(shape, generator=g)).to(dtype)
    b = None if groups == 0 else (0.1 * torch.randn(shape, generator=g)).to(dtype)
    return x, dy, w, b


def cuda(*tensors):
    return [None if t is None else t.cuda() for t in tensors]


def within(got, ref, bound, what):
    err = (got.cpu().double().reshape(ref.shape) - ref).abs()
    assert torch.all(err <= bound), f"{what}: {float((err / bound).max())} of the bound"


BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
CASES = [
    # rows, cols, groups, dtype
    (1, 1, 1, FP), (1, 8, 0, BF), (3, 1, 3, BF), (5, 7, 1, HF), (2, 2048, 2, BF),
    (252, 2048, 2, BF), (77, 4096, 1, BF), (1201, 512, 1, HF), (600, 4096, 3, FP),
    (333, 1000, 3, BF), (999, 1537, 1, FP), (64, 1537, 2, BF), (100, 2500, 0, HF),
    (40, 4097, 1, FP), (30, 8192, 2, BF), (12, 12288, 1, HF), (9, 16384, 3, BF),
    (7, 40000, 1, BF), (6, 20001, 2, FP), (2000, 64, 1000, BF), (50, 100, 50, FP),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_matches_definition(case):
    rows, cols, groups, dtype = case
    x, dy, w, b = inputs(*case)
    xd, dyd, wd, bd = cuda(x, dy, w, b)
    y, mean, rstd = ltxattn.layer_norm(xd, wd, bd, return_stats=True)
    ref, bound, m64, r64 = block_ops.layer_norm(x, w, b)
    within(y, ref, block_ops.rounded(ref, bound, dtype), "y")
    scale = 1 / r64
    within(mean, m64, 64 * block_ops.FP32 * (m64.abs() + scale), "mean")
    within(rstd, r64, 64 * block_ops.FP32 * r64 * (1 + (m64 * r64) ** 2), "rstd")
    dx, dw, db = ltxattn.layer_norm_backward(dyd, xd, mean, rstd, wd)
    (rx, ex), (rw, ew), (rb, eb) = block_ops.layer_norm_backward(dy, x, mean.cpu(), rstd.cpu(), w)
    within(dx, rx, block_ops.rounded(rx, ex, dtype), "dx")
    if w is None:
        assert dw is None and db is None
    else:
        assert dw.shape == w.shape and dw.dtype == torch.float32
        within(dw, rw, ew, "dweight")
        within(db, rb, eb, "dbias")
    again = ltxattn.layer_norm_backward(dyd, xd, mean, rstd, wd)
    assert all(a is None or torch.equal(a, c) for a, c in zip((dx, dw, db), again))


def test_large_offset_keeps_its_variance():
    # mean 1000, deviation 1: a difference of moments in fp32 would lose it
    g = torch.Generator().manual_seed(3)
    x = torch.randn(20, 2048, generator=g) + 1000
    y, mean, rstd = ltxattn.layer_norm(x.cuda(), return_stats=True)
    ref, bound, _, _ = block_ops.layer_norm(x)
    within(y, ref, block_ops.rounded(ref, bound, torch.float32), "y")


@pytest.mark.parametrize("cols", [4096, 1000, 1001, 40000])
def test_strided_rows_and_in_place(cols):
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(2, 10, cols + 24, generator=g).bfloat16().cuda()
    x = wide[0, :, 8:8 + cols]
    w = torch.rand(cols, generator=g).bfloat16().cuda()
    ref = ltxattn.layer_norm(x.contiguous(), w, w)
    out = torch.full_like(wide[0], 7.0)
    ltxattn.layer_norm(x, w, w, out[:, 16:16 + cols])
    assert torch.equal(out[:, 16:16 + cols], ref)
    assert torch.all(out[:, :16] == 7) and torch.all(out[:, 16 + cols:] == 7)
    dy = wide[1, :, 8:8 + cols]
    _, mean, rstd = ltxattn.layer_norm(x, w, w, return_stats=True)
    grads = ltxattn.layer_norm_backward(dy.contiguous(), x.contiguous(), mean, rstd, w)
    for into in ("dy", "x"):  # dx in place of either
        a, c = dy.clone(), x.clone()
        got = ltxattn.layer_norm_backward(a, c, mean, rstd, w, dx=a if into == "dy" else c)
        assert all(torch.equal(p, q) for p, q in zip(got, grads))
    inplace = x.clone()
    ltxattn.layer_norm(inplace, w, w, inplace)
    assert torch.equal(inplace, ref)
    # [batch, tokens, channels] with a weight per sample
    x3 = wide[:, :, :cols].contiguous()
    w2 = torch.rand(2, cols, generator=g).bfloat16().cuda()
    y3 = ltxattn.layer_norm(x3, w2)
    for s in range(2):
        assert torch.equal(y3[s], ltxattn.layer_norm(x3[s], w2[s]))


def test_gradients_against_differences():
    g = torch.Generator().manual_seed(11)
    x, dy, direction = torch.randn(3, 6, 40, generator=g).double()
    w, b, wdir = torch.randn(3, 2, 40, generator=g).double()

    def loss(x, w, b):
        y, _, _, _ = block_ops.layer_norm(x, w, b)
        return float((y * dy).sum())

    xf, wf = x.float().cuda(), w.float().cuda()
    _, mean, rstd = ltxattn.layer_norm(xf, wf, return_stats=True)
    dx, dw, db = ltxattn.layer_norm_backward(dy.float().cuda(), xf, mean, rstd, wf)
    h = 1e-4  # differences of the definition: off by h^2, gradients by fp32's rounding
    for grad, diff, of in (
            (dx, (loss(x + h * direction, w, b) - loss(x - h * direction, w, b)) / (2 * h), direction),
            (dw, (loss(x, w + h * wdir, b) - loss(x, w - h * wdir, b)) / (2 * h), wdir),
            (db, (loss(x, w, b + h * wdir) - loss(x, w, b - h * wdir)) / (2 * h), wdir)):
        got = float((grad.cpu().double() * of).sum())
        assert abs(got - diff) <= 1e-5 * float((grad.cpu().double() * of).abs().sum()) + 1e-6


def test_other_stream_and_two_graphs():
    x, dy, w, b = cuda(*inputs(500, 1024, 1, torch.bfloat16))
    y, mean, rstd = ltxattn.layer_norm(x, w, b, return_stats=True)
    ref = ltxattn.layer_norm_backward(dy, x, mean, rstd, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ltxattn.layer_norm_backward(dy, x, mean, rstd, w, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    # two captured backward calls replayed at once, each with its own workspace
    graphs, outs, ins = [], [], []
    for s in range(2):
        d = (dy * (s + 1)).clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = ltxattn.layer_norm_backward(d, x, mean, rstd, w)
        graphs.append(graph)
        outs.append(out)
        ins.append(d)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for out, d in zip(outs, ins):
        want = ltxattn.layer_norm_backward(d, x, mean, rstd, w)
        assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_refusals():
    x = torch.zeros(6, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    stats = torch.zeros(6, device="cuda")
    with pytest.raises(TypeError):
        ltxattn.layer_norm(x.double())
    with pytest.raises(TypeError):
        ltxattn.layer_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        ltxattn.layer_norm(x, None, w)                       # a bias without a weight
    with pytest.raises(ValueError):
        ltxattn.layer_norm(x, torch.ones(4, 32, device="cuda"))  # 6 rows, 4 groups
    with pytest.raises(ValueError):
        ltxattn.layer_norm(x.t())
    with pytest.raises(ValueError):  # four rows 64 apart, the next four 224 on: not 4 * 64
        ltxattn.layer_norm(torch.zeros(4, 7, 32, device="cuda")[:, ::2])
    with pytest.raises(ValueError):
        ltxattn.layer_norm(x[:0])
    with pytest.raises(ValueError):
        ltxattn.layer_norm_backward(x, x, stats[:5], stats, w)
    for call in (lambda: ltxattn.layer_norm(x, eps=-1.0),
                 lambda: ltxattn.layer_norm(x[:5], None, None, x[1:]),      # out overlaps x
                 lambda: ltxattn.layer_norm(x, w, None, w.expand(6, 32)),   # one row for all
                 lambda: ltxattn.layer_norm_backward(x[:5], x[:5], stats[:5], stats[:5], w,
                                                     dx=x[1:])):
        with pytest.raises(ltxattn.LtxAttnError) as e:
            call()
        assert e.value.status == ltxattn.ERR_INVALID_ARG
