"""Attention with masked, capped and distance-biased scores against its fp64 definition (needs
a B200).

Bounds, element by element (oracle/block_ops.py): the output's rounding, P rounded to bf16
ahead of the PV product, and fp32 scores.
"""
import math

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
    ltxattn.create()


def starts(rows):
    """Offsets from lists of lengths, an optional leading gap as a negative first entry."""
    out = []
    for lengths in rows:
        at = -lengths[0] if lengths[0] < 0 else 0
        line = [at]
        for n in lengths[1 if lengths[0] < 0 else 0:]:
            line.append(line[-1] + n)
        out.append(line)
    return torch.tensor(out, dtype=torch.int32)


def make(batch, q_len, kv_len, heads, kv_heads, dim, seed=0):
    g = torch.Generator().manual_seed(seed + q_len + 7 * kv_len)

    def draw(n, h):
        return torch.randn(batch, n, h, dim, generator=g).bfloat16()

    return draw(q_len, heads), draw(kv_len, kv_heads), draw(kv_len, kv_heads), draw(q_len, heads)


def options(heads, cap=0.0, bias=False, scale=None, **kw):
    slopes = torch.tensor([2.0 ** (-6.0 * (i + 1) / heads) for i in range(heads)]) if bias else None
    return dict(softcap=cap, slopes=slopes, scale=scale, **kw)


def cuda(opts):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in opts.items()}


def compare(got, ref, names):
    for n in names:
        want, err = ref[n], ref[n + "_err"]
        live = ~torch.isnan(want)
        g = got[n].cpu().double()
        same = g == want  # infinities
        assert torch.all((((g - want).abs() <= err + 1e-30) | same)[live]), \
            f"{n}: {float(((g - want).abs() / (err + 1e-30))[live & ~same].max())} of the bound"


def run(q, k, v, opts):
    """Forward into marked buffers; rows of no document must keep the marks."""
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), 5.0, device="cuda")
    ltxattn.masked_forward(q.cuda(), k.cuda(), v.cuda(), out, lse, **cuda(opts))
    ltxattn.check()
    return {"out": out, "lse": lse}


FORWARD = [
    # batch, q_len, kv_len, heads, kv_heads, dim, options
    (1, 1, 1, 1, 1, 64, {}),
    (2, 1, 1000, 4, 4, 128, {}),                                   # one query, key parts
    (2, 1, 1000, 8, 2, 64, dict(causal=True)),
    (1, 3, 700, 32, 1, 128, dict(causal=True, cap=5.0)),           # 96 packed rows
    (1, 130, 130, 2, 2, 64, {}),
    (2, 257, 300, 6, 2, 128, dict(bias=True)),                     # group of 3: not packed
    (1, 300, 257, 4, 2, 64, dict(causal=True)),                    # early queries see nothing
    (1, 640, 640, 2, 1, 128, dict(causal=True, cap=8.0, bias=True)),
    (2, 126, 2000, 2, 2, 64, {}),                                  # one tile, key parts
    (1, 126, 2000, 2, 2, 128, dict(bias=True, cap=3.0, causal=True)),
    (1, 33, 129, 3, 3, 128, dict(causal=True, prefix=[[40]])),
    (2, 500, 500, 4, 1, 64, dict(causal=True, prefix=[[0], [450]])),
    (1, 200, 200, 2, 2, 64, dict(causal=True, prefix=[[100000]])),  # beyond the keys: all
    (2, 300, 300, 4, 4, 64, dict(q=[[100, 0, 1, 190], [-5, 128, 129, 0, 20]][:1] * 2)),
    (2, 300, 310, 4, 2, 128, dict(q=[[-3, 50, 0, 200], [256, 1, 40]],
                                  kv=[[-1, 60, 30, 129], [0, 130, 180]])),
    (1, 290, 300, 8, 4, 64, dict(q=[[129, 1, 160]], kv=[[40, 0, 260]], causal=True, bias=True)),
    (1, 600, 600, 2, 2, 128, dict(q=[[5, 90, 17, 128, 200, 100]], causal=True, cap=4.0,
                                  prefix=[[2, 95, 0, 60, 30, 1]])),
    (1, 40, 40, 1, 1, 64, dict(q=[[1] * 40])),                     # forty documents of one
    (1, 6, 4000, 4, 4, 128, dict(q=[[1, 2, 3]], kv=[[1000, 2500, 500]], causal=True)),
]


@pytest.mark.parametrize("case", FORWARD, ids=lambda c: "-".join(str(x) for x in c))
def test_forward_matches_definition(case):
    batch, q_len, kv_len, heads, kv_heads, dim, o = case
    o = dict(o)
    qs = o.pop("q", None)
    if qs is not None:
        o["q_starts"], o["kv_starts"] = starts(qs), starts(o.pop("kv", qs))
    if "prefix" in o:
        o["prefix"] = torch.tensor(o["prefix"], dtype=torch.int32)
    opts = options(heads, **o)
    q, k, v, _ = make(batch, q_len, kv_len, heads, kv_heads, dim)
    ref = block_ops.masked(q, k, v, **opts)
    got = run(q, k, v, opts)
    compare(got, ref, ("out", "lse"))
    outside = torch.isnan(ref["out"])
    assert torch.all(got["out"].cpu()[outside] == 7)
    assert torch.all(got["lse"].cpu()[torch.isnan(ref["lse"])] == 5)


BACKWARD = [
    # batch, q_len, kv_len, heads, kv_heads, dim, options
    (1, 1, 1, 1, 1, 64, {}),
    (2, 5, 7, 2, 1, 128, dict(causal=True)),
    (1, 130, 130, 2, 2, 64, {}),
    (2, 257, 300, 6, 2, 128, dict(bias=True)),
    (1, 300, 257, 4, 2, 64, dict(causal=True)),                     # queries that see nothing
    (1, 257, 600, 2, 2, 128, dict(causal=True, cap=6.0)),
    (1, 640, 640, 2, 1, 128, dict(causal=True, cap=8.0, bias=True)),
    (1, 126, 2000, 2, 2, 64, dict(cap=4.0)),                        # dq in key parts
    (1, 2000, 126, 2, 1, 128, {}),                                  # dk, dv in query parts
    (2, 500, 500, 4, 1, 64, dict(causal=True, prefix=[[0], [450]])),
    (1, 33, 129, 3, 3, 128, dict(causal=True, prefix=[[40]], bias=True)),
    (2, 300, 310, 4, 2, 128, dict(q=[[-3, 50, 0, 200], [256, 1, 40]],
                                  kv=[[-1, 60, 30, 129], [0, 130, 180]])),
    (1, 290, 300, 8, 4, 64, dict(q=[[129, 1, 160]], kv=[[40, 0, 260]], causal=True, bias=True)),
    (1, 600, 600, 2, 2, 128, dict(q=[[5, 90, 17, 128, 200, 100]], causal=True, cap=4.0,
                                  prefix=[[2, 95, 0, 60, 30, 1]])),
    (1, 700, 2100, 2, 2, 64, dict(q=[[300, 400]], kv=[[1000, 1100]], causal=True)),
]


def run_backward(q, k, v, d_out, opts):
    """Forward and backward into marked buffers."""
    opts = cuda(opts)
    q, k, v, d_out = (t.cuda() for t in (q, k, v, d_out))
    out, lse = ltxattn.masked_forward(q, k, v, **opts)
    marked = [torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda") for t in (q, k, v)]
    ltxattn.masked_backward(d_out, q, k, v, out, lse, *marked, **opts)
    ltxattn.check()
    return dict(zip(("dq", "dk", "dv"), marked))


def covered(off, b, length):
    at = torch.zeros(length, dtype=torch.bool)
    at[0 if off is None else int(off[b, 0]):length if off is None else int(off[b, -1])] = True
    return at


@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: "-".join(str(x) for x in c))
def test_backward_matches_definition(case):
    batch, q_len, kv_len, heads, kv_heads, dim, o = case
    o = dict(o)
    qs = o.pop("q", None)
    if qs is not None:
        o["q_starts"], o["kv_starts"] = starts(qs), starts(o.pop("kv", qs))
    if "prefix" in o:
        o["prefix"] = torch.tensor(o["prefix"], dtype=torch.int32)
    opts = options(heads, **o)
    q, k, v, d_out = make(batch, q_len, kv_len, heads, kv_heads, dim)
    ref = block_ops.masked(q, k, v, d_out=d_out, **opts)
    got = run_backward(q, k, v, d_out, opts)
    for b in range(batch):
        for n, off, length in (("dq", opts.get("q_starts"), q_len),
                               ("dk", opts.get("kv_starts"), kv_len),
                               ("dv", opts.get("kv_starts"), kv_len)):
            inside = covered(off, b, length)
            assert torch.all(got[n][b].cpu()[~inside] == 7), n
            compare({n: got[n][b].cpu()[inside]},
                    {n: ref[n][b][inside], n + "_err": ref[n + "_err"][b][inside]}, (n,))
            # and as a whole: P, dS and the result are rounded, three independent errors of
            # 2^-8 / sqrt(3) rms at most; delta's own error adds as much again
            diff = got[n][b].cpu().double()[inside] - ref[n][b][inside]
            norm = float(ref[n][b][inside].norm())
            assert float(diff.norm()) <= 2 ** -7 * norm + 1e-6, n
    again = run_backward(q, k, v, d_out, opts)
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("dim", [64, 128])
def test_gradients_against_differences(dim):
    # a directional difference of the definition's loss: the gradients are within their bf16
    # rounding of it
    q, k, v, d_out = make(1, 40, 50, 2, 1, dim, seed=9)
    opts = options(2, cap=3.0, bias=True, causal=True)
    got = run_backward(q, k, v, d_out, opts)
    g = torch.Generator().manual_seed(1)

    def loss(*qkv):
        return float((block_ops.masked(*qkv, **opts)["out"] * d_out.double()).sum())

    for at, n in enumerate(("dq", "dk", "dv")):
        x = [q.double(), k.double(), v.double()]
        direction = torch.randn(x[at].shape, generator=g).double()
        h = 1e-4
        up, down = list(x), list(x)
        up[at], down[at] = x[at] + h * direction, x[at] - h * direction
        diff = (loss(*up) - loss(*down)) / (2 * h)
        terms = got[n].cpu().double() * direction
        # every element off by 2^-6 of itself at most on average (rounded three times)
        assert abs(float(terms.sum()) - diff) <= 2 ** -6 * float(terms.abs().sum())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_masked_rows_do_not_reach_a_gradient(bad):
    q, k, v, d_out = make(1, 170, 333, 2, 1, 64)
    opts = dict(q_starts=torch.tensor([[7, 90, 161]], dtype=torch.int32),
                kv_starts=torch.tensor([[3, 104, 305]], dtype=torch.int32))
    ref = block_ops.masked(q, k, v, d_out=d_out, **opts)
    for t in (q, d_out):
        t[:, :7], t[:, 161:] = bad, bad
    for t in (k, v):
        t[:, :3], t[:, 305:] = bad, bad
    got = run_backward(q, k, v, d_out, opts)
    for n, a, z in (("dq", 7, 161), ("dk", 3, 305), ("dv", 3, 305)):
        compare({n: got[n][:, a:z]}, {n: ref[n][:, a:z], n + "_err": ref[n + "_err"][:, a:z]}, (n,))


def test_backward_views_and_graph():
    g = torch.Generator().manual_seed(14)
    qkv = torch.randn(2, 150, 8 + 2 * 2, 64, generator=g).bfloat16().cuda()
    views = qkv[:, :, :8], qkv[:, :, 8:10], qkv[:, :, 10:]
    out, lse = ltxattn.masked_forward(*views, causal=True)
    d_out = torch.randn(2, 150, 8, 64, generator=g).bfloat16().cuda()
    ref = ltxattn.masked_backward(d_out, *(t.contiguous() for t in views), out, lse, causal=True)
    # the gradients as parts of the projection's gradient
    dqkv = torch.zeros_like(qkv)
    into = dqkv[:, :, :8], dqkv[:, :, 8:10], dqkv[:, :, 10:]
    ltxattn.masked_backward(d_out, *views, out, lse, *into, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(into, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, l2 = ltxattn.masked_forward(*views, causal=True)
        grads = ltxattn.masked_backward(d_out, *views, o2, l2, causal=True)
    graph.replay()
    torch.cuda.synchronize()
    ltxattn.check()
    assert all(torch.equal(a, b) for a, b in zip(grads, ref))


@pytest.mark.parametrize("dim,q_len", [(64, 1), (64, 200), (128, 90), (128, 300)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_masked_does_not_reach_a_result(dim, q_len, bad):
    # every row outside the documents, in q, k and v, is not finite
    q, k, v, _ = make(1, q_len + 20, 333, 2, 2, dim)
    opts = dict(q_starts=torch.tensor([[7, 7 + q_len // 2, 7 + q_len]], dtype=torch.int32),
                kv_starts=torch.tensor([[3, 104, 305]], dtype=torch.int32))
    ref = block_ops.masked(q, k, v, **opts)
    q[:, :7], q[:, 7 + q_len:] = bad, bad
    k[:, :3], k[:, 305:], v[:, :3], v[:, 305:] = bad, bad, bad, bad
    got = run(q, k, v, opts)
    compare(got, ref, ("out", "lse"))
    # and one document's rows do not reach the other's
    k[:, 104:305], v[:, 104:305] = bad, bad
    got = run(q, k, v, opts)
    first = slice(7, 7 + q_len // 2)
    for n, at in (("out", (slice(None), first)), ("lse", (slice(None), slice(None), first))):
        want, err = ref[n][at], ref[n + "_err"][at]
        assert torch.all((got[n].cpu().double()[at] - want).abs() <= err + 1e-30)


def test_scores_of_every_size():
    # weights that underflow, one key that takes all, scores far beyond the cap
    q, k, v, _ = make(1, 140, 400, 2, 1, 64)
    for scale, cap in ((30.0, 0.0), (1e-6, 0.0), (30.0, 2.0), (1e4, 50.0), (1e-5, 50.0)):
        opts = options(2, cap=cap, scale=scale, causal=True)
        compare(run(q, k, v, opts), block_ops.masked(q, k, v, **opts), ("out", "lse"))
    # growing scores: the running maximum moves in every key tile
    k = (k.float() * torch.linspace(0.1, 12, 400)[None, :, None, None]).bfloat16()
    opts = options(2, scale=1.0)
    compare(run(q, k, v, opts), block_ops.masked(q, k, v, **opts), ("out", "lse"))


@pytest.mark.parametrize("cap", [0.0, 6.0, 62.0, 63.0, 500.0])
def test_every_cap_and_slopes_of_both_signs(cap):
    # caps on either side of the form without a maximum; slopes that favour far keys; a query
    # stretch that lies wholly ahead of or behind its keys
    for q_len, kv_len, causal in ((200, 170, False), (90, 400, True), (400, 90, False)):
        q, k, v, d_out = make(1, q_len, kv_len, 4, 2, 64, seed=3)
        for slopes in ([0.5, 0.01, -0.02, -0.4], [3.0, 0.0, -3.0, 1e-4]):
            opts = dict(softcap=cap, slopes=torch.tensor(slopes), causal=causal, scale=0.6)
            ref = block_ops.masked(q, k, v, d_out=d_out, **opts)
            compare(run(q, k, v, opts), ref, ("out", "lse"))
            compare(run_backward(q, k, v, d_out, opts), ref, ("dq", "dk", "dv"))


@pytest.mark.parametrize("kv_len", [200, 5000])
def test_caps_far_from_the_scores(kv_len):
    """A huge cap changes nothing, a tiny one leaves the mean of v."""
    q, k, v, d_out = make(1, 40, kv_len, 2, 2, 128)
    q[:, 7:39] = 0
    plain = run(q, k, v, options(2))["lse"]
    # cap tanh(s / cap) is s (1 - s^2 / 3 cap^2); |s| < 9 in base 2 with a relative error of the
    # polynomial (3e-7), its eight roundings and those of the plain product (2^-24 each)
    huge = run(q, k, v, options(2, cap=1e6))["lse"]
    assert float((huge - plain).abs().max()) <= 9 * (3e-7 + 12 * 2.0 ** -24)
    opts = options(2, cap=1e-5)
    tiny = run(q, k, v, opts)
    # weights within e^(2 cap) of 1 / kv_len
    assert float((tiny["lse"].cpu() - math.log2(kv_len)).abs().max()) <= 2e-5
    mean = v.double().mean(1, keepdim=True)
    far = (tiny["out"].cpu().double() - mean).abs()
    # the result's rounding, P rounded to bf16 against a sum of it unrounded, 2 cap
    lim = 2.0 ** -8 * mean.abs() + 2.0 ** -8 * v.double().abs().mean(1, keepdim=True)
    assert torch.all(far <= lim + 2e-5 * 5)
    assert all(torch.isfinite(t).all() for t in run_backward(q, k, v, d_out, opts).values())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [3, 5, 7, 24, 96, 130])
def test_groups_of_every_size(group, dim):
    """Groups of query heads that fill a power of two of rows or do not, with heads of another
    group (or none) behind them."""
    for q_len, kv_len, kv_heads, o in ((1, 700, 2, dict(causal=True, bias=True)), (9, 300, 1, {}),
                                       (70, 90, 2, dict(causal=True, cap=5.0))):
        if group > 24 and q_len > 9:
            continue
        q, k, v, _ = make(2, q_len, kv_len, kv_heads * group, kv_heads, dim)
        opts = options(kv_heads * group, **o)
        compare(run(q, k, v, opts), block_ops.masked(q, k, v, **opts), ("out", "lse"))
    # packed documents, some without a query; rows of no document keep their marks
    q, k, v, _ = make(1, 60, 400, 2 * group, 2, dim)
    opts = options(2 * group, q_starts=starts([[-3, 1, 0, 30, 9, 10]]),
                   kv_starts=starts([[-8, 100, 50, 1, 200, 20]]))
    ref = block_ops.masked(q, k, v, **opts)
    got = run(q, k, v, opts)
    compare(got, ref, ("out", "lse"))
    assert torch.all(got["out"].cpu()[torch.isnan(ref["out"])] == 7)
    assert torch.all(got["lse"].cpu()[torch.isnan(ref["lse"])] == 5)


LONG = [
    # rows of more keys than the form without a running maximum starts at, in both plans
    (1, 150, 4200, 2, 2, 64, dict(causal=True, cap=30.0)),
    (1, 2500, 2500, 4, 2, 128, dict(causal=True, cap=20.0, prefix=[[700]])),
    (1, 300, 2300, 2, 1, 128, dict(cap=10.0, bias=True)),
    (1, 2200, 2300, 2, 2, 64, dict(causal=True, cap=50.0, bias=True)),
    (1, 700, 9000, 3, 3, 64, dict(cap=3.0, causal=True, q=[[200, 499]], kv=[[4000, 4990]])),
    (2, 1, 9000, 8, 2, 128, dict(cap=5.0, bias=True)),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(str(x) for x in c))
def test_long_capped_rows(case):
    test_forward_matches_definition(case)
    test_backward_matches_definition(case)


@pytest.mark.parametrize("cap", [10.0, 62.0])
def test_long_capped_rows_with_slopes_of_both_signs(cap):
    for q_len, kv_len, causal in ((200, 2170, False), (2400, 2400, True)):
        q, k, v, _ = make(1, q_len, kv_len, 4, 2, 64, seed=3)
        opts = dict(softcap=cap, slopes=torch.tensor([0.5, 0.01, -0.02, -0.4]), causal=causal,
                    scale=0.6)
        compare(run(q, k, v, opts), block_ops.masked(q, k, v, **opts), ("out", "lse"))


@pytest.mark.parametrize("cap", [0.0, 10.0, 500.0])
@pytest.mark.parametrize("dim", [64, 128])
def test_one_visible_key_has_all_the_weight(dim, cap):
    """A softmax over one key is exactly 1: out is v itself, and no score has a gradient."""
    q, k, v, d_out = make(2, 70, 70, 4, 2, dim)
    off = starts([[1] * 70])
    opts = options(4, cap=cap, q_starts=off.expand(2, -1).contiguous(),
                   kv_starts=off.expand(2, -1).contiguous())
    got = run(q, k, v, opts)
    assert torch.equal(got["out"].cpu(), v.repeat_interleave(2, dim=2))
    grads = run_backward(q, k, v, d_out, opts)
    # dP - delta is the same fp32 sum in two orders: dim terms of |dO v|, each order off by at
    # most dim 2^-24 of their sum of magnitudes; the products with K or Q then scale it
    dp = (d_out.double() * v.repeat_interleave(2, dim=2).double()).abs().sum(-1)
    lim = 2 * dim * 2.0 ** -24 * float(dp.max()) * dim ** -0.5
    assert float(grads["dq"].abs().max()) <= lim * float(k.abs().max()) * 1.01
    assert float(grads["dk"].abs().max()) <= lim * 2 * float(q.abs().max()) * 1.01


def test_strided_views_and_layouts():
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn(2, 150, 8 + 2 * 2, 64, generator=g).bfloat16()
    q, k, v = qkv[:, :, :8], qkv[:, :, 8:10], qkv[:, :, 10:]
    opts = options(8, causal=True)
    ref = block_ops.masked(q, k, v, **opts)
    dev = qkv.cuda()
    views = dev[:, :, :8], dev[:, :, 8:10], dev[:, :, 10:]
    out, lse = ltxattn.masked_forward(*views, causal=True)
    compare({"out": out, "lse": lse}, ref, ("out", "lse"))
    head_major = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in views]
    o2 = torch.empty(2, 8, 150, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    ltxattn.masked_forward(*head_major, o2, causal=True)
    assert torch.equal(o2, out)
    # the output as a part of the same rows
    wide = torch.cat([dev, torch.zeros(2, 150, 8, 64, dtype=torch.bfloat16, device="cuda")], 2)
    ltxattn.masked_forward(wide[:, :, :8], wide[:, :, 8:10], wide[:, :, 10:12], wide[:, :, 12:],
                           causal=True)
    assert torch.equal(wide[:, :, 12:], out) and torch.equal(wide[:, :, :12], dev)
    ltxattn.check()


def test_offsets_that_break_the_rules_stay_inside():
    # the kernel holds every offset inside the tensor; only that is checked here
    q, k, v, _ = make(1, 100, 100, 2, 2, 64)
    for line in ([-50, 30, 400], [90, 10, 95], [2 ** 31 - 1, -2 ** 31, 5]):
        s = torch.tensor([line], dtype=torch.int32)
        run(q, k, v, dict(q_starts=s, kv_starts=s))


def test_streams_and_two_graphs():
    q, k, v, _ = (t.cuda() for t in make(2, 4, 3000, 4, 4, 64))
    ref, ref_lse = ltxattn.masked_forward(q, k, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = ltxattn.masked_forward(q, k, v, stream=side)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    graphs, outs = [], []
    queries = [q, (q.float() * 2).bfloat16()]
    for x in queries:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(ltxattn.masked_forward(x, k, v))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    ltxattn.check()
    for x, (o, l) in zip(queries, outs):
        want, want_lse = ltxattn.masked_forward(x, k, v)
        assert torch.equal(o, want) and torch.equal(l, want_lse)


def test_refusals():
    q, k, v, _ = (t.cuda() for t in make(2, 8, 8, 4, 2, 64))
    s = torch.tensor([[0, 4, 8]] * 2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        ltxattn.masked_forward(q.float(), k, v)
    with pytest.raises(TypeError):
        ltxattn.masked_forward(q, k, v, q_starts=s.long(), kv_starts=s.long())
    with pytest.raises(ValueError):
        ltxattn.masked_forward(q, k, v[:, :4])
    with pytest.raises(ValueError):
        ltxattn.masked_forward(q, k, v, q_starts=s)
    with pytest.raises(ValueError):
        ltxattn.masked_forward(q, k, v, prefix=torch.zeros(2, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ltxattn.masked_forward(q, k, v, slopes=torch.zeros(2, device="cuda"))
    for status, call in (
            (ltxattn.ERR_INVALID_ARG, lambda: ltxattn.masked_forward(q[:, :, :3], k, v)),
            (ltxattn.ERR_INVALID_ARG, lambda: ltxattn.masked_forward(q, k, v, q)),
            (ltxattn.ERR_INVALID_ARG, lambda: ltxattn.masked_forward(q, k, v, softcap=-1.0)),
            (ltxattn.ERR_INVALID_ARG, lambda: ltxattn.masked_forward(q, k, v, scale=math.nan)),
            (ltxattn.ERR_INVALID_ARG,
             lambda: ltxattn.masked_forward(q, k[:1].expand(2, 8, 2, 64), v)),
            (ltxattn.ERR_UNSUPPORTED,
             lambda: ltxattn.masked_forward(*(t[..., :32].contiguous() for t in (q, k, v)))),
            (ltxattn.ERR_MISALIGNED, lambda: ltxattn.masked_forward(
                torch.zeros(2, 8, 4, 68, dtype=torch.bfloat16, device="cuda")[..., :64], k, v))):
        with pytest.raises(ltxattn.LtxAttnError) as e:
            call()
        assert e.value.status == status
    out, lse = ltxattn.masked_forward(q, k, v)
    with pytest.raises(ValueError):
        ltxattn.masked_backward(out, q, k, v, out, None)
    with pytest.raises(ValueError):
        ltxattn.masked_backward(out[:, :4], q, k, v, out, lse)
    for bad in (dict(dq=q), dict(dk=torch.empty_like(k), dv=k), dict(dq=out)):
        with pytest.raises(ltxattn.LtxAttnError) as e:
            ltxattn.masked_backward(out.clone(), q, k, v, out, lse, **bad)
        assert e.value.status == ltxattn.ERR_INVALID_ARG
