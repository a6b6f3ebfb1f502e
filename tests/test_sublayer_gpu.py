"""Layer norm, rotary axes and masked attention together, as one training step of a packed
attention sub-layer uses them (needs a B200).

    x -> layer norm (scale and shift per sample) -> q, k, v projection -> rotation at (t, y, x)
      -> attention within each clip -> y;   gradients back to x, the scale and shift and the
      projection

The projections are plain fp32 products on both sides.  The whole step is compared with the
same step in fp64, by the relative 2-norm of the difference: every stage rounds its bf16 result
(2^-8 / sqrt(3) of its norm at most, as independent errors), P and dS are rounded inside, and a
gradient passes through at most 8 rounded values, so sqrt(8) 2^-8 / sqrt(3) + what the
projection's rounded inputs add (two more): sqrt(10 / 3) 2^-8 = 0.71e-2 bounds it.
"""
import pytest
import torch

from joint_audio_video_flash_b200 import build, ltxattn
from oracle import block_ops

pytestmark = pytest.mark.gpu

BOUND = (10 / 3) ** 0.5 * 2 ** -8


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    ltxattn.create()


def step(x, w, b, proj, pos, dims, heads, kv_heads, dim, opts, d_out):
    """One step through the library: y and the gradients of x, w, b, proj."""
    batch, n, _ = x.shape
    freq = ltxattn.rope_frequencies(dims)
    h, mean, rstd = ltxattn.layer_norm(x, w, b, return_stats=True)
    qkv = (h.float() @ proj).bfloat16().view(batch, n, heads + 2 * kv_heads, dim)
    q, k, v = qkv.split([heads, kv_heads, kv_heads], dim=2)
    ltxattn.rope_axes(q, k, pos, freq, dims, q_out=q, k_out=k)       # in the projection's rows
    y, lse = ltxattn.masked_forward(q, k, v, **opts)
    d_qkv = torch.empty_like(qkv)
    dq, dk, dv = d_qkv.split([heads, kv_heads, kv_heads], dim=2)
    ltxattn.masked_backward(d_out, q, k, v, y, lse, dq, dk, dv, **opts)
    ltxattn.rope_axes(dq, dk, pos, freq, dims, q_out=dq, k_out=dk, inverse=True)
    flat = d_qkv.view(batch * n, -1).float()
    d_proj = h.view(batch * n, -1).float().T @ flat
    d_h = (flat @ proj.T).bfloat16().view(h.shape)
    dx, dw, db = ltxattn.layer_norm_backward(d_h, x, mean, rstd, w)
    return {"y": y, "x": dx, "w": dw, "b": db, "proj": d_proj}


def reference(x, w, b, proj, pos, dims, heads, kv_heads, dim, opts, d_out):
    """The same in fp64 on the CPU, nothing rounded."""
    batch, n, c = x.shape
    freq = ltxattn.rope_frequencies(dims)
    h, _, mean, rstd = block_ops.layer_norm(x.reshape(-1, c), w, b)
    qkv = (h @ proj.double()).view(batch, n, heads + 2 * kv_heads, dim)
    q, k, v = qkv.split([heads, kv_heads, kv_heads], dim=2)
    q, k = (block_ops.rope_axes(t, pos, freq, dims)[0] for t in (q, k))
    r = block_ops.masked(q, k, v, d_out=d_out, **opts)
    dq, dk = (block_ops.rope_axes(r[t], pos, freq, dims, inverse=True)[0] for t in ("dq", "dk"))
    flat = torch.cat([dq, dk, r["dv"]], dim=2).view(batch * n, -1)
    (dx, _), (dw, _), (db, _) = block_ops.layer_norm_backward(
        flat @ proj.double().T, x.reshape(-1, c), mean, rstd, w)
    return {"y": r["out"], "x": dx.view(x.shape), "w": dw, "b": db, "proj": h.T @ flat}


@pytest.mark.parametrize("kind", ["clips", "prefix"])
def test_one_training_step(kind):
    g = torch.Generator().manual_seed(8)
    batch, n, heads, kv_heads, dim, c = 2, 300, 4, 2, 64, 256
    dims = (24, 20, 20)
    x = torch.randn(batch, n, c, generator=g).bfloat16()
    w = (1 + 0.2 * torch.randn(batch, c, generator=g)).bfloat16()
    b = (0.2 * torch.randn(batch, c, generator=g)).bfloat16()
    proj = torch.randn(c, (heads + 2 * kv_heads) * dim, generator=g) / c ** 0.5
    pos = torch.rand(batch, n, 3, generator=g) * 50
    d_out = torch.randn(batch, n, heads, dim, generator=g).bfloat16()
    if kind == "clips":
        starts = torch.tensor([[0, 100, 100, 300], [0, 17, 180, 300]], dtype=torch.int32)
        opts = dict(q_starts=starts, kv_starts=starts)
    else:
        opts = dict(causal=True, prefix=torch.tensor([[40], [0]], dtype=torch.int32),
                    softcap=20.0, slopes=torch.tensor([0.1, 0.03, 0.01, 0.003]))
    cpu = (x, w, b, proj, pos)
    want = reference(*cpu, dims, heads, kv_heads, dim, opts, d_out)
    dev = [t.cuda() for t in cpu]
    on = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in opts.items()}
    d_out_dev = d_out.cuda()
    got = step(*dev, dims, heads, kv_heads, dim, on, d_out_dev)
    ltxattn.check()
    for name, ref in want.items():
        rel = float((got[name].cpu().double().view(ref.shape) - ref).norm() / ref.norm())
        assert rel <= BOUND, f"{name}: {rel:.2e}"
    # captured and replayed on other inputs, with an eager step in between
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(*dev, dims, heads, kv_heads, dim, on, d_out_dev)
    dev[0].copy_(torch.randn(x.shape, generator=g).bfloat16())
    eager = step(*dev, dims, heads, kv_heads, dim, on, d_out_dev)
    graph.replay()
    torch.cuda.synchronize()
    ltxattn.check()
    for name in ("y", "x", "w", "b"):
        assert torch.equal(captured[name], eager[name]), name

