"""Cases of the gradients' corrections, for the test on the CPU that a mistake shows and for the
one of the kernels."""
import torch

# batch, q_len, kv_len, heads, kv_heads, dim, options, parts of dq's walk, documents of one tile
CASES = [
    (1, 300, 300, 4, 2, 64, {}, False, False),
    (1, 300, 2000, 2, 2, 128, {}, True, False),
    (1, 200, 4200, 2, 1, 64, dict(softcap=30.0, scale=0.5), True, False),
    (1, 1300, 700, 16, 16, 64, dict(softcap=12.0, scale=0.5, causal=True), False, False),
    (2, 257, 900, 2, 2, 128, dict(bias=True, causal=True), True, False),
    (1, 512, 512, 2, 1, 64, dict(softcap=8.0, bias=True, docs=2), False, False),
    (2, 96, 96, 4, 2, 64, dict(docs=6), False, True),
    (1, 96, 96, 2, 2, 128, dict(docs=6, softcap=10.0, bias=True, causal=True), False, True),
    (1, 100, 3000, 2, 2, 64, {}, True, True),
    (1, 2000, 126, 2, 1, 128, {}, False, True),
]


def make(case):
    """q, k, v, d_out and the call's options.  The keys and queries have a mean of their own, so
    that sums of them over many rows do not vanish."""
    batch, q_len, kv_len, heads, kv_heads, dim, o, _, _ = case
    g = torch.Generator().manual_seed(q_len + 3 * kv_len + dim)

    def draw(n, h, mean=0.0):
        return (torch.randn(batch, n, h, dim, generator=g) + mean).bfloat16()

    q, k, v, d_out = draw(q_len, heads, 0.5), draw(kv_len, kv_heads, 1.0), \
        draw(kv_len, kv_heads), draw(q_len, heads)
    opts = {n: o[n] for n in ("softcap", "scale", "causal") if n in o}
    if o.get("bias"):
        opts["slopes"] = torch.tensor([2.0 ** (-3.0 - 4.0 * h / heads) for h in range(heads)])
    if "docs" in o:
        for name, n in (("q_starts", q_len), ("kv_starts", kv_len)):
            line = [n * d // o["docs"] for d in range(o["docs"] + 1)]
            opts[name] = torch.tensor([line] * batch, dtype=torch.int32)
    return q, k, v, d_out, opts


def spoiled(out, d_out):
    """An `out` that is far off in the direction that delta feels."""
    return (out.float() + 0.25 * d_out.float()).bfloat16()
