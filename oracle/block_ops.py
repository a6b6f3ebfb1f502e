"""fp64 definitions of the operators around attention, on the CPU, with the error that the
rounding of a kernel's operands and results may cost (test infrastructure only).

Every bound counts roundings: a value rounded to type t is off by at most
``finfo(t).eps / 2`` of itself, and an operand that is rounded before a product moves the
result by that much of the sum of the product's magnitudes.
"""
from __future__ import annotations

import math

import torch

BF16 = torch.finfo(torch.bfloat16).eps / 2  # 2^-8
FP32 = torch.finfo(torch.float32).eps / 2   # 2^-24


def rope_axes(x, positions, inv_freq, axis_dims, layout="pairs", inverse=False):
    """x [B, L, H, D] turned in fp64; also the error bound for an output of x's type."""
    y = x.double().clone()
    x = x.double()
    bound = torch.zeros_like(y)
    half = x.shape[-1] // 2
    pair = 0
    for axis, channels in enumerate(axis_dims):
        for _ in range(channels // 2):
            angle = positions[..., axis].double() * inv_freq[pair] * (-1 if inverse else 1)
            c, s = torch.cos(angle)[..., None], torch.sin(angle)[..., None]
            i, j = (2 * pair, 2 * pair + 1) if layout == "pairs" else (pair, pair + half)
            y[..., i] = x[..., i] * c - x[..., j] * s
            y[..., j] = x[..., i] * s + x[..., j] * c
            # sine and cosine to 2 ulp of 1 and an angle to 2^-22 radians: 2^-21 of the pair
            bound[..., i] = bound[..., j] = 2 ** -21 * (x[..., i].abs() + x[..., j].abs())
            pair += 1
    return y, bound


def rounded(y, bound, dtype):
    """`bound` plus the rounding of a result `y` that is off by up to `bound`."""
    return bound + torch.finfo(dtype).eps / 2 * (y.abs() + bound) + 1e-30


def layer_norm(x, weight=None, bias=None, eps=1e-6):
    """x [R, C]; weight, bias [C] or [G, C].  (y, bound, mean, rstd); the statistics' fp32
    sums have chains of up to 64 additions, so values are good to 64 * 2^-24 of the row's
    typical size."""
    x = x.double()
    rows, cols = x.shape
    mean = x.mean(1)
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    z = (x - mean[:, None]) * rstd[:, None]
    mag = z.abs() + (mean.abs() * rstd)[:, None] + 1
    if weight is None:
        return z, 64 * FP32 * mag, mean, rstd
    w = weight.double().reshape(-1, cols).repeat_interleave(rows // (weight.numel() // cols), 0)
    y, mag = z * w, mag * w.abs()
    if bias is not None:
        b = bias.double().reshape(-1, cols).repeat_interleave(rows // (bias.numel() // cols), 0)
        y, mag = y + b, mag + b.abs()
    return y, 64 * FP32 * mag, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None):
    """(dx, bound), (dweight, bound), (dbias, bound) from fp32 statistics; dweight and dbias
    [G, C] (without a weight: of one group).  Sums over columns have chains of up to 64
    additions, sums over rows up to 128."""
    rows, cols = x.shape
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    z = (x - mean) * rstd
    zmag = (x.abs() + mean.abs()) * rstd  # what z is a difference of
    groups = 1 if weight is None else weight.numel() // cols
    g = dy if weight is None else \
        dy * weight.double().reshape(-1, cols).repeat_interleave(rows // groups, 0)
    dx = rstd * (g - g.mean(1, keepdim=True) - z * (g * z).mean(1, keepdim=True))
    mag = rstd * (g.abs() + g.abs().mean(1, keepdim=True)
                  + zmag * (g.abs() * zmag).mean(1, keepdim=True))
    parts = (groups, rows // groups, cols)
    dw, db = (dy * z).view(parts).sum(1), dy.view(parts).sum(1)
    dw_mag, db_mag = (dy.abs() * zmag).view(parts).sum(1), dy.abs().view(parts).sum(1)
    return ((dx, 64 * FP32 * mag), (dw, 128 * FP32 * dw_mag + 1e-30),
            (db, 128 * FP32 * db_mag + 1e-30))


def documents(q_starts, kv_starts, q_len, kv_len, b):
    """(first query, queries, first key, keys) of every document of batch row b."""
    if q_starts is None:
        return [(0, q_len, 0, kv_len)]
    qs, ks = q_starts[b].tolist(), kv_starts[b].tolist()
    return [(q0, q1 - q0, k0, k1 - k0) for q0, q1, k0, k1 in zip(qs, qs[1:], ks, ks[1:])]


def masked(q, k, v, scale=None, softcap=0.0, slopes=None, causal=False, prefix=None,
           q_starts=None, kv_starts=None, d_out=None):
    """Attention with masked, capped and biased scores of CPU tensors in fp64.

    Returns a dict of out, lse and (with d_out) dq, dk, dv, and for each name "name_err": the
    bound on a bf16 result (lse: fp32) of kernels that hold scores and statistics in fp32 and
    round P and dS to bf16 for their products.  Rows of no document have NaN in out and lse
    (they are left alone) and 0 gradients.
    """
    batch, q_len, heads, dim = q.shape
    kv_len, kv_heads = k.shape[1:3]
    scale = 1 / math.sqrt(dim) if scale is None else scale
    r = {"out": torch.full(q.shape, math.nan, dtype=torch.float64),
         "lse": torch.full((batch, heads, q_len), math.nan, dtype=torch.float64),
         "dq": torch.zeros(q.shape, dtype=torch.float64),
         "dk": torch.zeros(k.shape, dtype=torch.float64),
         "dv": torch.zeros(k.shape, dtype=torch.float64)}
    r.update({n + "_err": torch.zeros_like(t) for n, t in list(r.items())})
    # fp32 scores of magnitude S (log2 units, tensor-core sums over dim products included) are
    # off by 2^-21 S; a weight is then off by that relatively, and 2^-22 for the exponential
    for b in range(batch):
        for d, (q0, nq, k0, nk) in enumerate(documents(q_starts, kv_starts, q_len, kv_len, b)):
            n_pre = 0 if prefix is None else int(prefix[b, d])
            i = torch.arange(nq)[:, None] + nk - nq
            j = torch.arange(nk)[None]
            seen = torch.ones(nq, nk, dtype=torch.bool) if not causal else (j <= i) | (j < n_pre)
            for h in range(heads):
                at, hk = slice(q0, q0 + nq), h // (heads // kv_heads)
                kat = slice(k0, k0 + nk)
                qh, kh, vh = q[b, at, h].double(), k[b, kat, hk].double(), v[b, kat, hk].double()
                s = qh @ kh.T * scale
                s_mag = qh.abs() @ kh.abs().T * scale
                bend = torch.ones_like(s)
                if softcap:
                    t = torch.tanh(s / softcap)
                    s, bend = softcap * t, 1 - t * t
                    s_mag = s_mag.clamp(max=softcap) + softcap
                if slopes is not None:
                    far = float(slopes[h]) * (i - j).abs()
                    s, s_mag = s - far, s_mag + far.abs()  # a magnitude, whatever the sign
                s = s.masked_fill(~seen, -math.inf)
                top = s.amax(1, keepdim=True) if nk else torch.full((nq, 1), -math.inf).double()
                top = torch.where(top == -math.inf, 0.0, top)
                e = torch.exp(s - top)
                total = e.sum(1, keepdim=True)
                p = e / torch.where(total == 0, 1.0, total)
                out = p @ vh
                # relative error of a weight; a weight that is 0 has none
                w_err = 2 ** -21 * (s_mag + (s_mag * p).sum(1, keepdim=True)) * 1.5 + 2 ** -20
                w_err = torch.where(seen, w_err, 0.0)
                o_err = (p * (BF16 * 1.01 + 2 * w_err)) @ vh.abs()
                r["out"][b, at, h] = out
                o_err = o_err + BF16 * (out.abs() + o_err)
                r["out_err"][b, at, h] = o_err
                lse = (total.log() + top)[:, 0] / math.log(2)
                r["lse"][b, h, at] = lse
                fine = torch.where(torch.isfinite(lse), lse, 0.0)
                r["lse_err"][b, h, at] = (p * w_err).sum(1) * 2 + 2 ** -21 * (1 + fine.abs())
                if d_out is None:
                    continue
                do = d_out[b, at, h].double()
                r["dv"][b, kat, hk] += p.T @ do
                r["dv_err"][b, kat, hk] += (p * (BF16 * 1.01 + 2 * w_err)).T @ do.abs()
                dp = do @ vh.T
                delta = (do * out).sum(1, keepdim=True)
                ds = p * (dp - delta) * bend
                # the kernel's own bf16 out enters delta
                delta_err = (do.abs() * o_err).sum(1, keepdim=True) * 1.01
                dp_err = 2 ** -20 * (do.abs() @ vh.abs().T)
                ds_err = ds.abs() * (BF16 * 1.01 + 2 * w_err) + p * bend * (delta_err + dp_err)
                if softcap:  # bend = 1 - t^2 with t off by 2^-21
                    ds_err = ds_err + p * (dp - delta).abs() * 2 ** -20
                r["dq"][b, at, h] = ds @ kh * scale
                r["dq_err"][b, at, h] = ds_err @ kh.abs() * scale
                r["dk"][b, kat, hk] += ds.T @ qh * scale
                r["dk_err"][b, kat, hk] += ds_err.T @ qh.abs() * scale
    for n in ("dq", "dk", "dv"):
        r[n + "_err"] = r[n + "_err"] * 1.01 + BF16 * (r[n].abs() + r[n + "_err"])
    return r
