"""The arithmetic of masked attention's gradients with its roundings, on the CPU (test
infrastructure only): what the kernels compute from a bf16 `out` that is not exact, how far that
may be from the fp64 gradients, and what a kernel with a mistake in it would compute.

A softmax's gradient needs delta_i = d_out_i . out_i.  From an `out` that is off, delta is off
by -e_i, e_i = sum_j P_ij (dP_ij - delta_i); the kernels sum e and take it off:
    dq_i = scale (sum_j [P b (dP - delta)]_ij k_j - e_i sum_j [P b]_ij k_j)
    dk_j = scale sum_i [P b (dP - (delta + e))]_ij q_i,   dv_j = sum_i [P]_ij d_out_i
([.]: rounded to bf16, or to two bf16 with `fine`; b: the cap's derivative), so that any `out`
gives the right gradients.  Rounding bounds are counted as in block_ops.
"""
from __future__ import annotations

import math

import torch

from .block_ops import BF16, documents

MISTAKES = {  # what a kernel would leave out
    "no correction": "e is 0",
    "wrong sign": "e is added where it should be taken off",
    "half of e": "the columns 64 .. 127 of every 128 are left out of e",
    "first half of e": "the second half of the keys is left out of e",
    "a tile of the sum": "the last 128 keys are left out of sum P b K",
    "half of the sum": "the second half of the keys is left out of sum P b K",
    "low halves": "fine operands lose their second half",
}


def gradients(q, k, v, d_out, out, scale=None, softcap=0.0, slopes=None, causal=False,
              q_starts=None, kv_starts=None, fine=False, mistake=None):
    """dq, dk, dv as the kernels compute them from `out`, without the last rounding ("dq"), the
    fp64 gradients ("dq_true") and the bound on the difference of the two ("dq_tol")."""
    batch, q_len, heads, dim = q.shape
    kv_len, group = k.shape[1], heads // k.shape[2]
    scale = 1 / math.sqrt(dim) if scale is None else scale
    r = {n + x: torch.zeros(t.shape, dtype=torch.float64)
         for n, t in (("dq", q), ("dk", k), ("dv", v)) for x in ("", "_true", "_tol")}
    one = BF16 * 1.01
    two = 2.0 ** -16 * 1.05 if fine else one

    def rounded(x):
        return x.bfloat16().double()

    def operand(x):
        if not fine or mistake == "low halves":
            return rounded(x)
        return rounded(x) + rounded(x - rounded(x))

    for b in range(batch):
        for q0, nq, k0, nk in documents(q_starts, kv_starts, q_len, kv_len, b):
            if nq == 0 or nk == 0:
                continue
            i, j = torch.arange(nq)[:, None] + nk - nq, torch.arange(nk)[None]
            for h in range(heads):
                at, kat, hk = slice(q0, q0 + nq), slice(k0, k0 + nk), h // group
                qh, do, o = (t[b, at, h].double() for t in (q, d_out, out))
                kh, vh = k[b, kat, hk].double(), v[b, kat, hk].double()
                s = qh @ kh.T * scale
                s_mag = qh.abs() @ kh.abs().T * scale
                bend = torch.ones_like(s)
                if softcap:
                    t = torch.tanh(s / softcap)
                    s, bend = softcap * t, 1 - t * t
                    s_mag = s_mag.clamp(max=softcap) + softcap
                if slopes is not None:
                    far = float(slopes[h]) * (i - j).abs()
                    s, s_mag = s - far, s_mag + far.abs()
                if causal:
                    s = s.masked_fill(j > i, -math.inf)
                p = torch.softmax(s, 1).nan_to_num(0.0)
                w = torch.where(p > 0, 2 ** -21 * (s_mag + (s_mag * p).sum(1, keepdim=True)) * 1.5
                                + 2 ** -20, 0.0)  # relative error of a weight
                dp = do @ vh.T
                true = (p * dp).sum(1, keepdim=True)  # delta
                seen = (do * o).sum(1, keepdim=True)
                raw = p * (dp - seen)
                e = raw.sum(1, keepdim=True)
                pb = rounded(p * bend)
                if mistake == "no correction":
                    e = e * 0
                elif mistake == "wrong sign":
                    e = -e
                elif mistake == "half of e":
                    e = (raw * (j % 128 < 64)).sum(1, keepdim=True)
                elif mistake == "first half of e":
                    e = (raw * (j < nk // 2)).sum(1, keepdim=True)
                elif mistake == "a tile of the sum":
                    pb = pb * (j < nk - 128)
                elif mistake == "half of the sum":
                    pb = pb * (j < nk // 2)
                ds = operand(p * bend * (dp - (seen + e)))
                r["dq"][b, at, h] = (operand(raw * bend) @ kh - e * (pb @ kh)) * scale
                r["dk"][b, kat, hk] += ds.T @ qh * scale
                r["dv"][b, kat, hk] += operand(p).T @ do
                exact = p * bend * (dp - true)
                r["dq_true"][b, at, h] = exact @ kh * scale
                r["dk_true"][b, kat, hk] += exact.T @ qh * scale
                r["dv_true"][b, kat, hk] += p.T @ do
                # the bounds: with ebar = |e| of a right kernel
                ebar = raw.sum(1, keepdim=True).abs()
                # dP in fp32, and delta + e: weights, a chain of nk / 4 + 8 additions of fp32
                d_err = 2 ** -20 * (do.abs() @ vh.abs().T)
                d_err = d_err + ((p * w * (dp.abs() + seen.abs() + d_err)).sum(1, keepdim=True)
                                 + (nk / 4 + 8) * 2.0 ** -24 * raw.abs().sum(1, keepdim=True)
                                 + (p * d_err).sum(1, keepdim=True))
                # a weight's error, the bend's (2^-20), a product's sum in fp32 (2^-20)
                soft = 2 * w * bend + 2 ** -20
                q_err = ((two + 2 ** -20) * raw.abs() * bend + (one + 2 ** -20) * ebar * p * bend
                         + p * soft * ((dp - seen).abs() + ebar) + p * bend * d_err)
                k_err = ((two + 2 ** -20) * exact.abs() + p * soft * (dp - true).abs()
                         + p * bend * d_err)
                r["dq_tol"][b, at, h] = q_err @ kh.abs() * scale * 1.05
                r["dk_tol"][b, kat, hk] += k_err.T @ qh.abs() * scale * 1.05
                r["dv_tol"][b, kat, hk] += (p * (two + 2 * w + 2 ** -20)).T @ do.abs() * 1.05
    return r


def outside(got, r, name):
    """Which elements of a bf16 result cannot be the rounding of a value within the bound."""
    low, high = ((r[name + "_true"] + side * (r[name + "_tol"] + 1e-30)).float().bfloat16()
                 for side in (-1, 1))
    got = got.cpu()
    return ~((got >= low) & (got <= high))
