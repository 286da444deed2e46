"""Capped, biased and masked attention over a paged cache in 64 bits, written
from the definition, with the error its tests allow.

Tolerance of one output.  The kernels round each softmax weight once, to bf16
(u = 2^-8 of the weight) or, over e4m3 caches, f16 (u = 2^-11), and the output
once to bf16.  With weights p (1 + e), |e| <= u, normalised by their own sum, the
output moves by at most sum p |e| |v - O| / (sum p (1 - u)) <= 1.01 u (sum w |v| + |O|);
where the sum is taken before the rounding, by at most u sum w |v|, which is less.
A score error delta moves the weights by factors within e^(+-2 delta), the
output by 2.1 delta (sum w |v| + |O|) while delta < 0.02:
  delta = 2^-17 scale max_j |q| . |k_j|     (128 fp32 additions of the products)
        + 2^-19 max |s|                      (scale, cap and bias in fp32: a few roundings; tanh 7e-7)
        + 2^-22                              (the exponential's own error).
f16 numbers below 2^-14 are multiples of 2^-24: over e4m3 caches a small weight is
off by up to 2^-25 instead, relative to a sum of weights that is at least 1 (the
reference is the maximum of some earlier tile, which weighs 1 there), so the
output by 2^-25 sum |v| over the seen keys; a small q by 2^-25, the score by
2^-25 scale sum_i |k_ij|."""
import math

import numpy as np
import torch


def gather(cache, scale, table, n):
    """Values [n, heads, d] of tokens 0 .. n - 1, in 64 bits."""
    bs = cache.shape[1]
    t = torch.arange(n, device=cache.device)
    x = cache[table.long()[t // bs], t % bs]
    return (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).double() * scale


def attend(q, k, v, pos, scale, softcap=0.0, slopes=None, starts=None, prefix=0, u=2.0 ** -8):
    """q [rows, hq, d], k and v [n, hkv, d] (64 bits), pos and starts [rows]:
    (output, tolerance), both [rows, hq, d]."""
    rows, hq, d = q.shape
    n, hkv = k.shape[:2]
    g = hq // hkv
    j = torch.arange(n, device=q.device)
    seen = j[None, :] <= pos[:, None]
    if starts is not None:
        seen = seen & (j[None, :] >= starts[:, None])
    seen = seen | (j < prefix)[None, :]
    out = torch.zeros(rows, hq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for h in range(hq):
        kh = k[:, h // g]
        qh = q[:, h].double()
        s = scale * (qh @ kh.T)
        mag = (scale * (qh.abs() @ kh.abs().T)).masked_fill(~seen, 0).amax(1, keepdim=True)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        if slopes is not None:
            s = s - float(slopes[h]) * (pos[:, None] - j[None, :]).abs()
        s = s.masked_fill(~seen, -math.inf)
        none = ~seen.any(1, keepdim=True)
        w = torch.softmax(s.masked_fill(none, 0.0), 1).masked_fill(none, 0.0)
        vh = v[:, h // g].masked_fill(~seen.any(0)[:, None], 0.0)
        o = w @ vh
        size = w @ vh.abs() + o.abs()
        top = s.amax(1, keepdim=True).abs().masked_fill(none, 0.0)
        delta = 2.0 ** -17 * mag + 2.0 ** -19 * top + 2.0 ** -22
        small = 0.0
        if u == 2.0 ** -11:
            delta = delta + 2.0 ** -25 * scale * kh.abs().sum(1)[None, :].masked_fill(~seen, 0).amax(1, keepdim=True)
            small = 2.0 ** -25 * (seen.double() @ vh.abs())
        assert float(delta.max()) < 0.02
        out[:, h] = o
        tol[:, h] = 2.0 ** -8 * o.abs() + (1.01 * u + 2.1 * delta) * size + small
    return out, tol


def reference(q, kc, vc, tables, seq_lens, q_lens, scale, softcap=0.0, slopes=None, key_starts=None,
              prefix_lens=None, k_scale=1.0, v_scale=1.0):
    """The packed batch's output and tolerance; q [total, hq, d]; lengths on the host."""
    u = 2.0 ** -11 if kc.dtype == torch.uint8 else 2.0 ** -8
    outs, tols, at = [], [], 0
    for r, (n, m) in enumerate(zip(np.asarray(seq_lens).tolist(), np.asarray(q_lens).tolist())):
        if m == 0:
            continue
        k, v = gather(kc, k_scale, tables[r], n), gather(vc, v_scale, tables[r], n)
        pos = torch.arange(n - m, n, device=q.device)
        prefix = min(max(int(prefix_lens[r]), 0), n) if prefix_lens is not None else 0
        starts = key_starts[at:at + m].long() if key_starts is not None else None
        o, t = attend(q[at:at + m], k, v, pos, scale, softcap, slopes, starts, prefix, u)
        outs.append(o)
        tols.append(t)
        at += m
    return torch.cat(outs), torch.cat(tols)


def assert_within(got, ref, tol):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} values off, worst "
                           f"{float((err / tol.clamp_min(1e-300)).max()):.2f} of the tolerance at "
                           f"{bad.nonzero()[0].tolist()}")
