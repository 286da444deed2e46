"""Attention of drafted token trees over a paged cache in 64 bits, written from the
definition, with the error its tests allow.

Tolerance of one output.  The kernel rounds each softmax weight once, to bf16
(u = 2^-8 of the weight) or, over e4m3 caches, f16 (u = 2^-11), after they were
summed: the output moves by at most u sum w |v|, and by 2^-8 |O| as it is rounded to
bf16.  A score error delta moves the weights by factors within e^(+-2 delta), the
output by 2.1 delta (sum w |v| + |O|) while delta < 0.02:
  delta = 2^-17 scale max_j |q| . |k_j|     (128 fp32 additions of the products)
        + 2^-19 max |s|                     (scale and reference in fp32: a few roundings)
        + 2^-20                             (the exponentials of a weight and of the two merges
                                             a piece goes through, 2^-22 each, and their products).
f16 numbers below 2^-14 are multiples of 2^-24: over e4m3 caches a small weight is
off by up to 2^-25 instead, relative to a sum of weights that is at least 1 in the piece
whose reference is the largest, so the output by 2^-25 sum |v| over the seen keys for each
of the two halves of a piece's keys, which have references of their own: 2^-24.  There q is the
sum of two e4m3 numbers in units in which its row's largest lies in [128, 256): the second is a
multiple of 2^-9, so a q that the first leaves finer bits of is off by up to 2^-10, that is 2^-17
of the row's largest, the score by 2^-17 scale max_i |q_i| sum_i |k_ij|; the products are twice as
many, 17/16 as large in all."""
import math

import torch

from masked_reference import gather


def attend(q, k, v, seen, scale, u):
    """q [rows, hq, d], k and v [n, hkv, d] (64 bits), seen [rows, n]: (output,
    tolerance), both [rows, hq, d]."""
    rows, hq, d = q.shape
    g = hq // k.shape[1]
    out = torch.zeros(rows, hq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    none = ~seen.any(1, keepdim=True)
    used = seen.any(0)
    for h in range(hq):
        kh = k[:, h // g].masked_fill(~used[:, None], 0.0)
        vh = v[:, h // g].masked_fill(~used[:, None], 0.0)
        qh = q[:, h].double()
        s = scale * (qh @ kh.T)
        mag = (scale * (qh.abs() @ kh.abs().T)).masked_fill(~seen, 0).amax(1, keepdim=True)
        s = s.masked_fill(~seen, -math.inf)
        w = torch.softmax(s.masked_fill(none, 0.0), 1).masked_fill(none, 0.0)
        o = w @ vh
        size = w @ vh.abs() + o.abs()
        top = s.abs().masked_fill(~seen, 0).amax(1, keepdim=True)
        delta = 2.0 ** -17 * mag + 2.0 ** -19 * top + 2.0 ** -20
        small = 0.0
        if u == 2.0 ** -11:
            k_sum = kh.abs().sum(1)[None, :].masked_fill(~seen, 0).amax(1, keepdim=True)
            delta = delta + (2.0 ** -16 * 17 / 16 - 2.0 ** -17) * mag
            delta = delta + 2.0 ** -17 * scale * qh.abs().amax(1, keepdim=True) * k_sum
            small = 2.0 ** -24 * (seen.double() @ vh.abs())
        assert float(delta.max()) < 0.02
        out[:, h] = o
        tol[:, h] = 2.0 ** -8 * o.abs() + (1.01 * u + 2.1 * delta) * size + small
    return out, tol


def reference(q, kc, vc, tables, seq_lens, q_lens, masks, scale, k_scale=1.0, v_scale=1.0):
    """The packed batch's output and tolerance; lengths on the host, masks: a Python
    integer for every row."""
    u = 2.0 ** -11 if kc.dtype == torch.uint8 else 2.0 ** -8
    outs, tols, at = [], [], 0
    for r, (n, m) in enumerate(zip(seq_lens, q_lens)):
        if m == 0:
            continue
        k, v = gather(kc, k_scale, tables[r], n), gather(vc, v_scale, tables[r], n)
        bits = torch.tensor([[mask >> i & 1 for i in range(m)] for mask in masks[at:at + m]], dtype=torch.bool)
        seen = torch.cat([torch.ones(m, n - m, dtype=torch.bool), bits], 1).to(q.device)
        o, t = attend(q[at:at + m], k, v, seen, scale, u)
        outs.append(o)
        tols.append(t)
        at += m
    return torch.cat(outs), torch.cat(tols)
