"""A closer error bound for the 4-bit decode than kv4_util's, for inputs where a lost
row, group or bit has to show.

First order in the errors e_j of the scores (natural log), the softmax moves by
p_j (e_j - sum p e), so a result moves by sum_j p_j e_j |v_j - out| at most; the second
order is covered by a factor exp(2 max e).
  e_j      K 2^-23 times scale sum |q| (15 s + |z|) of row j (K terms added in fp32, s q c
           and z q apart), 2^-22 of the score (its scaling and bias), 2^-21 for exp2 and
           for the joining of warps and splits by their references
  held     p s as two fp16 numbers for the product: half a step of the second, 2^-22, or half
           of fp16's least step, 2^-25, where the largest p s of the group in a warp's rows
           is put at 2^3 or more: at most 2^-28 of that largest p s a row
  sums     n terms in fp32, truncated: (n + 64) 2^-23 of the sum of p (15 s + |z|)
  result   half a step of its type, or of its least step below the normal range
"""
from __future__ import annotations

import math

import torch

import kv4_util as U

HELD = 2.0 ** -22
LEAST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the least step


def per_group(params, n):
    """|s| and |z| of rows [0, n), one per dimension: [n, K]."""
    p = params[:n].double().abs().repeat_interleave(64, -2)
    return p[..., 0], p[..., 1]


def decode_bound(q, cache, lens, scale, alibi=False):
    """out [B, Hq, K] and lse [B, Hq] in 64 bits, and the bounds of both."""
    kc, kp, vc, vp = cache
    B, Hq, K = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, K, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    e_out, e_lse = torch.zeros_like(out), torch.zeros_like(lse)
    slope = U.slopes(Hq)
    for b, n in enumerate(lens):
        for j in range(Hkv if n else 0):
            k, v = U.values(kc[b, j, :n], kp[b, j, :n]), U.values(vc[b, j, :n], vp[b, j, :n])
            ks, kz = per_group(kp[b, j], n)
            vs, vz = per_group(vp[b, j], n)
            for h in range(j * G, j * G + G):
                qd = q[b, h].double()
                x = k @ qd * scale
                e = ((15 * ks + kz) @ qd.abs()) * (scale * K * 2.0 ** -23)
                if alibi:
                    d = slope[h] * torch.arange(n - 1, -1, -1).double()
                    x, e = x - d, e + d * 2.0 ** -22
                e = e + x.abs() * 2.0 ** -22 + 2.0 ** -21
                L = torch.logsumexp(x, 0)
                p = torch.exp(x - L)
                o = p @ v
                second = math.exp(min(2 * float(e.amax()), 600.0))
                mag = p @ (15 * vs + vz)
                held = (p @ (15 * vs)) * HELD \
                    + 15 * n * 2.0 ** -28 * (p[:, None] * torch.maximum(vs, vz * 2.0 ** -12)).amax(0)
                lse[b, h], out[b, h] = L, o
                e_lse[b, h] = (p @ e) * second + n * 2.0 ** -24 + L.abs() * 2.0 ** -23 + 2.0 ** -21
                e_out[b, h] = (((p * e) @ (v - o).abs()) * second + held
                               + (n + 64) * 2.0 ** -23 * mag
                               + o.abs() * U.HALF[q.dtype] + LEAST[q.dtype])
    return (out, lse), (e_out, e_lse)
