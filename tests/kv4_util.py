"""Plain 64-bit forms of the cache operators (4-bit cache, key weights, eviction),
one (sequence, head) at a time, and the error bounds their tests use.

Bounds (u32 = 2^-24 a rounding of fp32, 2^-23 a truncating tensor-core addition;
h16 = half a step of the 16-bit type, 2^-8 bf16 or 2^-11 fp16, relative):
  score  a dot product of K terms summed in fp32 is off by at most K 2^-23 times
         the sum of its terms' magnitudes.  The 4-bit decode sums s q c and z q apart:
         magnitudes |q| (15 s + |z|).
  weight exp of a score off by e is off by a factor e^e; exp2 itself by 2^-22.  The
         4-bit decode multiplies p s held as one fp16 number (half a step 2^-11) for
         bf16 results and as two (2^-21) for fp16 results.
  sum    n terms added in fp32: n 2^-24 of the sum of magnitudes.
"""
from __future__ import annotations

import math

import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
HELD = {torch.float16: 2.0 ** -21, torch.bfloat16: 2.0 ** -11}  # of p s


def quantise(x):
    """x 16-bit [..., K] -> codes 0..15 int64 [..., K/64, 64], s, z of x.dtype."""
    xg = x.double().unflatten(-1, (x.shape[-1] // 64, 64))
    bad = ~torch.isfinite(xg).all(-1)
    safe = torch.where(bad[..., None], torch.zeros_like(xg), xg)
    mn, mx = safe.amin(-1), safe.amax(-1)
    s = ((mx - mn) / 15).float().to(x.dtype)
    z = mn.to(x.dtype)
    sd, zd = s.double()[..., None], z.double()[..., None]
    c = torch.where(sd > 0, (safe - zd) / torch.where(sd > 0, sd, torch.ones_like(sd)),
                    torch.zeros_like(safe)).round().clamp(0, 15)
    c = torch.where(bad[..., None], torch.zeros_like(c), c).long()
    s, z = s.clone(), z.clone()
    s[bad] = math.nan
    z[bad] = math.nan
    return c, s, z


def pack(c):
    c = c.flatten(-2).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def planes(x):
    """Rows x [B, n, H, K] as (codes [B, H, n, K/2], params [B, H, n, K/64, 2])."""
    c, s, z = quantise(x.transpose(1, 2).contiguous())
    return pack(c), torch.stack((s, z), -1)


def values(codes, params):
    """[..., K/2] codes and [..., K/64, 2] params -> 64-bit [..., K]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    p = params.double()
    return (c.unflatten(-1, (p.shape[-2], 64)) * p[..., 0:1] + p[..., 1:2]).flatten(-2)


def slopes(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float64)


def decode(q, cache, lens, scale, alibi=False):
    """(out, lse, gathered weight) in 64 bits and (out bound, lse bound, weight bound);
    q [B, Hq, K], cache four CPU planes."""
    kc, kp, vc, vp = cache
    B, Hq, K = q.shape
    Hkv, cap = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, K, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    w = torch.zeros(B, Hkv, cap, dtype=torch.float64)
    e_out, e_lse, e_w = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(w)
    sl = slopes(Hq)
    for b, n in enumerate(lens):
        for j in range(Hkv if n else 0):
            k, v = values(kc[b, j, :n], kp[b, j, :n]), values(vc[b, j, :n], vp[b, j, :n])
            s, z = kp[b, j, :n, :, 0].double(), kp[b, j, :n, :, 1].double()
            mag = (15 * s.abs() + z.abs()).repeat_interleave(64, -1)  # [n, K]
            vs = vp[b, j, :n, :, 0].double().abs()
            vz = vp[b, j, :n, :, 1].double().abs()
            vmag = (15 * vs + vz).amax(0).repeat_interleave(64)  # [K]
            for g in range(G):
                h = j * G + g
                qd = q[b, h].double()
                x = k @ qd * scale
                e = (mag @ qd.abs()).amax() * scale * K * 2.0 ** -23
                if alibi:
                    dist = torch.arange(n - 1, -1, -1).double()
                    x = x - sl[h] * dist
                    e = e + sl[h] * n * 2.0 ** -22
                e = float(e) + float(x.abs().amax()) * 2.0 ** -22 + 2.0 ** -20
                L = torch.logsumexp(x, 0)
                p = torch.exp(x - L)
                lse[b, h], out[b, h] = L, p @ v
                w[b, j, :n] += p
                e_lse[b, h] = e + n * 2.0 ** -24
                # a weight and their sum off by a factor e^e each, n sums, the held p s
                rel = 2 * (math.expm1(e) + n * 2.0 ** -23)
                e_out[b, h] = vmag * (rel + HELD[q.dtype]) + out[b, h].abs() * HALF[q.dtype]
                e_w[b, j, :n] += p * rel
    return (out, lse, w), (e_out, e_lse, e_w)


def key_weights(q, k, lse, past, new, causal, scale, alibi=False):
    """Gathered weight of every key and its bound; past / new per sequence (the keys of
    sequence b are rows [0, past + new), or all N with new None)."""
    B, M, Hq, K = q.shape
    N, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    w = torch.zeros(B, Hkv, N, dtype=torch.float64)
    bound = torch.zeros_like(w)
    sl = slopes(Hq)
    for b in range(B):
        m = M if new is None else new[b]
        p0 = N - M if new is None else past[b]
        n = N if new is None else p0 + m
        pos = torch.arange(m)[:, None] + p0
        kj = torch.arange(n)[None]
        for h in range(Hq):
            qd, kd = q[b, :m, h].double(), k[b, :n, h // G].double()
            x = qd @ kd.T * scale
            e = (qd.abs() @ kd.abs().T) * scale * K * 2.0 ** -23 + x.abs() * 2.0 ** -22
            if alibi:
                d = sl[h] * (pos - kj).abs().double()
                x, e = x - d, e + d * 2.0 ** -22
            L = lse[b, h, :m].double()[:, None]
            e = e + L.abs().nan_to_num(0, 0, 0) * 2.0 ** -22 + 2.0 ** -20
            p = torch.exp(x - L)
            p = torch.where(torch.isneginf(L), torch.zeros_like(p), p)
            if causal:
                p = torch.where(kj <= pos, p, torch.zeros_like(p))
            w[b, h // G, :n] += p.sum(0)
            bound[b, h // G, :n] += (p * torch.expm1(e)).sum(0) + p.sum(0) * m * G * 2.0 ** -24
    return w, bound


def choose(w, n, budget, recent):
    """Rows of weights w [cap] kept of n, ascending (ties to the lowest row, NaN least)."""
    if n <= budget:
        return list(range(n))
    old = n - recent
    ws = [-math.inf if math.isnan(x) else x for x in w[:old].tolist()]
    nan = [math.isnan(x) for x in w[:old].tolist()]
    rows = sorted(range(old), key=lambda j: (nan[j], -ws[j], j))
    return sorted(rows[:budget - recent]) + list(range(old, n))
