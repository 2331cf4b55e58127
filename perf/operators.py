"""Cases of the key/value cache operators: a cache held in 4 bits (store, load,
attend), the attention weight each cached key has gathered, and eviction by it.

``own`` false: every operator in its plain form, elementary torch operations in
32 bits (64 where a value next to a border decides a code).  ``own`` true: the
same passes through memory_efficient_exact_mea_b200.

The 4-bit cache: per (sequence, key/value head, row) the K dimensions in groups
of 64; a group keeps 64 codes c in 0..15 (dimension d in byte d/2, even d in the
low four bits) and two 16-bit numbers, step s and zero z, and stands for z + s c.
  codes  uint8 [B, Hkv, rows, K/2]     params 16-bit [B, Hkv, rows, K/64, 2]
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # One new token per sequence put into the cache between two decode steps of a
        # full serving batch, and read back.
        dict(name="store_token", kind="store", B=64, M=1, Hkv=8, K=128, dtype="bf16", cap=1024,
             past_lo=0, past_hi=1000, new_lo=1, new_hi=1),
        # A batch of prompts of unequal length put into an empty cache after prefill.
        dict(name="store_prompts", kind="store", B=8, M=4096, Hkv=8, K=128, dtype="bf16",
             cap=5000, past_lo=0, past_hi=0, new_lo=1001, new_hi=4096),
        # Two short histories brought back to 16 bits for the next chunk of a chat.
        dict(name="load_short", kind="load", B=2, Hkv=16, K=64, dtype="f16", cap=1024, n_lo=300,
             n_hi=999),
        # Long histories brought back to 16 bits before a chunk of prefill.
        dict(name="load_long", kind="load", B=8, Hkv=8, K=128, dtype="bf16", cap=8192,
             n_lo=4097, n_hi=8191),
        # One token of a single short conversation: latency.
        dict(name="decode_single", kind="decode", B=1, Hq=16, Hkv=16, K=64, dtype="f16",
             cap=1024, n_lo=777, n_hi=777, alibi=False, weigh=False),
        # The decode step of the benchmark (B = 64, lengths 512..8192, 32 query heads over 8)
        # on a 4-bit cache.
        dict(name="decode_batch", kind="decode", B=64, Hq=32, Hkv=8, K=128, dtype="bf16",
             cap=8192, n_lo=512, n_hi=8192, alibi=False, weigh=False),
        # Few very long contexts, the weights gathered for a later eviction.
        dict(name="decode_long_weighed", kind="decode", B=4, Hq=32, Hkv=8, K=128, dtype="bf16",
             cap=65536, n_lo=50001, n_hi=65521, alibi=False, weigh=True),
        # The benchmark's grouped-query causal prompt: what each key of it gathered.
        dict(name="weigh_prompt", kind="weigh", B=4, M=4096, Hq=32, Hkv=8, K=128, dtype="bf16",
             cap=4096, past_lo=0, past_hi=0, new_lo=4096, new_hi=4096, causal=True, alibi=False),
        # The benchmark's two-sided forward (B = 8, H = 16, K = 64, M = N = 2048).
        dict(name="weigh_two_sided", kind="weigh", B=8, M=2048, Hq=16, Hkv=16, K=64, dtype="f16",
             cap=2048, past_lo=0, past_hi=0, new_lo=2048, new_hi=2048, causal=False,
             alibi=False),
        # One decode step of a 16-bit cache: the newest query of each sequence.
        dict(name="weigh_token", kind="weigh", B=16, M=1, Hq=32, Hkv=8, K=128, dtype="bf16",
             cap=8192, past_lo=4000, past_hi=8191, new_lo=1, new_hi=1, causal=True,
             alibi=False),
        # Prompts cut down to the decode cache's budget after prefill, 16-bit cache.
        dict(name="evict_prompts", kind="evict", B=8, Hkv=8, K=128, dtype="bf16", cap=8192,
             n_lo=900, n_hi=8192, budget=2048, recent=128, out_rows=2304, four=False),
        # A serving batch on a 4-bit cache cut back when it nears its capacity.
        dict(name="evict_four_bit", kind="evict", B=32, Hkv=8, K=128, dtype="bf16", cap=2048,
             n_lo=1500, n_hi=2047, budget=1000, recent=50, out_rows=1001, four=True),
    ]


def draw(rng: random.Random):
    def size(lo, hi):  # spread over the logarithm
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["store", "load", "decode", "decode", "weigh", "weigh", "evict"])
    K = rng.choice([64, 128])
    dtype = rng.choice(["f16", "bf16"])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    G = rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    if kind == "store":
        M = size(1, 4096)
        past = rng.choice([0, size(1, 2000)])
        B = size(1, max(1, min(64, 262144 // (M * Hkv))))
        return dict(kind=kind, B=B, M=M, Hkv=Hkv, K=K, dtype=dtype, cap=past + M + size(1, 100),
                    past_lo=past // 2, past_hi=past, new_lo=rng.choice([0, M // 2, M]), new_hi=M)
    if kind == "load":
        n = size(1, 8192)
        B = size(1, max(1, min(64, 400000 // (n * Hkv))))
        return dict(kind=kind, B=B, Hkv=Hkv, K=K, dtype=dtype, cap=n + size(1, 500), n_lo=n // 3,
                    n_hi=n)
    if kind == "decode":
        n = size(1, 65536)
        B = size(1, max(1, min(64, 2000000 // (n * Hkv))))
        return dict(kind=kind, B=B, Hq=Hkv * G, Hkv=Hkv, K=K, dtype=dtype, cap=n + size(1, 300),
                    n_lo=n // 3, n_hi=n, alibi=rng.random() < 0.3, weigh=rng.random() < 0.5)
    if kind == "weigh":
        M = rng.choice([1, size(2, 40), size(16, 4096), size(64, 4096)])
        past = rng.choice([0, size(1, 8000)])
        room = 1_000_000_000 // (Hkv * G * M * (past + M))
        B = size(1, max(1, min(16, room)))
        return dict(kind=kind, B=B, M=M, Hq=Hkv * G, Hkv=Hkv, K=K, dtype=dtype,
                    cap=past + M + rng.choice([0, size(1, 300)]), past_lo=past // 2,
                    past_hi=past, new_lo=rng.choice([M, M // 2]), new_hi=M,
                    causal=rng.random() < 0.7, alibi=rng.random() < 0.3)
    n = size(2, 16384)
    B = size(1, max(1, min(64, 400000 // (n * Hkv))))
    budget = size(1, n)
    return dict(kind=kind, B=B, Hkv=Hkv, K=K, dtype=dtype, cap=n + size(1, 100), n_lo=n // 2,
                n_hi=n, budget=budget, recent=rng.choice([0, budget // 8, budget // 2, budget]),
                out_rows=budget + size(1, 200), four=rng.random() < 0.4)


def _spread(case, lo, hi, what):
    """One length a sequence, the same for every seed: hi first, the rest between lo and hi."""
    r = random.Random(f"{what}/{case['B']}/{lo}/{hi}")
    return [hi] + [r.randint(lo, hi) for _ in range(case["B"] - 1)]


def _lens(case):
    if case["kind"] in ("store", "weigh"):
        return (_spread(case, case["past_lo"], case["past_hi"], "past"),
                _spread(case, case["new_lo"], case["new_hi"], "new"))
    return _spread(case, case["n_lo"], case["n_hi"], "n")


def work(case):
    B, Hkv, K, kind = case["B"], case["Hkv"], case["K"], case["kind"]
    row16 = 2 * K * 2                    # key and value of one row and head, 16 bits
    row4 = 2 * (K // 2 + K // 64 * 4)    # the same in 4 bits
    if kind == "store":
        past, new = _lens(case)
        rows = sum(new) * Hkv
        # in 16-bit rows, out 4-bit rows; and those back into 16 bits
        return dict(bytes=rows * (2 * row16 + row4) + 8 * B, flops=rows * 2 * K * 8)
    if kind == "load":
        rows = sum(_lens(case)) * Hkv
        return dict(bytes=rows * (row16 + row4) + 4 * B, flops=rows * 2 * K * 2)
    if kind == "decode":
        n = sum(_lens(case))
        by = n * Hkv * row4 + B * case["Hq"] * (K * 4 + 4) + 4 * B
        if case["weigh"]:
            by += n * Hkv * 4 + B * Hkv * case["cap"] * 4
        return dict(bytes=by, flops=4 * K * case["Hq"] * n)
    if kind == "weigh":
        past, new = _lens(case)
        G = case["Hq"] // Hkv
        pairs = sum(m * p + (m * (m + 1) // 2 if case["causal"] else m * m)
                    for p, m in zip(past, new))
        keys = sum(p + m for p, m in zip(past, new))
        by = (keys * Hkv * (K * 2 + 4) + B * Hkv * case["cap"] * 4
              + sum(new) * case["Hq"] * (K * 2 + 4))
        return dict(bytes=by, flops=2 * K * pairs * Hkv * G)
    lens = _lens(case)
    kept = [min(n, case["budget"]) for n in lens]
    row = row4 if case["four"] else row16
    by = (sum(lens) * Hkv * 4                       # every weight once
          + sum(kept) * Hkv * (2 * row + 4)         # the kept rows and weights, moved
          + B * Hkv * case["budget"] * 4            # their indices
          + (B * case["out_rows"] - sum(kept)) * Hkv * 4)  # the weights of rows to come: zero
    if case["four"]:
        by += sum(kept) * Hkv * (row4 + row16)      # and back in 16 bits
    return dict(bytes=by, flops=sum(lens) * Hkv * 4)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _keys(shape, dtype, g, lift):
    """Keys and values as models have them: N(0, 1), a few dimensions of the keys far
    from zero, rounded to 16 bits.  shape [..., K]."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if lift:
        x[..., ::37] += 4.0
    return x.to(dtype)


def _fold(x):
    """16-bit rows [..., K] -> (codes uint8 [..., K/2], params [..., K/64, 2]); input making
    only, in 32 bits."""
    K = x.shape[-1]
    xg = x.float().unflatten(-1, (K // 64, 64))
    mn, mx = xg.amin(-1), xg.amax(-1)
    s, z = ((mx - mn) / 15).to(x.dtype), mn.to(x.dtype)
    c = ((xg - z.float()[..., None]) / s.float()[..., None].clamp_min(1e-30)).round()
    c = c.clamp_(0, 15).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack((s, z), -1)


def _four_bit_cache(case, lens, g):
    """A filled 4-bit cache; rows past a sequence's length are zeros."""
    B, Hkv, K, cap = case["B"], case["Hkv"], case["K"], case["cap"]
    dt = _DT[case["dtype"]]
    planes = []
    for lift in (True, False):
        codes = torch.zeros(B, Hkv, cap, K // 2, dtype=torch.uint8, device="cuda")
        params = torch.zeros(B, Hkv, cap, K // 64, 2, dtype=dt, device="cuda")
        for b, n in enumerate(lens):
            if n:
                c, p = _fold(_keys((Hkv, n, K), dt, g, lift))
                codes[b, :, :n], params[b, :, :n] = c, p
        planes += [codes, params]
    return planes  # k_codes, k_params, v_codes, v_params


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _slopes(Hq):
    return [2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)]


def _scores(q, k, case, past, h, wide):
    """Scaled scores of query head h, biased and masked (q [m, K], k [n, K])."""
    s = (q.to(wide) @ k.to(wide).T) * (case["K"] ** -0.5)
    pi = torch.arange(q.shape[0], device="cuda")[:, None] + past
    kj = torch.arange(k.shape[0], device="cuda")[None, :]
    if case["alibi"]:
        s = s - _slopes(case["Hq"])[h] * (pi - kj).abs().to(wide)
    if case["causal"]:
        s = s.masked_fill(kj > pi, -math.inf)
    return s


def prepare(case, seed):
    g = _gen(seed)
    kind, B, Hkv, K = case["kind"], case["B"], case["Hkv"], case["K"]
    dt = _DT[case["dtype"]]
    st = dict(case=case)
    if kind == "store":
        past, new = _lens(case)
        st["past"], st["new"] = past, new
        st["past_t"], st["new_t"] = _int(past), _int(new)
        st["k"] = _keys((B, case["M"], Hkv, K), dt, g, True)
        st["v"] = _keys((B, case["M"], Hkv, K), dt, g, False)
        st["cache"] = _four_bit_cache(case, [0] * B, g)
        st["k_out"], st["v_out"] = torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
    elif kind == "load":
        st["n"] = _lens(case)
        st["n_t"] = _int(st["n"])
        st["cache"] = _four_bit_cache(case, st["n"], g)
        st["k_out"] = torch.zeros(B, case["cap"], Hkv, K, dtype=dt, device="cuda")
        st["v_out"] = torch.zeros_like(st["k_out"])
    elif kind == "decode":
        st["n"] = _lens(case)
        st["n_t"] = _int(st["n"])
        st["q"] = torch.randn(B, case["Hq"], K, generator=g, device="cuda").to(dt)
        st["cache"] = _four_bit_cache(case, st["n"], g)
        if case["weigh"]:
            st["weights"] = torch.rand(B, Hkv, case["cap"], generator=g, device="cuda")
        if own:
            import memory_efficient_exact_mea_b200 as mea

            need = mea.mea_decode_kv4_workspace_size(B, case["Hq"], Hkv, K, max(st["n"]),
                                                     case["weigh"])
            st["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    elif kind == "weigh":
        past, new = _lens(case)
        st["past"], st["new"] = past, new
        st["past_t"], st["new_t"] = _int(past), _int(new)
        st["q"] = torch.randn(B, case["M"], case["Hq"], K, generator=g, device="cuda").to(dt)
        st["k"] = _keys((B, case["cap"], Hkv, K), dt, g, True)
        st["weights"] = torch.rand(B, Hkv, case["cap"], generator=g, device="cuda")
        # the log-sum-exp that the attention of these queries returned
        lse = torch.zeros(B, case["Hq"], case["M"], device="cuda")
        G = case["Hq"] // Hkv
        for b in range(B):
            for h in range(case["Hq"]):
                if new[b]:
                    s = _scores(st["q"][b, :new[b], h], st["k"][b, :past[b] + new[b], h // G],
                                case, past[b], h, torch.float32)
                    lse[b, h, :new[b]] = torch.logsumexp(s, -1)
        st["lse"] = lse
    else:
        st["n"] = _lens(case)
        st["n_t"] = _int(st["n"])
        cap, R = case["cap"], case["out_rows"]
        # weights as attention leaves them: a few heavy keys, many light ones, and
        # some (those just added) still at zero
        w = torch.randn(B, Hkv, cap, generator=g, device="cuda").mul_(2).exp_()
        w = w * (torch.rand(B, Hkv, cap, generator=g, device="cuda") > 0.02)
        st["weights"] = w
        if case["four"]:
            st["cache"] = _four_bit_cache(case, st["n"], g)
            st["out"] = [torch.zeros(B, Hkv, R, *p.shape[3:], dtype=p.dtype, device="cuda")
                         for p in st["cache"]]
            st["k_out"] = torch.zeros(B, R, Hkv, K, dtype=dt, device="cuda")
            st["v_out"] = torch.zeros_like(st["k_out"])
        else:
            st["cache"] = [_keys((B, cap, Hkv, K), dt, g, x) for x in (True, False)]
            st["out"] = [torch.zeros(B, R, Hkv, K, dtype=dt, device="cuda") for _ in range(2)]
        st["kept"] = torch.zeros(B, Hkv, case["budget"], dtype=torch.int32, device="cuda")
        st["weights_out"] = torch.zeros(B, Hkv, R, device="cuda")
        st["new_n"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return st


# ----------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------
def _run_own(st):
    import memory_efficient_exact_mea_b200 as mea

    case, kind = st["case"], st["case"]["kind"]
    if kind == "store":
        cache = mea.Kv4Cache(*st["cache"])
        mea.mea_kv4_append(st["k"], st["v"], cache, st["past_t"], st["new_t"])
        return mea.mea_kv4_read(cache, st["new_t"], first_rows=st["past_t"], k_out=st["k_out"],
                                v_out=st["v_out"])
    if kind == "load":
        return mea.mea_kv4_read(mea.Kv4Cache(*st["cache"]), st["n_t"], k_out=st["k_out"],
                                v_out=st["v_out"])
    if kind == "decode":
        cache = mea.Kv4Cache(*st["cache"])
        if case["weigh"]:
            return mea.mea_decode_kv4(st["q"], cache, st["n_t"], max(st["n"]),
                                      alibi=case["alibi"], weights=st["weights"],
                                      return_weights=True, workspace=st["ws"])
        return mea.mea_decode_kv4(st["q"], cache, st["n_t"], max(st["n"]), alibi=case["alibi"],
                                  workspace=st["ws"])
    if kind == "weigh":
        return mea.mea_key_weights(st["q"], st["k"], st["lse"], st["past_t"], st["new_t"],
                                   causal=case["causal"], alibi=case["alibi"],
                                   weights=st["weights"])
    four = case["four"]
    src = mea.Kv4Cache(*st["cache"]) if four else tuple(st["cache"])
    dst = mea.Kv4Cache(*st["out"]) if four else tuple(st["out"])
    new_n, kept, w = mea.mea_cache_evict(src, st["weights"], st["n_t"], case["budget"],
                                         case["recent"], out=dst, weights_out=st["weights_out"],
                                         new_seqlens=st["new_n"], kept=st["kept"])
    if four:
        k, v = mea.mea_kv4_read(dst, new_n, k_out=st["k_out"], v_out=st["v_out"])
        return k, v, w, kept, new_n
    return dst[0], dst[1], w, kept, new_n


# ----------------------------------------------------------------------------
# the plain form
# ----------------------------------------------------------------------------
def _quantise(x):
    """16-bit rows [..., K] -> (codes 0..15 [..., K/64, 64], s, z): z the least value of a
    group, s a fifteenth of its range, c the nearest whole number to (x - z) / s."""
    xg = x.double().unflatten(-1, (x.shape[-1] // 64, 64))
    mn, mx = xg.amin(-1), xg.amax(-1)
    s, z = ((mx - mn) / 15).float().to(x.dtype), mn.to(x.dtype)
    sd = s.double()[..., None]
    c = torch.where(sd > 0, (xg - z.double()[..., None]) / sd, 0.0).round().clamp(0, 15)
    return c, s, z


def _pack(c):
    c = c.to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _values(codes, params):
    """What codes [..., K/2] and params [..., K/64, 2] stand for, in 32 bits [..., K]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    p = params.float()
    c = c.unflatten(-1, (params.shape[-2], 64))
    return (c * p[..., 0:1] + p[..., 1:2]).flatten(-2)


def _plain_store(st):
    kc, kp, vc, vp = st["cache"]
    for x, codes, params, out in ((st["k"], kc, kp, st["k_out"]), (st["v"], vc, vp, st["v_out"])):
        for b, (p, m) in enumerate(zip(st["past"], st["new"])):
            if m:
                c, s, z = _quantise(x[b, :m].transpose(0, 1))
                codes[b, :, p:p + m] = _pack(c)
                params[b, :, p:p + m] = torch.stack((s, z), -1)
                out[b, :m] = _values(codes[b, :, p:p + m], params[b, :, p:p + m]).transpose(
                    0, 1).to(out.dtype)
    return st["k_out"], st["v_out"]


def _plain_load(planes, lens, k_out, v_out):
    for codes, params, out in ((planes[0], planes[1], k_out), (planes[2], planes[3], v_out)):
        for b, n in enumerate(lens):
            out[b, :n] = _values(codes[b, :, :n], params[b, :, :n]).transpose(0, 1).to(out.dtype)
    return k_out, v_out


def _plain_decode(st):
    case = st["case"]
    Hq, Hkv, K, cap = case["Hq"], case["Hkv"], case["K"], case["cap"]
    G = Hq // Hkv
    q = st["q"].float()
    out = torch.zeros_like(st["q"])
    lse = torch.full((case["B"], Hq), -math.inf, device="cuda")
    w = torch.zeros(case["B"], Hkv, cap, device="cuda") if case["weigh"] else None
    slope = torch.tensor(_slopes(Hq), device="cuda").view(Hkv, G, 1)
    kc, kp, vc, vp = st["cache"]
    for b, n in enumerate(st["n"]):
        if n == 0:
            continue
        k = _values(kc[b, :, :n], kp[b, :, :n])
        v = _values(vc[b, :, :n], vp[b, :, :n])
        s = q[b].view(Hkv, G, K) @ k.transpose(1, 2) * K ** -0.5
        if case["alibi"]:
            s = s - slope * (n - 1 - torch.arange(n, device="cuda")).float()
        m = s.amax(-1, keepdim=True)
        e = (s - m).exp()
        l = e.sum(-1, keepdim=True)
        out[b] = ((e @ v) / l).reshape(Hq, K).to(out.dtype)
        lse[b] = (m + l.log()).reshape(Hq)
        if w is not None:
            w[b, :, :n] = st["weights"][b, :, :n] + (e / l).sum(1)
    return (out, lse) if w is None else (out, lse, w)


def _plain_weigh(st):
    case = st["case"]
    G = case["Hq"] // case["Hkv"]
    w = torch.zeros_like(st["weights"])
    for b, (p, m) in enumerate(zip(st["past"], st["new"])):
        n = p + m
        w[b, :, :n] = st["weights"][b, :, :n]
        for h in range(case["Hq"] if m else 0):
            s = _scores(st["q"][b, :m, h], st["k"][b, :n, h // G], case, p, h, torch.float32)
            w[b, h // G, :n] += (s - st["lse"][b, h, :m, None]).exp().sum(0)
    return w


def _choose(w, n, budget, recent):
    """The rows kept of weights w [Hkv, n], ascending: [Hkv, min(n, budget)]."""
    if n <= budget:
        return torch.arange(n, device="cuda").expand(w.shape[0], n)
    order = torch.sort(w[:, :n - recent], dim=-1, descending=True, stable=True).indices
    old = order[:, :budget - recent].sort(-1).values
    new = torch.arange(n - recent, n, device="cuda").expand(w.shape[0], recent)
    return torch.cat((old, new), -1)


def _plain_evict(st):
    case = st["case"]
    R, four = case["out_rows"], case["four"]
    st["weights_out"].zero_()
    st["kept"].fill_(-1)
    for b, n in enumerate(st["n"]):
        idx = _choose(st["weights"][b], n, case["budget"], case["recent"])
        c = idx.shape[1]
        st["new_n"][b] = c
        st["kept"][b, :, :c] = idx.to(torch.int32)
        st["weights_out"][b, :, :c] = st["weights"][b].gather(1, idx)
        heads = torch.arange(case["Hkv"], device="cuda")[:, None]
        for src, dst in zip(st["cache"], st["out"]):
            if four:
                dst[b, :, :c] = src[b, heads, idx]
            else:
                dst[b, :c] = src[b, idx, heads].transpose(0, 1)
    tail = (st["weights_out"], st["kept"], st["new_n"])
    if four:
        new = [min(n, case["budget"]) for n in st["n"]]
        return (*_plain_load(st["out"], new, st["k_out"], st["v_out"]), *tail)
    return (st["out"][0], st["out"][1], *tail)


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind == "store":
        return _plain_store(state)
    if kind == "load":
        return _plain_load(state["cache"], state["n"], state["k_out"], state["v_out"])
    if kind == "decode":
        return _plain_decode(state)
    if kind == "weigh":
        return _plain_weigh(state)
    return _plain_evict(state)


# ----------------------------------------------------------------------------
# the definitions in 64 bits, one (sequence, head) at a time
# ----------------------------------------------------------------------------
def _stands_for(codes, params):
    """[n, K/2] codes and [n, K/64, 2] params -> [n, K] in 64 bits."""
    n, half = codes.shape
    x = torch.empty(n, 2 * half, dtype=torch.float64, device="cuda")
    x[:, 0::2] = (codes % 16).double()
    x[:, 1::2] = (codes // 16).double()
    for gr in range(half // 32):
        cut = x[:, 64 * gr:64 * gr + 64]
        cut.mul_(params[:, gr, 0, None].double()).add_(params[:, gr, 1, None].double())
    return x


def _exact_store(st):
    outs = []
    for x in (st["k"], st["v"]):
        o = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for b, m in enumerate(st["new"]):
            for gr in range(x.shape[-1] // 64):
                y = x[b, :m, :, 64 * gr:64 * gr + 64].double()
                if m == 0:
                    continue
                low = y.min(-1, keepdim=True).values
                step = ((y.max(-1, keepdim=True).values - low) / 15).to(x.dtype).double()
                c = torch.round((y - low) / step).clamp(0, 15)
                o[b, :m, :, 64 * gr:64 * gr + 64] = torch.where(step > 0, low + step * c, low)
        outs.append(o)
    return tuple(outs)


def _exact_load(planes, lens, shape):
    outs = []
    for codes, params in ((planes[0], planes[1]), (planes[2], planes[3])):
        o = torch.zeros(shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            for h in range(codes.shape[1]):
                o[b, :n, h] = _stands_for(codes[b, h, :n], params[b, h, :n])
        outs.append(o)
    return tuple(outs)


def _exact_decode(st):
    case = st["case"]
    B, Hq, Hkv, K = case["B"], case["Hq"], case["Hkv"], case["K"]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, K, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    w = torch.zeros(B, Hkv, case["cap"], dtype=torch.float64, device="cuda")
    kc, kp, vc, vp = st["cache"]
    slopes = torch.tensor(_slopes(Hq), dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["n"]):
        for j in range(Hkv if n else 0):
            heads = slice(j * G, j * G + G)
            x = _stands_for(kc[b, j, :n], kp[b, j, :n]) @ st["q"][b, heads].double().T
            x = x / math.sqrt(K)                                      # [n, G]
            if case["alibi"]:
                back = torch.arange(n - 1, -1, -1, device="cuda").double()
                x = x - back[:, None] * slopes[None, heads]
            L = torch.logsumexp(x, 0)
            p = torch.exp(x - L)
            lse[b, heads] = L
            out[b, heads] = p.T @ _stands_for(vc[b, j, :n], vp[b, j, :n])
            if case["weigh"]:
                w[b, j, :n] = st["weights"][b, j, :n].double() + p.sum(1)
    return (out, lse, w) if case["weigh"] else (out, lse)


def _exact_weigh(st):
    case = st["case"]
    Hq, G = case["Hq"], case["Hq"] // case["Hkv"]
    w = torch.zeros(st["weights"].shape, dtype=torch.float64, device="cuda")
    for b, (p, m) in enumerate(zip(st["past"], st["new"])):
        n = p + m
        w[b, :, :n] = st["weights"][b, :, :n].double()
        kj = torch.arange(n, device="cuda")
        for i0 in range(0, m, 1024):
            i1 = min(m, i0 + 1024)
            pos = torch.arange(p + i0, p + i1, device="cuda")
            for h in range(Hq):
                x = st["k"][b, :n, h // G].double() @ st["q"][b, i0:i1, h].double().T
                x = x / math.sqrt(case["K"])                          # [n, rows]
                if case["alibi"]:
                    x -= 2.0 ** (-8.0 * (h + 1) / Hq) * (pos[None] - kj[:, None]).abs().double()
                e = torch.exp(x - st["lse"][b, h, None, i0:i1].double())
                if case["causal"]:
                    e = torch.where(kj[:, None] <= pos[None], e, 0.0)
                w[b, h // G, :n] += e.sum(1)
    return w


def _exact_evict(st):
    case = st["case"]
    B, Hkv, K, R = case["B"], case["Hkv"], case["K"], case["out_rows"]
    kept = torch.full((B, Hkv, case["budget"]), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(B, Hkv, R, dtype=torch.float64, device="cuda")
    k = torch.zeros(B, R, Hkv, K, dtype=torch.float64, device="cuda")
    v = torch.zeros_like(k)
    new = []
    for b, n in enumerate(st["n"]):
        for h in range(Hkv):
            rows = list(range(n))
            if n > case["budget"]:
                old = n - case["recent"]
                ws = st["weights"][b, h, :old].double().tolist()
                rows = sorted(range(old), key=lambda j: (-ws[j], j))
                rows = sorted(rows[:case["budget"] - case["recent"]]) + list(range(old, n))
            c = len(rows)
            ix = torch.tensor(rows, dtype=torch.int64, device="cuda")
            kept[b, h, :c] = ix.to(torch.int32)
            w[b, h, :c] = st["weights"][b, h][ix].double()
            if case["four"]:
                kc, kp, vc, vp = st["cache"]
                k[b, :c, h] = _stands_for(kc[b, h][ix], kp[b, h][ix])
                v[b, :c, h] = _stands_for(vc[b, h][ix], vp[b, h][ix])
            else:
                k[b, :c, h] = st["cache"][0][b, ix, h].double()
                v[b, :c, h] = st["cache"][1][b, ix, h].double()
        new.append(c)
    return k, v, w, kept, _int(new)


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "store":
        return _exact_store(st)
    if kind == "load":
        return _exact_load(st["cache"], st["n"], st["k_out"].shape)
    if kind == "decode":
        return _exact_decode(st)
    if kind == "weigh":
        return _exact_weigh(st)
    return _exact_evict(st)
