"""Eviction by gathered weight: rows chosen, moved and counted exactly as sorted lists
say, for 16-bit and 4-bit caches, into another cache and in place."""
import math

import pytest
import torch

import kv4_util as U
from parity_util import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def mea():
    import memory_efficient_exact_mea_b200 as m

    return m


@pytest.fixture(autouse=True)
def status(mea):
    mea.read_device_status()
    yield
    torch.cuda.synchronize()
    assert mea.read_device_status() == 0


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(four, B, cap, Hkv, K, seed):
    """CPU planes of random bytes (16-bit ones as int16 patterns of finite numbers)."""
    if four:
        out = []
        for i in range(2):
            out.append(torch.randint(0, 256, (B, Hkv, cap, K // 2), generator=gen(seed + i),
                                     dtype=torch.uint8))
            out.append(torch.randn(B, Hkv, cap, K // 64, 2, generator=gen(seed + 2 + i)).half())
        return out
    return [torch.randn(B, cap, Hkv, K, generator=gen(seed + i)).bfloat16() for i in range(2)]


def weights(kind, B, Hkv, cap, seed):
    w = torch.rand(B, Hkv, cap, generator=gen(seed))
    if kind == "ties":
        w = (w * 4).floor() / 4
    elif kind == "equal":
        w = torch.full_like(w, 0.5)
    elif kind == "odd":  # NaN, infinities, signed zeros, negative numbers, subnormals
        pick = torch.randint(0, 9, w.shape, generator=gen(seed + 1))
        for i, x in enumerate((math.nan, math.inf, -math.inf, 0.0, -0.0, -1.5, 1e-42)):
            w = torch.where(pick == i, torch.tensor(x), w)
    elif kind == "wide":
        w = torch.exp(30 * (w - 0.5))
    return w


def row_of(four, plane, b, h, idx):
    return plane[b, h, idx] if four else plane[b, idx, h]


def run(mea, four, kind, lens, budget, recent, K=128, Hkv=2, cap=None, in_place=False,
        out_rows=None, seed=0):
    B = len(lens)
    cap = max(max(lens), 1) + 3 if cap is None else cap
    R = cap if in_place else (budget + 2 if out_rows is None else out_rows)
    src = make(four, B, cap, Hkv, K, seed)
    w = weights(kind, B, Hkv, cap, seed + 50)
    wrap = (lambda p: mea.Kv4Cache(*p)) if four else tuple
    dev = [t.to(DEV) for t in src]
    wd = w.to(DEV)
    gk = Guarded((B, Hkv, budget), torch.float32, DEV)  # viewed as int32
    kw = dict(kept=gk.t.view(torch.int32))
    if not in_place:
        shape = (lambda t: (B, Hkv, R, *t.shape[3:])) if four else (lambda t: (B, R, Hkv, K))
        go = [Guarded(shape(t), t.dtype, DEV) for t in src]
        gw = Guarded((B, Hkv, R), torch.float32, DEV)
        old = [g.t.clone() for g in go]
        kw.update(out=wrap([g.t for g in go]), weights_out=gw.t)
    new, kept, wo = mea.mea_cache_evict(wrap(dev), wd, i32(lens), budget, recent, **kw)
    torch.cuda.synchronize()
    gk.check("kept")
    if in_place:
        got, old = dev, src
    else:
        for g in go:
            g.check("out")
        gw.check("weights")
        got = [g.t for g in go]
        assert all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip(dev, src)), "the source was written"
    for b, n in enumerate(lens):
        for h in range(Hkv):
            rows = U.choose(w[b, h], n, budget, recent)
            c = len(rows)
            assert kept[b, h].tolist() == rows + [-1] * (budget - c)
            for s, d, o in zip(src, got, old):
                want = row_of(four, s, b, h, torch.tensor(rows, dtype=torch.long))
                have = row_of(four, d.cpu(), b, h, torch.arange(c))
                assert torch.equal(have.contiguous().view(torch.uint8),
                                   want.contiguous().view(torch.uint8))
                rest = torch.arange(c, R)
                assert torch.equal(row_of(four, d.cpu(), b, h, rest).contiguous().view(torch.uint8),
                                   row_of(four, o.cpu(), b, h, rest).contiguous().view(torch.uint8))
            wr = w[b, h][torch.tensor(rows, dtype=torch.long)]
            assert torch.equal(wo[b, h, :c].cpu().view(torch.int32), wr.view(torch.int32))
            assert (wo[b, h, c:] == 0).all()
        assert int(new[b]) == min(n, budget)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd", "wide"])
def test_choice(mea, four, in_place, kind):
    run(mea, four, kind, [0, 1, 40, 41, 100, 333], 40, 7, in_place=in_place)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (64, 64), (64, 0), (299, 10), (700, 3)])
def test_budgets(mea, four, in_place, budget, recent):
    cap = 800 if in_place else None
    run(mea, four, "random", [300, 64, 700], budget, recent, K=64, Hkv=3, cap=cap,
        in_place=in_place, seed=3)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["random", "ties"])
def test_long(mea, in_place, kind):
    """Several counting and moving tiles; odd capacity (rows of weights not 16-byte aligned)."""
    run(mea, False, kind, [9001, 5000], 4100, 100, K=64, Hkv=1, cap=9007, in_place=in_place)


@pytest.mark.parametrize("cap,lens,Hkv", [(20000, [20000, 9], 1), (70001, [70000], 2),
                                          (140000, [131072], 1), (140000, [140000, 30000], 1)])
@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
def test_clusters(mea, cap, lens, Hkv, kind):
    """Long caches of few heads: the rows of one choice shared by 2 to 8 CTAs."""
    run(mea, True, kind, lens, 3000, 17, K=64, Hkv=Hkv, cap=cap, out_rows=3001)


def test_many_heads(mea):
    run(mea, True, "wide", [150] * 40, 33, 5, K=64, Hkv=16, cap=151)


def test_in_place_equals_out_of_place(mea):
    src = [t.to(DEV) for t in make(False, 2, 3000, 4, 128, 1)]
    w = weights("random", 2, 4, 3000, 2).to(DEV)
    dst = tuple(torch.empty_like(t[:, :1000]) for t in src)
    _, kept, wo = mea.mea_cache_evict(tuple(src), w, i32([3000, 2222]), 1000, 64, out=dst)
    a = [t.clone() for t in src]
    _, kept2, w2 = mea.mea_cache_evict(tuple(a), w, i32([3000, 2222]), 1000, 64)
    assert torch.equal(kept, kept2) and torch.equal(wo, w2[:, :, :1000])
    assert all(torch.equal(x[:, :1000], y) for x, y in zip(a, dst))


def test_strided_and_interleaved_caches(mea):
    """[B, H, rows, K] storage with keys and values side by side, cut in place."""
    B, H, cap, K, n, budget = 2, 3, 200, 64, 190, 50
    both = torch.randn(B, H, cap, 2, K, generator=gen(4)).half().to(DEV)
    before = both.clone()
    k, v = both[:, :, :, 0].transpose(1, 2), both[:, :, :, 1].transpose(1, 2)
    w = weights("random", B, H, cap, 5)
    new, kept, _ = mea.mea_cache_evict((k, v), w.to(DEV), i32([n, n]), budget, 10)
    for b in range(B):
        for h in range(H):
            rows = U.choose(w[b, h], n, budget, 10)
            assert kept[b, h].tolist() == rows
            assert torch.equal(both[b, h, :budget], before[b, h, rows])
            assert torch.equal(both[b, h, budget:], before[b, h, budget:])


def test_one_array_as_keys_and_values_is_refused(mea):
    x = torch.zeros(1, 20, 1, 64, device=DEV).half()
    w = torch.zeros(1, 1, 20, device=DEV)
    with pytest.raises(mea.MeaError):
        mea.mea_cache_evict((x, x), w, i32([20]), 5, 1)
    # read from one array into two it is a copy like any other
    out = (torch.empty_like(x), torch.empty_like(x))
    new, kept, _ = mea.mea_cache_evict((x, x), w, i32([20]), 5, 1, out=out)
    assert kept.tolist() == [[[0, 1, 2, 3, 19]]] and new.tolist() == [5]


def test_bad_lengths_are_reported(mea):
    src = [t.to(DEV) for t in make(False, 2, 50, 2, 64, 1)]
    w = weights("random", 2, 2, 50, 2).to(DEV)
    before = [t.clone() for t in src]
    for bad in (-1, 51, 2 ** 31 - 1):
        new, kept, _ = mea.mea_cache_evict(tuple(src), w.clone(), i32([10, bad]), 20, 5)
        assert mea.read_device_status() == -1
        assert new.tolist() == [10, 0] and (kept[1] == -1).all()
        assert all(torch.equal(a, b) for a, b in zip(src, before))


def test_graph_and_stream(mea):
    """Captured eviction replayed on other weights and lengths; another stream."""
    src = tuple(t.to(DEV) for t in make(False, 2, 400, 2, 64, 7))
    dst = tuple(torch.zeros_like(t[:, :60]) for t in src)
    w, n = torch.zeros(2, 2, 400, device=DEV), i32([400, 400])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new, kept, wo = mea.mea_cache_evict(src, w, n, 50, 9, out=dst)
    for seed, lens in ((1, [400, 77]), (2, [20, 399])):
        w.copy_(weights("ties", 2, 2, 400, seed))
        n.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert new.tolist() == [min(x, 50) for x in lens]
        for b in range(2):
            for h in range(2):
                rows = U.choose(w[b, h].cpu(), lens[b], 50, 9)
                assert kept[b, h, :len(rows)].tolist() == rows
                assert torch.equal(dst[0][b, :len(rows), h], src[0][b, rows, h])
                assert torch.equal(wo[b, h, :len(rows)], w[b, h, rows])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    new2, kept2, wo2 = mea.mea_cache_evict(src, w, n, 50, 9, stream=side,
                                           out=tuple(torch.zeros_like(t) for t in dst))
    side.synchronize()
    assert torch.equal(kept, kept2) and torch.equal(wo, wo2) and torch.equal(new, new2)


def test_two_streams_at_once(mea):
    """Calls on two streams with buffers of their own, interleaved, give what they give alone."""
    a = mea.mea_kv4_alloc(2, 700, 2, 128, torch.bfloat16, DEV)
    b = mea.mea_kv4_alloc(2, 700, 2, 128, torch.bfloat16, DEV)
    x = torch.randn(2, 700, 2, 128, generator=gen(1)).bfloat16().to(DEV)
    q = torch.randn(2, 8, 128, generator=gen(2)).bfloat16().to(DEV)
    for c in (a, b):
        mea.mea_kv4_append(x, x, c, i32([0, 0]))
    n, w = i32([700, 600]), weights("random", 2, 2, 700, 3).to(DEV)
    want = mea.mea_decode_kv4(q, a, n, 700, weights=w, return_weights=True)
    out = mea.mea_kv4_alloc(2, 300, 2, 128, torch.bfloat16, DEV)
    _, kept, _ = mea.mea_cache_evict(a, want[2], n, 300, 30, out=out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [mea.mea_kv4_alloc(2, 300, 2, 128, torch.bfloat16, DEV) for _ in streams]
    for _ in range(5):
        got = []
        for s, c, o in zip(streams, (a, b), outs):
            with torch.cuda.stream(s):
                r = mea.mea_decode_kv4(q, c, n, 700, weights=w, return_weights=True)
                got.append((r, mea.mea_cache_evict(c, r[2], n, 300, 30, out=o)[1]))
        torch.cuda.synchronize()
        for (r, k), o in zip(got, outs):
            assert all(torch.equal(x, y) for x, y in zip(r, want)) and torch.equal(k, kept)
            assert all(torch.equal(x, y) for x, y in zip(o, out))


def test_serving_run(mea):
    """Prompt into the 4-bit cache, its keys weighed, cut to the budget, decode steps that
    keep weighing, cut again in place, decode: every step against the plain forms."""
    B, M, Hq, Hkv, K, budget = 2, 200, 8, 2, 128, 96
    g = gen(6)
    q = torch.randn(B, M, Hq, K, generator=g).bfloat16()
    k = torch.randn(B, M, Hkv, K, generator=g).bfloat16()
    v = torch.randn(B, M, Hkv, K, generator=g).bfloat16()
    out, lse = mea.mea_fwd(q.to(DEV), k.to(DEV), v.to(DEV), bias="causal")
    w = mea.mea_key_weights(q.to(DEV), k.to(DEV), lse)
    ref, bound = U.key_weights(q, k, lse.cpu(), None, None, True, K ** -0.5)
    assert ((w.double().cpu() - ref).abs() <= bound + ref * 2.0 ** -22).all()
    big = mea.mea_kv4_alloc(B, M, Hkv, K, device=DEV)
    mea.mea_kv4_append(k.to(DEV), v.to(DEV), big, i32([0, 0]))
    cap = budget + 8
    small = mea.mea_kv4_alloc(B, cap, Hkv, K, device=DEV)
    wcpu, bigcpu = w.cpu(), [t.cpu() for t in big]
    n, kept, w = mea.mea_cache_evict(big, w, i32([M, M]), budget, 16, out=small)
    for b in range(B):
        for h in range(Hkv):
            rows = U.choose(wcpu[b, h], M, budget, 16)
            assert kept[b, h].tolist() == rows
            for s, d in zip(bigcpu, small):
                assert torch.equal(d[b, h, :budget].cpu(), s[b, h, rows])
    for step in range(12):
        if step == 8:  # the small cache is full: cut it in place
            n, _, w = mea.mea_cache_evict(small, w, n, budget, 16)
        x = torch.randn(B, 1, Hkv, K, generator=g).bfloat16().to(DEV)
        y = torch.randn(B, 1, Hkv, K, generator=g).bfloat16().to(DEV)
        qq = torch.randn(B, Hq, K, generator=g).bfloat16()
        mea.mea_kv4_append(x, y, small, n)
        n = n + 1
        w0 = w.cpu().double()
        o, l, _ = mea.mea_decode_kv4(qq.to(DEV), small, n, cap, weights=w, weights_out=w)
        lens = n.tolist()
        (ro, rl, rw), (eo, el, ew) = U.decode(qq, [t.cpu() for t in small], lens, K ** -0.5)
        assert ((o.double().cpu() - ro).abs() <= eo + 2.0 ** -24).all()
        assert ((l.double().cpu() - rl).abs() <= el).all()
        for b, m in enumerate(lens):
            want = rw[b, :, :m] + w0[b, :, :m]
            assert ((w[b, :, :m].double().cpu() - want).abs()
                    <= ew[b, :, :m] + want * 2.0 ** -22).all()
    assert n.tolist() == [budget + 4] * B
