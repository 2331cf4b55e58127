"""The 4-bit cache: rows put into it, read back, and one decode step against it,
against their plain 64-bit forms (bounds derived in kv4_util)."""
import math

import pytest
import torch

import kv4_util as U
from parity_util import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


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


def rows(shape, dtype, seed):
    x = torch.randn(*shape, generator=gen(seed))
    x[..., ::37] += 4.0
    return x.to(DT[dtype])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bits(t):
    return t.contiguous().view(torch.uint8 if t.dtype == torch.uint8 else torch.int16)


def same_params(got, ref):
    """Equal bits, any NaN counting as any other."""
    nan = torch.isnan(ref.float())
    assert torch.equal(torch.isnan(got.float()), nan)
    assert torch.equal(bits(got)[~nan.view(got.shape)], bits(ref)[~nan.view(ref.shape)])


def guarded_cache(mea, B, cap, Hkv, K, dtype):
    gs = []
    for _ in range(2):
        gs.append(Guarded((B, Hkv, cap, K // 2), torch.uint8, DEV, fill=0xEE))
        gs.append(Guarded((B, Hkv, cap, K // 64, 2), DT[dtype], DEV, fill=7.0))
    return mea.Kv4Cache(*(g.t for g in gs)), gs


@pytest.mark.parametrize("K,dtype,Hkv,M,past,new", [
    (128, "bf16", 8, 1, [0, 5, 63], [1, 1, 1]),
    (64, "f16", 3, 1, [0, 1], [1, 0]),
    (128, "f16", 2, 77, [0, 10, 3], [77, 0, 41]),
    (64, "bf16", 5, 130, [17, 0], [129, 130]),
    (128, "bf16", 1, 300, [0], [300]),
])
def test_append_writes_the_definition(mea, K, dtype, Hkv, M, past, new):
    B, cap = len(past), max(p + n for p, n in zip(past, new)) + 3
    k, v = rows((B, M, Hkv, K), dtype, 1), rows((B, M, Hkv, K), dtype, 2)
    cache, gs = guarded_cache(mea, B, cap, Hkv, K, dtype)
    before = [t.clone() for t in cache]
    mea.mea_kv4_append(k.to(DEV), v.to(DEV), cache, i32(past), i32(new))
    torch.cuda.synchronize()
    for g in gs:
        g.check("append")
    for x, (ci, pi) in ((k, (0, 1)), (v, (2, 3))):
        codes, params = U.planes(x)
        for b, (p, n) in enumerate(zip(past, new)):
            want_c, want_p = before[ci][b].cpu(), before[pi][b].cpu()
            want_c[:, p:p + n], want_p[:, p:p + n] = codes[b, :, :n], params[b, :, :n]
            assert torch.equal(cache[ci][b].cpu(), want_c)
            assert torch.equal(bits(cache[pi][b].cpu()), bits(want_p))


def test_append_without_q_seqlens_and_strided_rows(mea):
    """[B, H, M, K] storage, K and V views of one array, and no q_seqlens."""
    B, M, H, K = 2, 19, 3, 64
    both = rows((B, H, M, 2, K), "f16", 3).to(DEV)
    k, v = both[:, :, :, 0].transpose(1, 2), both[:, :, :, 1].transpose(1, 2)
    cache = mea.mea_kv4_alloc(B, M, H, K, torch.float16, DEV)
    mea.mea_kv4_append(k, v, cache, i32([0, 0]))
    for x, (ci, pi) in ((k, (0, 1)), (v, (2, 3))):
        codes, params = U.planes(x.cpu())
        assert torch.equal(cache[ci].cpu(), codes) and torch.equal(cache[pi].cpu(), params)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_hard_values(mea, dtype):
    """Equal values, signed zeros, exact halves between codes, the type's largest and
    smallest numbers, and groups that hold a NaN or an infinity."""
    dt = DT[dtype]
    big, tiny = torch.finfo(dt).max, torch.finfo(dt).smallest_normal
    g = torch.zeros(10, 64)
    g[0] = 3.25
    g[1, ::2] = -0.0
    g[2] = torch.arange(64) * 0.25                      # step 1.05: inexact
    g[3] = (torch.arange(64) % 31) * 0.5                # step 1: every other value a tie
    g[4, 0], g[4, 1] = big, -big
    g[5] = torch.arange(64) * tiny / 64
    g[6, 3] = math.nan
    g[7, 63] = math.inf
    g[8, 0] = -math.inf
    g[9] = 1000.0 + (torch.arange(64) % 16) * 8.0
    x = g.to(dt).reshape(1, 5, 1, 128)
    cache = mea.mea_kv4_alloc(1, 5, 1, 128, dt, DEV)
    mea.mea_kv4_append(x.to(DEV), x.to(DEV), cache, i32([0]))
    codes, params = U.planes(x)
    assert torch.equal(cache.k_codes.cpu(), codes) and torch.equal(cache.v_codes.cpu(), codes)
    same_params(cache.k_params.cpu(), params)
    k, _ = mea.mea_kv4_read(cache, i32([5]))
    assert torch.equal(torch.isnan(k.cpu()).view(10, 64).all(1), torch.tensor(
        [i in (6, 7, 8) for i in range(10)]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_random_codes_are_exact(mea, dtype):
    """Every code of 2^20 elements, over steps of many sizes (ties among them)."""
    x = torch.randn(1, 4096, 2, 128, generator=gen(5)) * torch.exp2(
        torch.randint(-10, 8, (1, 4096, 2, 1), generator=gen(6)).float())
    x = (x * 8).round().div(8).to(DT[dtype])
    cache = mea.mea_kv4_alloc(1, 4096, 2, 128, DT[dtype], DEV)
    mea.mea_kv4_append(x.to(DEV), x.to(DEV), cache, i32([0]))
    codes, params = U.planes(x)
    assert torch.equal(cache.v_codes.cpu(), codes)
    assert torch.equal(cache.v_params.cpu(), params)


@pytest.mark.parametrize("K,dtype,Hkv,first,count", [
    (128, "bf16", 4, None, [0, 1, 33]), (64, "f16", 3, [5, 0, 30], [20, 0, 7]),
    (64, "bf16", 1, [1, 2, 3], [34, 1, 2]), (128, "f16", 8, None, [37, 36, 1])])
def test_read(mea, K, dtype, Hkv, first, count):
    B, cap, R = len(count), 37, max(count) + 2
    codes = [torch.randint(0, 256, (B, Hkv, cap, K // 2), generator=gen(i), dtype=torch.uint8)
             for i in (1, 2)]
    params = [torch.randn(B, Hkv, cap, K // 64, 2, generator=gen(i)).to(DT[dtype])
              for i in (3, 4)]
    cache = mea.Kv4Cache(*(t.to(DEV) for t in (codes[0], params[0], codes[1], params[1])))
    gk = Guarded((B, R, Hkv, K), DT[dtype], DEV, fill=9.0)
    gv = Guarded((B, R, Hkv, K), DT[dtype], DEV, fill=9.0)
    mea.mea_kv4_read(cache, i32(count), None if first is None else i32(first), k_out=gk.t,
                     v_out=gv.t)
    torch.cuda.synchronize()
    gk.check("k"), gv.check("v")
    for i, got in enumerate((gk.t, gv.t)):
        ref = U.values(codes[i], params[i]).transpose(1, 2)
        for b, n in enumerate(count):
            f = 0 if first is None else first[b]
            want = ref[b, f:f + n]
            err = (got[b, :n].double().cpu() - want).abs()
            # one rounding to 16 bits (half the least step below the normal range), one in fp32
            tol = want.abs() * (U.HALF[DT[dtype]] + 2.0 ** -23) + 2.0 ** -25 + 15 * 2.0 ** -22
            assert (err <= tol).all()
            assert (got[b, n:] == 9.0).all()


def make_cache(mea, lens, cap, Hkv, K, dtype, seed=0, spoil=True):
    """A cache holding lens[b] rows per sequence; the rest spoiled (NaN params)."""
    B, m = len(lens), max(max(lens), 1)
    cache = mea.mea_kv4_alloc(B, cap, Hkv, K, DT[dtype], DEV)
    if spoil:
        for i in (0, 2):
            cache[i].fill_(0xFF)
            cache[i + 1].fill_(math.nan)
    k, v = rows((B, m, Hkv, K), dtype, seed + 1), rows((B, m, Hkv, K), dtype, seed + 2)
    mea.mea_kv4_append(k.to(DEV), v.to(DEV), cache, i32([0] * B), i32(lens))
    return cache


def check_decode(mea, cache, q, lens, scale, alibi=False, weigh=True, bound=None, **kw):
    B, Hq, K = q.shape
    Hkv, cap = cache.k_codes.shape[1:3]
    bound = max(max(lens), 1) if bound is None else bound
    go = Guarded(tuple(q.shape), q.dtype, DEV, fill=float("nan"))
    gl = Guarded((B, Hq), torch.float32, DEV, fill=5.0)
    gw = Guarded((B, Hkv, cap), torch.float32, DEV, fill=5.0)
    ws = Guarded((max(1, mea.mea_decode_kv4_workspace_size(B, Hq, Hkv, K, bound, weigh)),),
                 torch.uint8, DEV)
    win = torch.rand(B, Hkv, cap, generator=gen(99))
    res = mea.mea_decode_kv4(q.to(DEV), cache, i32(lens), bound, scale=scale, alibi=alibi,
                             weights=win.to(DEV) if weigh else None,
                             weights_out=gw.t if weigh else None, out=go.t, lse=gl.t,
                             workspace=ws.t, **kw)
    torch.cuda.synchronize()
    for g, what in ((go, "out"), (gl, "lse"), (gw, "weights"), (ws, "workspace")):
        g.check(what)
    cpu = [t.cpu() for t in cache]
    (out, lse, w), (eo, el, ew) = U.decode(q, cpu, lens, scale, alibi)
    got = go.t.double().cpu()
    assert ((got - out).abs() <= eo + 2.0 ** -24).all(), (got - out).abs().max()
    assert torch.equal(torch.isneginf(gl.t.cpu()), torch.isneginf(lse))
    fin = ~torch.isneginf(lse)
    assert ((gl.t.double().cpu() - lse).abs()[fin] <= el[fin]).all()
    if weigh:
        for b, n in enumerate(lens):
            ref = w[b, :, :n] + win[b, :, :n].double()
            err = (gw.t[b, :, :n].double().cpu() - ref).abs()
            assert (err <= ew[b, :, :n] + ref * 2.0 ** -22).all()
            assert (gw.t[b, :, n:] == 0).all()
    return res


@pytest.mark.parametrize("K,dtype", [(64, "f16"), (64, "bf16"), (128, "f16"), (128, "bf16")])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (6, 2), (8, 1), (15, 3), (9, 1), (20, 1)])
def test_decode_ragged(mea, K, dtype, Hq, Hkv):
    lens = [0, 1, 31, 33, 127, 129, 300]
    cache = make_cache(mea, lens, 305, Hkv, K, dtype, seed=Hq)
    q = torch.randn(len(lens), Hq, K, generator=gen(7)).to(DT[dtype])
    check_decode(mea, cache, q, lens, K ** -0.5, alibi=Hq == 6)


@pytest.mark.parametrize("K,dtype,lens,bound", [
    (128, "bf16", [4500, 1, 1023, 2048], 4500), (64, "f16", [1025, 1024, 999, 2500], 2600),
    (128, "f16", [3000], 3000)])
@pytest.mark.parametrize("weigh", [False, True])
def test_decode_splits(mea, K, dtype, lens, bound, weigh):
    cache = make_cache(mea, lens, 4601, 2, K, dtype)
    q = torch.randn(len(lens), 8, K, generator=gen(8)).to(DT[dtype])
    check_decode(mea, cache, q, lens, K ** -0.5, weigh=weigh, bound=bound)


def test_decode_single_split_full_grid(mea):
    """Enough sequences that each gets one split: the result is written in one launch."""
    lens = [(37 * i) % 900 for i in range(120)]
    cache = make_cache(mea, lens, 1000, 8, 64, "bf16")
    q = torch.randn(120, 8, 64, generator=gen(9)).bfloat16()
    check_decode(mea, cache, q, lens, 0.125, weigh=False, bound=1000)
    check_decode(mea, cache, q, lens, 0.125, weigh=True, bound=1000)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_moving_maximum(mea, dtype):
    """Scores that climb along the rows: the running maximum is raised again and again."""
    n, K = 700, 128
    q = torch.randn(1, 2, K, generator=gen(10)).to(DT[dtype])
    k = q[:, None, :1].float() * torch.linspace(-3, 6, n).view(1, n, 1, 1)
    k = (k + 0.1 * torch.randn(1, n, 1, K, generator=gen(11))).to(DT[dtype])
    cache = mea.mea_kv4_alloc(1, n, 1, K, DT[dtype], DEV)
    mea.mea_kv4_append(k.to(DEV), rows((1, n, 1, K), dtype, 12).to(DEV), cache, i32([0]))
    check_decode(mea, cache, q, [n], K ** -0.5)


@pytest.mark.parametrize("dtype,mag", [("f16", 30000.0), ("f16", 6e-6), ("bf16", 1e30),
                                       ("bf16", 1e-30)])
def test_decode_q_of_any_size(mea, dtype, mag):
    """q near the ends of its type's range, the scale making up for it."""
    lens, K = [200, 77], 128
    cache = make_cache(mea, lens, 210, 2, K, dtype)
    q = (torch.rand(2, 4, K, generator=gen(31)) * 2 - 1)
    q = (q.abs() + 0.5 if mag in (30000.0, 1e30) else q) * (mag / 1.5)
    check_decode(mea, cache, q.to(DT[dtype]), lens, K ** -0.5 / mag)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_steps_of_many_sizes(mea, dtype):
    """Rows whose values differ by factors up to 2^16, so that the reference of the weights
    moves with the steps as well as with the scores."""
    n, K = 500, 64
    size = torch.exp2(torch.randint(-8, 9, (1, n, 1, 1), generator=gen(41)).float())
    k = torch.randn(1, n, 1, K, generator=gen(42)).to(DT[dtype])
    v = (torch.randn(1, n, 1, K, generator=gen(43)) * size).to(DT[dtype])
    v[0, 100:140] = 3.0  # steps of zero
    cache = mea.mea_kv4_alloc(1, n, 1, K, DT[dtype], DEV)
    mea.mea_kv4_append(k.to(DEV), v.to(DEV), cache, i32([0]))
    q = torch.randn(1, 3, K, generator=gen(44)).to(DT[dtype])
    check_decode(mea, cache, q, [n], K ** -0.5)


def test_decode_scale_zero_and_steps_of_zero(mea):
    cache = mea.mea_kv4_alloc(1, 50, 1, 64, torch.float16, DEV)
    k = torch.full((1, 50, 1, 64), 2.0).half()
    mea.mea_kv4_append(k.to(DEV), k.to(DEV), cache, i32([0]))
    q = torch.randn(1, 4, 64, generator=gen(1)).half()
    out, lse = check_decode(mea, cache, q, [50], 0.0, weigh=False)
    assert (out == 2.0).all()


def test_decode_nan_stays_in_its_head(mea):
    """A NaN key makes its own (sequence, kv head) NaN and no other."""
    B, n, H, K = 2, 200, 2, 64
    k = rows((B, n, H, K), "bf16", 1)
    k[0, 77, 1, 3] = math.nan
    cache = mea.mea_kv4_alloc(B, n, H, K, torch.bfloat16, DEV)
    mea.mea_kv4_append(k.to(DEV), k.to(DEV), cache, i32([0, 0]))
    q = torch.randn(B, 4, K, generator=gen(2)).bfloat16().to(DEV)
    out, lse, w = mea.mea_decode_kv4(q, cache, i32([n, n]), n, return_weights=True)
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    assert torch.isnan(w[0, 1]).all()
    assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1]).all()
    assert torch.isfinite(w[0, 0]).all() and torch.isfinite(w[1]).all()


@pytest.mark.parametrize("Hq", [4, 6])
def test_decode_nan_value_stays_in_its_group(mea, Hq):
    """A NaN among one group of V's dimensions leaves the other group's results alone, also
    while the maximum is moving."""
    n, K = 300, 128
    q = torch.randn(1, Hq, K, generator=gen(51)).bfloat16()
    k = (q[:, None, :1].float() * torch.linspace(-3, 6, n).view(1, n, 1, 1)).bfloat16()
    v = rows((1, n, 1, K), "bf16", 52)
    clean = mea.mea_kv4_alloc(1, n, 1, K, torch.bfloat16, DEV)
    mea.mea_kv4_append(k.to(DEV), v.to(DEV), clean, i32([0]))
    want, lse = mea.mea_decode_kv4(q.to(DEV), clean, i32([n]), n)
    _, (eo, el, _) = U.decode(q, [t.cpu() for t in clean], [n], K ** -0.5)
    v[0, ::7, 0, 3] = math.nan
    mea.mea_kv4_append(k.to(DEV), v.to(DEV), clean, i32([0]))
    got, lse2 = mea.mea_decode_kv4(q.to(DEV), clean, i32([n]), n)
    assert torch.isnan(got[..., :64]).all() and torch.isfinite(got[..., 64:]).all()
    # the reference may move at other rows: each side lies within its bound of the value
    assert ((got - want).double().cpu().abs() <= 2 * eo)[..., 64:].all()
    assert ((lse - lse2).double().cpu().abs() <= 2 * el).all()


def test_decode_bad_lengths_are_reported(mea):
    lens = [10, 10, 10]
    cache = make_cache(mea, lens, 20, 2, 64, "f16", spoil=False)
    q = torch.randn(3, 4, 64, generator=gen(3)).half()
    for bad, bound in (([10, -1, 10], 20), ([10, 21, 10], 30), ([10, 15, 10], 12)):
        w0 = torch.full((3, 2, 20), 3.0, device=DEV)
        out, lse, w = mea.mea_decode_kv4(q.to(DEV), cache, i32(bad), bound, weights_out=w0)
        assert mea.read_device_status() == -1
        assert (out[1] == 0).all() and torch.isnan(lse[1]).all() and (w[1] == 3.0).all()
        (ref, _, _), (eo, _, _) = U.decode(q, [t.cpu() for t in cache], [10, 0, 10], 0.125)
        for b in (0, 2):
            assert ((out[b].double().cpu() - ref[b]).abs() <= eo[b] + 2.0 ** -24).all()


def test_append_and_read_bad_ranges_are_reported(mea):
    cache = make_cache(mea, [4, 4], 8, 1, 64, "f16", spoil=False)
    x = rows((2, 3, 1, 64), "f16", 1).to(DEV)
    before = [t.clone() for t in cache]
    for past, new in (([6, -1], [3, 1]), ([0, 0], [4, -1]), ([2 ** 31 - 1, 8], [3, 1])):
        mea.mea_kv4_append(x, x, cache, i32(past), i32(new))
        assert mea.read_device_status() == -1
        assert all(torch.equal(a, b) for a, b in zip(before, cache))
    k = torch.full((2, 8, 1, 64), 5.0, dtype=torch.float16, device=DEV)
    for count, first in (([9, -1], None), ([8, 1], [1, 8]), ([1, 1], [-1, 2 ** 31 - 1])):
        mea.mea_kv4_read(cache, i32(count), None if first is None else i32(first), k_out=k,
                         v_out=torch.empty_like(k))
        assert mea.read_device_status() == -1
        assert (k == 5.0).all()


def test_offsets_past_32_bits(mea):
    """The last head of the last sequence lies beyond 2^32 bytes of codes."""
    B, H, K, cap = 2, 16, 128, 2_200_000
    lens = [5, 70]
    cache = mea.mea_kv4_alloc(B, cap, H, K, torch.bfloat16, DEV)
    x = rows((B, 70, H, K), "bf16", 1)
    past = [0, cap - 70]  # the second sequence's rows at the very end of its slot
    mea.mea_kv4_append(x.to(DEV), x.to(DEV), cache, i32(past), i32(lens))
    k, _ = mea.mea_kv4_read(cache, i32(lens), i32(past), out_rows=70)
    codes, params = U.planes(x)
    ref = U.values(codes, params).transpose(1, 2)
    assert ((k[1].double().cpu() - ref[1]).abs() <= ref[1].abs() * 2.0 ** -7 + 1e-6).all()
    mea.mea_kv4_append(x.to(DEV), x.to(DEV), cache, i32([0, 0]), i32(lens))
    q = torch.randn(B, H, K, generator=gen(2)).bfloat16()
    out, _ = mea.mea_decode_kv4(q.to(DEV), cache, i32(lens), 128)
    small = [t[:, :, :70].cpu() for t in cache]
    (want, _, _), (eo, _, _) = U.decode(q, small, lens, K ** -0.5)
    assert ((out.double().cpu() - want).abs() <= eo + 2.0 ** -24).all()


def test_other_stream_and_graph(mea):
    """The same bits on another stream and from a captured graph replayed on new inputs."""
    lens = [900, 333]
    cache = make_cache(mea, lens, 1000, 2, 128, "bf16")
    q = torch.randn(2, 8, 128, generator=gen(4)).bfloat16().to(DEV)
    st = i32(lens)
    want = mea.mea_decode_kv4(q, cache, st, 1000, return_weights=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mea.mea_decode_kv4(q, cache, st, 1000, return_weights=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    qq, sl = torch.zeros_like(q), i32([1, 1])
    new = rows((2, 1, 2, 128), "bf16", 5).to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mea.mea_kv4_append(new, new, cache, sl)
        sl.add_(1)
        res = mea.mea_decode_kv4(qq, cache, sl, 1000, return_weights=True)
    for step in range(2):  # two steps: each appends a row and attends to it
        qq.copy_(q)
        if step == 0:
            sl.copy_(st)
        graph.replay()
        torch.cuda.synchronize()
        n = [x + step + 1 for x in lens]
        ref = mea.mea_decode_kv4(q, cache, i32(n), 1000, return_weights=True)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, res))


def test_weights_in_place(mea):
    lens = [300, 40]
    cache = make_cache(mea, lens, 310, 2, 64, "f16")
    q = torch.randn(2, 4, 64, generator=gen(4)).half().to(DEV)
    w = torch.rand(2, 2, 310, generator=gen(5)).to(DEV)
    want = mea.mea_decode_kv4(q, cache, i32(lens), 300, weights=w, return_weights=True)[2]
    mea.mea_decode_kv4(q, cache, i32(lens), 300, weights=w, weights_out=w)
    assert torch.equal(want, w)


def test_read_back_feeds_a_chunk_of_prefill(mea):
    """History out of the 4-bit cache into a 16-bit one, then a chunk against it: the same
    as attention over the values the codes stand for."""
    B, H, K, hist, M = 2, 2, 64, [130, 77], 20
    cache = make_cache(mea, hist, 160, H, K, "f16")
    kc, vc = mea.mea_kv4_read(cache, i32(hist))
    k = rows((B, M, H, K), "f16", 21).to(DEV)
    v = rows((B, M, H, K), "f16", 22).to(DEV)
    q = torch.randn(B, M, 4, K, generator=gen(6)).half().to(DEV)
    out, lse = mea.mea_prefill_chunk(q, k, v, kc, vc, i32(hist))
    mea.mea_kv4_append(k, v, cache, i32(hist))
    cpu = [t.cpu() for t in cache]
    for b, n in enumerate(hist):
        for h in range(4):
            kk = torch.cat((U.values(cpu[0][b, h // 2, :n], cpu[1][b, h // 2, :n]),
                            k[b, :, h // 2].double().cpu()))
            vv = torch.cat((U.values(cpu[2][b, h // 2, :n], cpu[3][b, h // 2, :n]),
                            v[b, :, h // 2].double().cpu()))
            s = q[b, :, h].double().cpu() @ kk.T * K ** -0.5
            s = s.masked_fill(torch.arange(n + M)[None] > torch.arange(M)[:, None] + n, -math.inf)
            ref = torch.softmax(s, -1) @ vv
            # keys rounded to 16 bits (2^-11 each): scores off by |q||k| 2^-11 scale
            e = (q[b, :, h].double().cpu().abs() @ kk.abs().T).amax() * K ** -0.5 * 2.0 ** -11
            tol = 2 * math.expm1(e) * vv.abs().amax() + 2e-3 + 1e-2 * ref.abs()
            assert ((out[b, :, h].double().cpu() - ref).abs() <= tol).all()
