"""The 4-bit decode over its whole range of values: groups of very different size, values
near the ends of the type, and every row's place in the result (bounds in kv4_bounds)."""
import math
from fractions import Fraction

import pytest
import torch

import kv4_util as U
from kv4_bounds import decode_bound

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


def randn(shape, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def filled(mea, k, v, lens):
    """A 4-bit cache that holds rows k, v [B, n, Hkv, K]."""
    B, n, Hkv, K = k.shape
    cache = mea.mea_kv4_alloc(B, n, Hkv, K, k.dtype, DEV)
    mea.mea_kv4_append(k.to(DEV), v.to(DEV), cache, i32([0] * B), i32(lens))
    return cache


def check(mea, q, k, v, lens, scale, alibi=False):
    cache = filled(mea, k, v, lens)
    out, lse = mea.mea_decode_kv4(q.to(DEV), cache, i32(lens), max(lens), scale=scale, alibi=alibi)
    (ro, rl), (eo, el) = decode_bound(q, [t.cpu() for t in cache], lens, scale, alibi)
    err = (out.double().cpu() - ro).abs()
    assert torch.isfinite(out).all()
    assert (err <= eo).all(), float((err / eo).max())
    fin = ~torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse.cpu()), ~fin)
    assert ((lse.double().cpu() - rl).abs()[fin] <= el[fin]).all()
    return out, cache


SIZES = [("bf16", 1.0, 1e-3), ("bf16", 1e-5, 1.0), ("bf16", 1.0, 1e-6), ("bf16", 1.0, 1e-8),
         ("bf16", 1e30, 1e-30), ("bf16", 1e-23, 1e-23), ("bf16", 1e-25, 1e-25), ("bf16", 1e-32, 1.0),
         ("bf16", 1e37, 1e37), ("f16", 1e4, 1e-3), ("f16", 1e-3, 1e4), ("f16", 1e-4, 1e-4),
         ("f16", 1e4, 1e4)]


@pytest.mark.parametrize("dtype,a,b", SIZES)
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (6, 2), (6, 1), (9, 1)])
@pytest.mark.parametrize("even", [True, False])
def test_groups_of_any_size(mea, dtype, a, b, Hq, Hkv, even):
    """Each group of 64 dimensions keeps its bits, whatever the other's size.  Equal weights
    (scale 0) leave the values alone to be seen."""
    n, K = 300, 128
    v = randn((2, n, Hkv, K), 1) * torch.tensor([a, b]).repeat_interleave(64)
    k, q = randn((2, n, Hkv, K), 2).to(DT[dtype]), randn((2, Hq, K), 3).to(DT[dtype])
    check(mea, q, k, v.to(DT[dtype]), [n, 37], 0.0 if even else K ** -0.5)


@pytest.mark.parametrize("dtype,K", [("bf16", 64), ("bf16", 128), ("f16", 128)])
def test_rows_of_any_size(mea, dtype, K):
    """Rows whose sizes climb and fall by powers of two, against scores that do the reverse:
    the reference of the scores and the factor of the values move apart."""
    n = 900
    size = torch.exp2(12 * torch.sin(torch.arange(n) / 70.0)).view(1, n, 1, 1)
    v = (randn((1, n, 1, K), 4) * size).to(DT[dtype])
    q = randn((1, 3, K), 5)
    k = q[:, None, :1] * (-torch.log2(size) * 0.6) / q[0, 0].square().sum() * K ** 0.5
    k = (k + 0.05 * randn((1, n, 1, K), 6)).to(DT[dtype])
    check(mea, q.to(DT[dtype]), k, v, [n], K ** -0.5)
    check(mea, q.to(DT[dtype]), k, v, [n], K ** -0.5, alibi=True)


@pytest.mark.parametrize("K,Hq", [(64, 2), (128, 2), (128, 6)])
@pytest.mark.parametrize("z", [1e21, -3e38, 1e-30])
def test_equal_values_after_zeros(mea, K, Hq, z):
    """Rows of zeros (step and zero both 0), then rows of one large value each."""
    n = 300
    v = torch.zeros(1, n, 1, K)
    v[:, 140:] = z
    k, q = 0.1 * randn((1, n, 1, K), 7), randn((1, Hq, K), 8)
    check(mea, q.bfloat16(), k.bfloat16(), v.bfloat16(), [n], K ** -0.5)


@pytest.mark.parametrize("dtype,mag", [("bf16", 1e33), ("bf16", 1e37), ("bf16", 1e-30),
                                       ("bf16", 1e-36), ("f16", 1e4), ("f16", 1e-4)])
@pytest.mark.parametrize("K,Hq", [(64, 2), (128, 3), (128, 6)])
def test_keys_of_any_size(mea, dtype, mag, K, Hq):
    """Keys near the ends of the type's range, q making up for it."""
    n = 333
    k, q = randn((2, n, 1, K), 21) * mag, randn((2, Hq, K), 22) / mag
    v = randn((2, n, 1, K), 23)
    check(mea, q.to(DT[dtype]), k.to(DT[dtype]), v.to(DT[dtype]), [n, 60], K ** -0.5)
    check(mea, q.to(DT[dtype]), k.to(DT[dtype]), v.to(DT[dtype]), [n, 60], K ** -0.5, alibi=True)


@pytest.mark.parametrize("K,Hq", [(64, 2), (128, 3), (128, 6)])
def test_a_huge_query_leaves_the_other_heads_alone(mea, K, Hq):
    n = 200
    q, k, v = randn((1, Hq, K), 24), randn((1, n, 1, K), 25), randn((1, n, 1, K), 26)
    q[:, 0] *= 1e35
    q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
    cache = filled(mea, k, v, [n])
    out, lse = mea.mea_decode_kv4(q.to(DEV), cache, i32([n]), n)
    (ro, rl), (eo, el) = decode_bound(q, [t.cpu() for t in cache], [n], K ** -0.5)
    assert ((out.double().cpu() - ro).abs() <= eo)[:, 1:].all()
    assert ((lse.double().cpu() - rl).abs() <= el)[:, 1:].all()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype,mag", [("f16", 3e2), ("f16", 6e4), ("bf16", 1e9), ("bf16", 1e15)])
@pytest.mark.parametrize("K,Hq", [(64, 2), (128, 3), (128, 6)])
@pytest.mark.parametrize("alibi", [False, True])
def test_scores_of_any_size(mea, dtype, mag, K, Hq, alibi):
    """Scores far beyond 2^24: the largest takes all the weight."""
    n = 300
    k, v = randn((1, n, 1, K), 27), randn((1, n, 1, K), 28)
    k[:, 177] = 4.0 * randn((K,), 29).sign()
    q = k[:, None, 177, 0] * torch.linspace(1, 2, Hq).view(1, Hq, 1) / 8
    k, q = (k * mag / 4).to(DT[dtype]), (q * mag).to(DT[dtype]).squeeze(1)
    cache = filled(mea, k, v.to(DT[dtype]), [n])
    out, lse = mea.mea_decode_kv4(q.to(DEV), cache, i32([n]), n, alibi=alibi)
    (ro, rl), _ = decode_bound(q, [t.cpu() for t in cache], [n], K ** -0.5, alibi)
    # the row's own values, one rounding; the scores' relative error for the lse
    half, held = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype], 2.0 ** -21
    row = mea.mea_kv4_read(cache, i32([n]))[1][0, 177, 0].double().cpu()
    assert ((ro[0] - row).abs() <= row.abs() * half + 2.0 ** -25).all()
    mag_v = cache.v_params[0, 0, 177].double().abs().cpu() @ torch.tensor([15.0, 1.0]).double()
    tol = ro.abs() * half + mag_v.repeat_interleave(64) * (held + 2.0 ** -20)
    assert ((out.double().cpu() - ro).abs() <= tol).all()
    assert ((lse.double().cpu() - rl).abs() <= rl.abs() * K * 2.0 ** -21).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K,Hq", [(64, 2), (128, 2), (128, 6)])
def test_equal_rows_give_that_row(mea, dtype, K, Hq):
    """Rows of -8 .. 7 (step 1, zero -8, exact) at two scores whose weights are no short
    numbers: the weights' bits cancel between the codes' sum and the zeros'."""
    n = 40
    v = (torch.arange(K) % 16 - 8.0).expand(1, n, 1, K)
    q = randn((1, Hq, K), 31)
    k = torch.zeros(1, n, 1, K)
    k[:, 5] = q[:, :1] * 0.3
    check(mea, q.to(DT[dtype]), k.to(DT[dtype]), v.to(DT[dtype]), [n], K ** -0.5)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_the_largest_numbers_stay_finite(mea, dtype):
    """Groups that reach the type's largest number: z + 15 s passes it by the step's rounding,
    and is held to it, read back or attended to; groups with a NaN or infinity stay NaN."""
    dt = DT[dtype]
    top = torch.finfo(dt).max
    x = torch.zeros(8, 64)
    x[0, 7] = top
    x[1, 0], x[1, 1] = top, -top
    x[2, 5] = -top
    x[3] = top * (torch.arange(64) / 63.0)
    x[4] = top * (torch.arange(64) / 31.5 - 1.0)
    x[5, 9], x[6, 9], x[7, 9] = math.inf, -math.inf, math.nan
    x = x.to(dt).reshape(8, 1, 1, 64).repeat(1, 1, 1, 2)
    cache = filled(mea, x, x, [1] * 8)
    want = U.values(*[t.cpu() for t in cache[:2]]).transpose(1, 2).clamp(-top, top)
    k, v = mea.mea_kv4_read(cache, i32([1] * 8))
    q = torch.zeros(8, 2, 128).to(dt).to(DEV)
    out, _ = mea.mea_decode_kv4(q, cache, i32([1] * 8), 1)
    out6, _ = mea.mea_decode_kv4(torch.zeros(8, 6, 128, dtype=dt, device=DEV), cache, i32([1] * 8), 1)
    for got in (k, v, out[:, :1, None], out[:, 1:, None], out6[:, 5:, None]):
        got = got.reshape(8, 1, 1, 128).double().cpu()
        assert torch.isnan(got[5:]).all() and torch.isfinite(got[:5]).all()
        tol = want.abs() * (U.HALF[dt] + 2.0 ** -20)
        assert ((got - want).abs() <= tol)[:5].all()
    # the listed top itself comes back
    assert (k[0, 0, 0, 7] == top).item() and (k[1, 0, 0, 0] == top).item()


@pytest.mark.parametrize("dtype,step", [("bf16", 101), ("bf16", 110), ("bf16", 20), ("bf16", -101),
                                        ("bf16", -118), ("f16", 2), ("f16", -5)])
@pytest.mark.parametrize("least", [-1.0, 0.0, 1.0])
def test_codes_beside_a_tie(mea, dtype, step, least):
    """Values at halves of steps above zero, the group's least value a hair off zero (so far
    below them that a difference of the two may round it away): fractions decide the codes."""
    dt = DT[dtype]
    hair = torch.finfo(dt).smallest_normal if step > 0 else torch.finfo(dt).tiny / 64
    s = 2.0 ** step
    x = torch.tensor([least * hair] + [s * i / 2 for i in range(31)] + [s * 15.0] * 32)
    x = x.clamp_min(least * hair).to(dt)
    cache = filled(mea, *[x.view(1, 1, 1, 64)] * 2, [1])
    param = cache.k_params[0, 0, 0, 0].double().tolist()
    fs, fz = Fraction(param[0]), Fraction(param[1])
    assert fs == Fraction(s) and fz == Fraction(float(x.double().min()))
    want = [min(15, max(0, round((Fraction(float(t)) - fz) / fs))) for t in x.double()]  # ties to even
    got = cache.k_codes[0, 0, 0].cpu()
    assert torch.stack((got & 15, got >> 4), -1).flatten().tolist() == want


PROBES = [0, 1, 31, 32, 33, 127, 128, 129, 255, 256, 1000, 1535, 1536, 1537, 2047, 2048, 4095, 4096,
          4498, 4499]


@pytest.mark.parametrize("K,dtype,Hq,copies", [(128, "bf16", 4, 1), (128, "f16", 6, 1),
                                               (64, "f16", 2, 1), (64, "bf16", 2, 30)])
def test_one_row_at_a_time(mea, K, dtype, Hq, copies):
    """A key that takes all the weight at each of many rows (copies: enough sequences for the
    longest splits): the result is that row's values, the others' weight below e^-40."""
    n, B = 4500, len(PROBES) * copies
    k, v = 0.1 * randn((1, n, 1, K), 9), randn((1, n, 1, K), 10)
    q = randn((1, Hq, K), 11).sign() + 0.25 * randn((1, Hq, K), 12)
    base = filled(mea, k.to(DT[dtype]), v.to(DT[dtype]), [n])
    cache = mea.Kv4Cache(*(t.repeat(B, *[1] * (t.dim() - 1)).contiguous() for t in base))
    key = q[:, None, :1] * 8  # scores 8 |q|^2 / sqrt(K) >= 60 for head 0
    rows = (PROBES * copies)[:B]
    for t in (0, 1):
        spot = filled(mea, key.to(DT[dtype]), key.to(DT[dtype]), [1])[t]
        for b, r in enumerate(rows):
            cache[t][b, :, r] = spot[0, :, 0]
    qd = q.to(DT[dtype]).repeat(B, 1, 1)
    out, lse = mea.mea_decode_kv4(qd.to(DEV), cache, i32([n] * B), n)
    few = mea.Kv4Cache(*(t[:len(PROBES)] for t in cache))
    (ro, rl), (eo, el) = decode_bound(qd[:len(PROBES), :1].contiguous(), [t.cpu() for t in few],
                                      [n] * len(PROBES), K ** -0.5)
    k16, v16 = mea.mea_kv4_read(base, i32([n]))
    for i, r in enumerate(PROBES):  # the oracle itself says that this row is the answer
        assert ((ro[i, 0] - v16[0, r, 0].double().cpu()).abs() <= 2.0 ** -7 * 8).all()
    for c in range(copies):
        at = slice(c * len(PROBES), (c + 1) * len(PROBES))
        assert ((out[at, :1].double().cpu() - ro).abs() <= eo).all()
        assert ((lse[at, :1].double().cpu() - rl).abs() <= el).all()


@pytest.mark.parametrize("K,dtype,Hq,B", [(128, "bf16", 4, 2), (128, "f16", 8, 2), (64, "bf16", 3, 2),
                                          (64, "f16", 4, 160)])
@pytest.mark.parametrize("n", [4500, 4481, 1536, 129, 33])
def test_every_row_counts_once(mea, K, dtype, Hq, B, n):
    """Equal weights, values that are zero but in a few rows -- the last one, the last tile,
    the edges of tiles, warps and splits: each such row adds 1/n of its values."""
    v = torch.zeros(1, n, 1, K)
    rows = sorted({r for r in (0, 31, 32, 127, 128, 1535, 1536, n - 32, n - 2, n - 1) if r < n})
    v[0, rows, 0] = randn((len(rows), K), 13)
    k, q = randn((1, n, 1, K), 14).to(DT[dtype]), randn((1, Hq, K), 15).to(DT[dtype])
    base = filled(mea, k, v.to(DT[dtype]), [n])
    cache = mea.Kv4Cache(*(t.repeat(B, *[1] * (t.dim() - 1)).contiguous() for t in base))
    out, _ = mea.mea_decode_kv4(q.repeat(B, 1, 1).to(DEV), cache, i32([n] * B), n, scale=0.0)
    (ro, _), (eo, _) = decode_bound(q, [t.cpu() for t in base], [n], 0.0)
    assert ((out.double().cpu() - ro).abs() <= eo).all()
    assert (ro.abs() > 8 * eo).double().mean() > 0.5  # a lost row would show


@pytest.mark.parametrize("K,dtype,Hq,Hkv,lens", [
    (128, "bf16", 8, 2, [4500, 1, 1023]), (128, "f16", 8, 1, [3000, 77]), (64, "f16", 6, 2, [2500]),
    (64, "bf16", 20, 1, [700])])
@pytest.mark.parametrize("alibi", [False, True])
def test_close_bound(mea, K, dtype, Hq, Hkv, lens, alibi):
    """Ordinary inputs within the closer bound."""
    n, B = max(lens), len(lens)
    k, v = randn((B, n, Hkv, K), 16), randn((B, n, Hkv, K), 17)
    k[..., ::37] += 4.0
    q = randn((B, Hq, K), 18)
    check(mea, q.to(DT[dtype]), k.to(DT[dtype]), v.to(DT[dtype]), lens, K ** -0.5, alibi)
