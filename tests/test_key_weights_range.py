"""Gathered key weights where rows take no weight whatever they hold, at the ends of the
exponential's range, and with sums of many terms."""
import math

import pytest
import torch

import kv4_util as U
from test_key_weights import check, plain_lse
from test_key_weights import randn as host_randn

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


def randn(shape, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dtype]).to(DEV)


@pytest.mark.parametrize("K,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("M", [3, 40, 256, 300])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_without_weight_may_hold_anything(mea, K, dtype, M, causal):
    """Rows with lse = -inf (padding, say) add nothing, whether q is a number there, a NaN or
    an infinity: the same bits as with zeros."""
    q, k = randn((2, M, 4, K), dtype, 1), randn((2, 400, 2, K), dtype, 2)
    lse = 5.0 + torch.rand(2, 4, M, generator=torch.Generator().manual_seed(3)).to(DEV)
    pad = torch.zeros(2, M, dtype=torch.bool, device=DEV)
    pad[0, M // 2:] = True
    pad[1, 1] = True
    lse.masked_fill_(pad[:, None], -math.inf)
    want = mea.mea_key_weights(q.masked_fill(pad[:, :, None, None], 0.0), k, lse, causal=causal)
    assert torch.isfinite(want).all() and (want > 0).any()
    for x in (math.nan, math.inf, -math.inf):
        got = mea.mea_key_weights(q.masked_fill(pad[:, :, None, None], x), k, lse, causal=causal)
        assert torch.equal(got, want)


POWERS = [-300.0, -127.4, -126.6, -126.2, -125.9, -100.3, -1.5, -0.5, 0.0, 0.4999, 0.5, 0.7, 64.3, 126.4,
          126.6, 127.3, 127.7, 128.4, 200.0, math.inf, -math.inf, math.nan]


@pytest.mark.parametrize("K,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("M", [1, 256])
def test_the_exponential_over_its_range(mea, K, dtype, M):
    """One row's weight 2^x at every place of a tile (each takes one of two exponentials), all
    other rows' at 2^-300.  Below the normal range the result may be 0; between 127.5 and 128
    it may be infinite."""
    H = min(M, 64)
    x = torch.tensor(POWERS, dtype=torch.float64)
    q = torch.zeros(len(POWERS), M, H, K, dtype=DT[dtype], device=DEV)
    k = torch.zeros(len(POWERS), 256, H, K, dtype=DT[dtype], device=DEV)
    lse = torch.full((len(POWERS), H, M), 300.0 * math.log(2))
    for h in range(H):
        lse[:, h, h * M // H] = (-x * math.log(2)).float()
    w = mea.mea_key_weights(q, k, lse.to(DEV), causal=False).double().cpu()
    for i, p in enumerate(POWERS):
        exact = torch.exp(-lse[i, 0, 0].double())  # of the lse that fp32 holds
        if math.isnan(p):
            assert torch.isnan(w[i]).all()
        elif p == math.inf:  # lse = -inf: a row without weight
            assert (w[i] == 0).all()
        elif exact >= 2.0 ** 128:
            assert torch.isposinf(w[i]).all(), p
        else:
            # -lse log2(e) in fp32 (two roundings), exp2's 2^-21, and the subnormals
            tol = exact * ((abs(p) + 1) * 2.0 ** -23 + 2.0 ** -21)
            tol = tol if exact > 2.0 ** -125.5 else 2.0 ** -125.5
            ok = (w[i] - exact).abs() <= tol
            if exact > 2.0 ** 127.4:
                ok |= torch.isposinf(w[i])
            assert ok.all(), (p, w[i].min(), w[i].max(), exact)


@pytest.mark.parametrize("K,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("lse", [0.1, 2.0, 7.7])
def test_sums_of_many_equal_terms(mea, K, dtype, lse):
    """32768 equal weights a key: sums of 64 within a tile, then one term a tile and joined
    parts: 64 + 128 + 8 additions of 2^-24 in a row at most, beside each weight's own
    -lse log2(e) and exp2."""
    M, G = 8192, 4
    for N, H in ((4096, 10), (128, 1)):  # a CTA a key block, and clusters that share one
        q = torch.zeros(1, M, G * H, K, dtype=DT[dtype], device=DEV)
        k = torch.zeros(1, N, H, K, dtype=DT[dtype], device=DEV)
        w = mea.mea_key_weights(q, k, torch.full((1, G * H, M), lse, device=DEV), causal=False)
        exact = M * G * math.exp(-float(torch.tensor(lse)))
        tol = exact * (200 * 2.0 ** -24 + (1.5 * lse + 1) * 2.0 ** -23 + 2.0 ** -21)
        assert ((w.double() - exact).abs() <= tol).all(), (w.double() / exact - 1).abs().max()


@pytest.mark.parametrize("K,dtype,rows", [
    (128, "bf16", [(1, 127), (1, 128), (2, 88), (2, 89), (8, 22), (8, 23), (44, 4), (177, 1)]),
    (64, "f16", [(1, 127), (2, 127), (3, 112), (4, 84), (4, 85), (16, 21), (16, 22), (337, 1)])])
@pytest.mark.parametrize("alibi", [False, True])
def test_both_sides_of_the_few_row_rule(mea, K, dtype, rows, alibi):
    """(heads a kv head, rows) at the last size of one kernel and the first of the other."""
    for G, M in rows:
        q, k = host_randn((2, M, G, K), dtype, 41), host_randn((2, 200 + M, 1, K), dtype, 42)
        check(mea, q, k, [200, 7], [M, M - 1], alibi=alibi)


@pytest.mark.parametrize("K,dtype,M,N,Hq,Hkv,causal", [
    (128, "bf16", 700, 700, 8, 2, True), (64, "f16", 515, 600, 4, 4, False),
    (128, "f16", 16, 900, 8, 2, True), (64, "bf16", 1500, 300, 6, 1, False)])
def test_norm_of_the_error(mea, K, dtype, M, N, Hq, Hkv, causal):
    """Relative error in norm.  A product q.k is summed 16 terms at a time, each partial sum
    (at most 64 for these inputs) cut at 2^-24 of itself: K/16 64 2^-23 / sqrt(K), 5.4e-6 at
    K = 128; the score's scaling against lse, 2 x 2^-24 of 20; exp2 2^-21.  2^-16 holds them."""
    q, k = host_randn((2, M, Hq, K), dtype, 51), host_randn((2, N, Hkv, K), dtype, 52)
    lse = plain_lse(q, k, None, None, causal, K ** -0.5, False)
    got = mea.mea_key_weights(q.to(DEV), k.to(DEV), lse.to(DEV), causal=causal).double().cpu()
    want, _ = U.key_weights(q, k, lse, None, None, causal, K ** -0.5)
    assert float((got - want).norm() / want.norm()) <= 2.0 ** -16
