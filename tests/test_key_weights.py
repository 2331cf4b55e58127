"""Gathered key weights against the plain 64-bit sum (bounds derived in kv4_util)."""
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


def randn(shape, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dtype])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def plain_lse(q, k, past, new, causal, scale, alibi):
    B, M, Hq, K = q.shape
    N, G = k.shape[1], Hq // k.shape[2]
    lse = torch.zeros(B, Hq, M)
    for b in range(B):
        m = M if new is None else new[b]
        p0 = N - M if new is None else past[b]
        n = N if new is None else p0 + m
        pos, kj = torch.arange(m)[:, None] + p0, torch.arange(n)[None]
        for h in range(Hq):
            x = q[b, :m, h].double() @ k[b, :n, h // G].double().T * scale
            if alibi:
                x = x - U.slopes(Hq)[h] * (pos - kj).abs()
            if causal:
                x = x.masked_fill(kj > pos, -math.inf)
            lse[b, h, :m] = torch.logsumexp(x, -1).float()
    return lse


def check(mea, q, k, past=None, new=None, causal=True, alibi=False, scale=None, lse=None,
          weigh=True):
    B, M, Hq, K = q.shape
    N, Hkv = k.shape[1], k.shape[2]
    scale = K ** -0.5 if scale is None else scale
    if lse is None:
        lse = plain_lse(q, k, past, new, causal, scale, alibi)
    win = torch.rand(B, Hkv, N, generator=torch.Generator().manual_seed(5)) if weigh else None
    go = Guarded((B, Hkv, N), torch.float32, DEV, fill=float("nan"))
    mea.mea_key_weights(q.to(DEV), k.to(DEV), lse.to(DEV),
                        None if past is None else i32(past), None if new is None else i32(new),
                        causal=causal, scale=scale, alibi=alibi,
                        weights=win.to(DEV) if weigh else None, out=go.t)
    torch.cuda.synchronize()
    go.check("weights")
    if past is not None and new is None:
        new = [M] * B
    w, e = U.key_weights(q, k, lse, past, new, causal, scale, alibi)
    if weigh:
        for b in range(B):
            n = N if new is None else past[b] + new[b]
            w[b, :, :n] += win[b, :, :n].double()
    err = (go.t.double().cpu() - w).abs()
    assert (err <= e + w.abs() * 2.0 ** -22 + 1e-30).all(), float((err - e).max())
    return go.t


@pytest.mark.parametrize("K,dtype", [(64, "f16"), (128, "bf16"), (64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("M,N", [(128, 128), (200, 200), (17, 300), (129, 500), (300, 257),
                                 (260, 100)])
@pytest.mark.parametrize("causal", [False, True])
def test_forward_shapes(mea, K, dtype, M, N, causal):
    """Dense keys, bottom-right causal; M > N leaves rows that see nothing (lse = -inf)."""
    q, k = randn((2, M, 6, K), dtype, 1), randn((2, N, 2, K), dtype, 2)
    check(mea, q, k, causal=causal)


@pytest.mark.parametrize("K,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (5, 1), (21, 1), (32, 2)])
@pytest.mark.parametrize("M", [1, 2, 7, 16, 33, 64, 65])
def test_few_rows(mea, K, dtype, Hq, Hkv, M):
    """Decode steps and short chunks: the heads of a group share a tile."""
    past, new = [0, 5, 250, 128], [M, M - 1, M, M]
    N = 250 + M + 3
    q, k = randn((4, M, Hq, K), dtype, 3), randn((4, N, Hkv, K), dtype, 4)
    check(mea, q, k, past, new, alibi=Hq == 8)


@pytest.mark.parametrize("K,dtype,causal,alibi", [(64, "bf16", True, True), (128, "f16", False, True),
                                                  (128, "bf16", True, False)])
def test_ragged_chunks(mea, K, dtype, causal, alibi):
    """Padded chunks after different histories; padded rows hold NaN and count for nothing."""
    past, new = [0, 100, 257, 0], [140, 0, 33, 1]
    q, k = randn((4, 140, 4, K), dtype, 5), randn((4, 300, 2, K), dtype, 6)
    lse = plain_lse(q, k, past, new, causal, K ** -0.5, alibi)
    for b in range(4):
        q[b, new[b]:] = math.nan
        lse[b, :, new[b]:] = math.nan
        k[b, past[b] + new[b]:] = math.nan
    q2, k2 = q.clone(), k.clone()
    got = check(mea, q2, k2, past, new, causal, alibi, lse=lse)
    for b in range(4):
        assert (got[b, :, past[b] + new[b]:] == 0).all()
    check(mea, randn((4, 140, 4, K), dtype, 5), randn((4, 400, 2, K), dtype, 6), [0, 100, 257, 3],
          None, causal, alibi)


def test_many_steps(mea):
    """More tiles than stages and buffers, heads and row blocks together."""
    q, k = randn((1, 1000, 10, 128), "bf16", 7), randn((1, 1100, 2, 128), "bf16", 8)
    check(mea, q, k, [100], [1000])
    check(mea, q, k, causal=False, weigh=False)


@pytest.mark.parametrize("K,dtype,Hq,Hkv,M,N", [(128, "bf16", 16, 1, 700, 600), (64, "f16", 4, 1, 600, 300),
                                                (128, "f16", 9, 1, 260, 900), (64, "bf16", 3, 3, 515, 515)])
@pytest.mark.parametrize("causal", [False, True])
def test_few_key_blocks(mea, K, dtype, Hq, Hkv, M, N, causal):
    """Too few key blocks to fill the GPU: clusters share each block's queries."""
    q, k = randn((1, M, Hq, K), dtype, 21), randn((1, N, Hkv, K), dtype, 22)
    a = check(mea, q, k, causal=causal, alibi=Hkv == 3)
    b = check(mea, q, k, causal=causal, alibi=Hkv == 3)
    assert torch.equal(a, b)


def test_weights_add_up_to_the_rows(mea):
    """A softmax's weights sum to one: with mea_fwd's own lse the keys gather M per head."""
    q, k = randn((2, 513, 8, 64), "f16", 9).to(DEV), randn((2, 700, 2, 64), "f16", 10).to(DEV)
    v = torch.randn_like(k)
    for bias in ("none", "causal"):
        _, lse = mea.mea_fwd(q, k, v, bias=bias)
        w = mea.mea_key_weights(q, k, lse, causal=bias == "causal")
        assert ((w.double().sum(-1) - 513 * 4).abs() <= 513 * 4 * 1e-3).all()  # lse within 1e-3


def test_strided_and_in_place(mea):
    """[B, H, M, K] storage; adding into the weights themselves; equal bits every time."""
    q = randn((2, 4, 300, 64), "bf16", 11).to(DEV).transpose(1, 2)
    k = randn((2, 2, 300, 64), "bf16", 12).to(DEV).transpose(1, 2)
    lse = plain_lse(q.cpu(), k.cpu(), None, None, True, 0.125, False).to(DEV)
    w = torch.rand(2, 2, 300, device=DEV)
    want = mea.mea_key_weights(q, k, lse, weights=w)
    want2 = mea.mea_key_weights(q.contiguous(), k.contiguous(), lse, weights=w)
    mea.mea_key_weights(q, k, lse, weights=w, out=w)
    assert torch.equal(w, want) and torch.equal(want, want2)


@pytest.mark.parametrize("M", [1, 140])
def test_lse_of_minus_infinity_and_nan(mea, M):
    q, k = randn((1, M, 2, 64), "f16", 13), randn((1, 200, 2, 64), "f16", 14)
    lse = plain_lse(q, k, [200 - M], [M], True, 0.125, False)
    lse[0, 0] = -math.inf
    w = mea.mea_key_weights(q.to(DEV), k.to(DEV), lse.to(DEV), i32([200 - M]))
    assert (w[0, 0] == 0).all() and torch.isfinite(w).all() and (w[0, 1] > 0).any()
    lse[0, 1, -1] = math.nan
    w = mea.mea_key_weights(q.to(DEV), k.to(DEV), lse.to(DEV), i32([200 - M]))
    assert (w[0, 0] == 0).all() and torch.isnan(w[0, 1]).all()


@pytest.mark.parametrize("M", [4, 64])
def test_bad_lengths_are_reported(mea, M):
    q, k = randn((2, M, 2, 64), "f16", 15).to(DEV), randn((2, 100, 2, 64), "f16", 16).to(DEV)
    lse = torch.zeros(2, 2, M, device=DEV)
    for past, new in (([0, -1], [1, 1]), ([0, 100], [1, 1]), ([0, 0], [1, M + 1]),
                      ([0, 0], [1, -1]), ([0, 2 ** 31 - 1], [1, M])):
        w = torch.full((2, 2, 100), 3.0, device=DEV)
        mea.mea_key_weights(q, k, lse, i32(past), i32(new), out=w)
        assert mea.read_device_status() == -1
        assert (w[1] == 3.0).all() and (w[0, :, 1:] == 0).all()


def test_graph_and_stream(mea):
    q, k = randn((1, 260, 4, 128), "bf16", 17).to(DEV), randn((1, 400, 2, 128), "bf16", 18).to(DEV)
    lse = plain_lse(q.cpu(), k.cpu(), [140], [260], True, 128 ** -0.5, False).to(DEV)
    past = i32([140])
    want = mea.mea_key_weights(q, k, lse, past)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mea.mea_key_weights(q, k, lse, past, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    acc = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mea.mea_key_weights(q, k, lse, past, weights=acc, out=acc)
    acc.zero_()
    graph.replay()
    assert torch.equal(acc, want)
