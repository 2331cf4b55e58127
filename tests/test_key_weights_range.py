"""Gathered key weights where rows take no weight whatever they hold, at the ends of the
exponential's range, and with sums of many terms."""
import math

import pytest
import torch

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
