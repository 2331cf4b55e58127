"""A 16-bit cache that has been evicted goes on being attended to and appended to: its slots of
unequal lengths are mea_prefill_chunk's, a decode step is a chunk of one row."""
import pytest
import torch

import kv4_util as U
from parity_util import assert_lse_close, assert_out_close

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("K,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_prompt_evict_decode(K, dtype, in_place):
    """Prompts of unequal lengths, their keys weighed, cut to the budget; then steps that
    append, attend and weigh, cut again in place when the slots are full."""
    import memory_efficient_exact_mea_b200 as mea

    B, M, Hq, Hkv, budget, recent, cap = 3, 150, 6, 2, 64, 9, 70
    g = torch.Generator().manual_seed(7)
    new = [150, 64, 31]
    mk = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    q, k, v = mk(B, M, Hq, K), mk(B, M, Hkv, K), mk(B, M, Hkv, K)
    kc, vc = mk(B, M if in_place else M + 3, Hkv, K), mk(B, M if in_place else M + 3, Hkv, K)
    mea.read_device_status()
    zero, n = i32([0] * B), i32(new)
    _, lse = mea.mea_prefill_chunk(q, k, v, kc, vc, zero, n)
    w = mea.mea_key_weights(q, kc, lse, zero, n)
    host = [[[t[b, :m].double().cpu() for b, m in enumerate(new)] for t in (k, v)]][0]
    wh = w.cpu()
    rows = [[U.choose(wh[b, h], new[b], budget, recent) for h in range(Hkv)] for b in range(B)]
    if in_place:
        n, _, w = mea.mea_cache_evict((kc, vc), w, n, budget, recent)
    else:
        small = (torch.zeros(B, cap, Hkv, K, dtype=dtype, device=DEV) for _ in range(2))
        small = tuple(small)
        n, _, w = mea.mea_cache_evict((kc, vc), w, n, budget, recent, out=small)
        kc, vc = small
    # what each (sequence, head) now holds, in 64 bits
    keep = [[[host[t][b][rows[b][h], h] for h in range(Hkv)] for b in range(B)] for t in range(2)]
    for step in range(9):
        if int(n.max()) == cap:
            wh, lens = w.cpu(), n.tolist()
            n, _, w = mea.mea_cache_evict((kc, vc), w, n, budget, recent)
            for b in range(B):
                for h in range(Hkv):
                    at = U.choose(wh[b, h], lens[b], budget, recent)
                    for t in range(2):
                        keep[t][b][h] = keep[t][b][h][at]
        q1, k1, v1 = mk(B, 1, Hq, K), mk(B, 1, Hkv, K), mk(B, 1, Hkv, K)
        out, lse = mea.mea_prefill_chunk(q1, k1, v1, kc, vc, n)
        w = mea.mea_key_weights(q1, kc, lse, n, weights=w, out=w)
        n = n + 1
        ref, ref_lse = torch.zeros(B, Hq, K, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
        for b in range(B):
            for h in range(Hkv):
                for t, x in ((0, k1), (1, v1)):
                    keep[t][b][h] = torch.cat((keep[t][b][h], x[b, :, h].double().cpu()))
            for hq in range(Hq):
                h = hq // (Hq // Hkv)
                s = keep[0][b][h] @ q1[b, 0, hq].double().cpu() * K ** -0.5
                ref_lse[b, hq] = torch.logsumexp(s, 0)
                ref[b, hq] = torch.softmax(s, 0) @ keep[1][b][h]
        assert n.tolist() == [len(keep[0][b][0]) for b in range(B)]
        assert_out_close(out[:, 0], ref, f"step {step}")
        assert_lse_close(lse[..., 0], ref_lse, f"step {step}")
    assert mea.read_device_status() == 0
