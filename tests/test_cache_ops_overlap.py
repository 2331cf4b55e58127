"""Where the cache operators' outputs may lie: two rows of outputs in one place, or an output
over an input, is refused on the host; interleaved rows of one array are not."""
import pytest
import torch

import kv4_util as U
import memory_efficient_exact_mea_b200 as m
from test_cache_ops_host import APPEND, DECODE, I64, INVALID, P, READ, WEIGH, call, evict

M24, M25 = 1 << 24, 1 << 25


# evict(): sources [2, 10, 2] rows of 16 bytes at 1 << 24 (strides 320, 32, 16), destinations
# [2, 6, 2] at 1 << 25 (192, 32, 16), weights 1 << 20 -> 2 << 20, lens 16, new 64, kept 4096
@pytest.mark.parametrize("kw", [
    dict(n=2, dst=M25 + 1024 + 32),                       # one row on from the other plane
    dict(n=2, dst=M25 + 1024 + 16),                       # one head on
    dict(n=2, dst=M25 + 1024 + 192),                      # one sequence on
    dict(n=2, dst=M25 + 1024 - 176),                      # the last row over the other's first
    dict(dst_strides=I64(192, 32, 0)), dict(dst_strides=I64(192, 0, 16)),
    dict(dst_strides=I64(0, 32, 16)),                     # rows of one plane in one place
    dict(dst_strides=I64(192, 32, 12)), dict(dst_strides=I64(188, 32, 16)),
    dict(dst_strides=I64(96, 16, 96)),                    # heads over sequences
    dict(n=2, dst=M25 + 1024, dst_strides=I64(192, 16, 96)),  # the same bytes in another order
    dict(kept=P(M25 + 8)), dict(kept=P(M24 + 8)), dict(kept=P(64)), dict(kept=P(16)),
    dict(kept=P(1 << 20)), dict(kept=P(2 << 20)),
    dict(new=P(20)), dict(new=P(12)), dict(new=P(M25)), dict(new=P(M24)), dict(new=P(1 << 20)),
    dict(lens=P(M25 + 4)), dict(lens=P(2 << 20)),
])
def test_evict(kw):
    assert evict(**kw) == INVALID


def test_evict_in_place():
    """Two planes of one array, cut in place, a row or a head apart."""
    for off in (32, 16, 8, 0):
        p = (m._Plane * 2)()
        for i in range(2):
            at = M24 + i * off
            p[i] = m._Plane(at, at, I64(320, 32, 16), I64(320, 32, 16), 16)
        assert m.lib.mea_cache_evict(p, 2, P(1 << 20), P(1 << 20), P(16), P(64), P(4096), 2, 2, 10,
                                     10, 5, 1, None) == INVALID


@pytest.mark.parametrize("fn,base,kw", [
    ("mea_kv4_append", APPEND, dict()),                   # all planes at one address
    ("mea_kv4_append", APPEND, dict(kc=P(M24), kp=P(M25), vc=P(M24 + 512), vp=P(1 << 26))),
    ("mea_kv4_append", APPEND, dict(kc=P(M24), kp=P(M24 + 624), vc=P(M25), vp=P(1 << 26))),
    ("mea_kv4_append", APPEND, dict(kc=P(M24), kp=P(M25), vc=P(1 << 26), vp=P(M25 + 64))),
    # rows [2, 5, 1] of 128 bytes
    ("mea_kv4_read", READ, dict()),
    ("mea_kv4_read", READ, dict(k=P(M24), v=P(M24 + 128))),
    ("mea_kv4_read", READ, dict(k=P(M24), v=P(M24 + 2048))),
    ("mea_kv4_read", READ, dict(k=P(M24), v=P(M24 + 16))),
    ("mea_kv4_read", READ, dict(k=P(M24), v=P(M25), ks=I64(1024, 32, 64))),
    ("mea_kv4_read", READ, dict(k=P(M24), v=P(M25), vs=I64(64, 64, 64))),
    # weights [2, 2, 100] and [2, 2, 9]
    ("mea_decode_kv4", DECODE, dict(win=P(M24), wout=P(M24 + 4))),
    ("mea_decode_kv4", DECODE, dict(win=P(M24 + 1596), wout=P(M24))),
    ("mea_key_weights", WEIGH, dict(win=P(M24), wout=P(M24 + 140))),
    ("mea_key_weights", WEIGH, dict(win=P(M24 + 36), wout=P(M24))),
])
def test_others(fn, base, kw):
    assert call(getattr(m.lib, fn), base, **kw) == INVALID


VIEWS = {  # [B, rows, H, K] views of one array for keys and values, side by side
    "rows": lambda B, R, H, K, new: new(B, R, H, 2, K).unbind(3),
    "heads": lambda B, R, H, K, new: new(B, R, 2, H, K).unbind(2),
    "sequences": lambda B, R, H, K, new: new(B, 2, R, H, K).unbind(1),
    "planes": lambda B, R, H, K, new: new(2, B, R, H, K).unbind(0),
    "head major": lambda B, R, H, K, new: [t.transpose(1, 2) for t in new(B, H, R, 2, K).unbind(3)],
    "head blocks": lambda B, R, H, K, new: [t.transpose(1, 2) for t in new(B, H, 2, R, K).unbind(2)],
    "padded": lambda B, R, H, K, new: [t[:, 1:-1] for t in new(B, R + 2, 2, H, K).unbind(2)],
    "halves": lambda B, R, H, K, new: new(B, R, H, 2 * K).split(K, -1),
}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", list(VIEWS))
@pytest.mark.parametrize("B,H", [(2, 3), (1, 1), (3, 1)])
def test_interleaved_arrays_are_taken(kind, B, H):
    """Into such arrays and in place, each kept row where it belongs and nothing else written."""
    g = torch.Generator().manual_seed(3)
    R, K, n, budget, recent, out_rows = 90, 64, 80, 30, 4, 33
    new = lambda *s: torch.randn(*s, generator=g).half().to("cuda")  # noqa: E731
    w = torch.rand(B, H, R, generator=g)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    src, dst = VIEWS[kind](B, R, H, K, new), VIEWS[kind](B, out_rows, H, K, new)
    before, old = [t.cpu() for t in src], [t.cpu() for t in dst]
    m.mea_cache_evict(tuple(src), w.to("cuda"), lens, budget, recent, out=tuple(dst))
    after = [t.cpu() for t in src]
    m.mea_cache_evict(tuple(src), w.to("cuda"), lens, budget, recent)
    for i in range(2):
        assert torch.equal(after[i], before[i])
        for b in range(B):
            for h in range(H):
                rows = U.choose(w[b, h], n, budget, recent)
                for got, rest in ((dst[i].cpu(), old[i]), (src[i].cpu(), before[i])):
                    assert torch.equal(got[b, :budget, h], before[i][b, rows, h])
                    assert torch.equal(got[b, budget:, h], rest[b, budget:, h])
    cache = m.mea_kv4_alloc(B, n, H, K, torch.float16)
    m.mea_kv4_append(src[0][:, :n], src[1][:, :n], cache, torch.zeros_like(lens))
    want = m.mea_kv4_read(cache, lens)
    m.mea_kv4_read(cache, lens, k_out=src[0], v_out=src[1])
    for i in range(2):
        assert torch.equal(src[i][:, :n], want[i])
    assert m.read_device_status() == 0
