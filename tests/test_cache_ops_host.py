"""Refusals of the cache operators (4-bit cache, key weights, eviction), found on the
host before any launch: the C entry points with made-up addresses, and the binding's
own checks.  Needs no GPU."""
import ctypes

import pytest
import torch

import memory_efficient_exact_mea_b200 as m

I64 = ctypes.c_int64 * 3
P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
NAN = float("nan")


def call(fn, defaults, **kw):
    a = {**defaults, **kw}
    assert not set(kw) - set(defaults)
    return fn(*(ctypes.c_float(x) if isinstance(x, float) else x for x in a.values()))


ST = I64(1024, 64, 64)
APPEND = dict(k=P(4096), v=P(4096), kc=P(4096), kp=P(4096), vc=P(4096), vp=P(4096), lens=P(16),
              qlens=None, B=2, M=3, rows=10, Hkv=1, K=64, ks=ST, vs=ST, dtype=0, stream=None)
READ = dict(kc=P(4096), kp=P(4096), vc=P(4096), vp=P(4096), rows_t=P(16), first=None, k=P(4096),
            v=P(4096), B=2, rows=10, out=5, Hkv=1, K=64, ks=ST, vs=ST, dtype=0, stream=None)
DECODE = dict(q=P(4096), kc=P(4096), kp=P(4096), vc=P(4096), vp=P(4096), lens=P(16), o=P(4096),
              lse=None, win=None, wout=None, B=2, Hq=4, Hkv=2, K=64, rows=100, bound=100, dtype=0,
              alibi=0, scale=0.125, ws=P(4096), bytes=1 << 30, stream=None)
WEIGH = dict(q=P(4096), k=P(4096), lse=P(16), clen=None, qlen=None, win=None, wout=P(16), B=2, M=3,
             N=9, Hq=4, Hkv=2, K=64, qs=ST, ks=ST, dtype=0, causal=1, alibi=0, scale=0.125,
             stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(M=-1), INVALID), (dict(rows=-1), INVALID), (dict(Hkv=0), INVALID),
    (dict(dtype=2), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
    (dict(k=None), INVALID), (dict(vp=None), INVALID), (dict(lens=None), INVALID),
    (dict(K=96), UNSUPPORTED), (dict(k=P(4104)), UNSUPPORTED), (dict(kp=P(4100)), UNSUPPORTED),
    (dict(ks=I64(1024, 60, 64)), UNSUPPORTED), (dict(vs=I64(1024, 0, 64)), UNSUPPORTED),
    (dict(B=1 << 16, M=1 << 16), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(B=0), OK), (dict(M=0), OK)])
def test_append(kw, code):
    assert call(m.lib.mea_kv4_append, APPEND, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(out=-1), INVALID), (dict(rows=-1), INVALID), (dict(Hkv=0), INVALID),
    (dict(dtype=-1), INVALID), (dict(ks=None), INVALID), (dict(kc=None), INVALID),
    (dict(rows_t=None), INVALID), (dict(v=None), INVALID), (dict(K=32), UNSUPPORTED),
    (dict(v=P(4098)), UNSUPPORTED), (dict(vs=I64(1024, 64, -64)), UNSUPPORTED),
    (dict(B=1 << 16, out=1 << 16), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(B=0), OK), (dict(out=0), OK)])
def test_read(kw, code):
    assert call(m.lib.mea_kv4_read, READ, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hq=5), INVALID), (dict(rows=-1), INVALID),
    (dict(bound=-1), INVALID), (dict(dtype=7), INVALID), (dict(scale=NAN), INVALID),
    (dict(win=P(16)), INVALID), (dict(q=None), INVALID), (dict(o=None), INVALID),
    (dict(lens=None), INVALID), (dict(kp=None), INVALID), (dict(K=256), UNSUPPORTED),
    (dict(q=P(4104)), UNSUPPORTED), (dict(vc=P(4104)), UNSUPPORTED),
    (dict(B=70000), UNSUPPORTED), (dict(bound=4000, bytes=16), WORKSPACE),
    (dict(bound=4000, ws=None), WORKSPACE), (dict(bound=4000, ws=P(4112)), WORKSPACE),
    (dict(wout=P(16), ws=None), WORKSPACE), (dict(bound=(1 << 30) + 1), UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(B=0), OK)])
def test_decode(kw, code):
    if kw.get("B") == 70000:
        kw = dict(kw, bound=10)
    assert call(m.lib.mea_decode_kv4, DECODE, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(Hq=3), INVALID),
    (dict(Hkv=0), INVALID), (dict(dtype=3), INVALID), (dict(causal=2), INVALID),
    (dict(scale=NAN), INVALID), (dict(qlen=P(16)), INVALID), (dict(M=0), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(lse=None), INVALID),
    (dict(wout=None), INVALID), (dict(qs=None), INVALID), (dict(scale=-1.0), UNSUPPORTED),
    (dict(K=80), UNSUPPORTED), (dict(k=P(4104)), UNSUPPORTED),
    (dict(ks=I64(1024, 65, 64)), UNSUPPORTED), (dict(N=(1 << 30) + 1), UNSUPPORTED),
    (dict(B=0), OK), (dict(N=0), OK)])
def test_key_weights(kw, code):
    assert call(m.lib.mea_key_weights, WEIGH, **kw) == code


def evict(plane=None, n=1, w=P(1 << 20), wo=P(2 << 20), lens=P(16), new=P(64), kept=P(4096), B=2, H=2,
          rows=10, out=6, budget=5, recent=1, **over):
    """Source rows of 16 bytes [2, 10, 2] at 1 << 24, destination at 1 << 25."""
    p = (m._Plane * 5)()
    for i in range(5):
        p[i] = m._Plane((1 << 24) + i * 1024, (1 << 25) + i * 1024, I64(320, 32, 16),
                        I64(192, 32, 16), 16)
    for k, x in over.items():
        setattr(p[0], k, x)
    return m.lib.mea_cache_evict(p, n, w, wo, lens, new, kept, B, H, rows, out, budget, recent, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(H=0), INVALID), (dict(n=0), INVALID), (dict(n=5), INVALID),
    (dict(budget=0), INVALID), (dict(budget=7), INVALID), (dict(recent=-1), INVALID),
    (dict(recent=6), INVALID), (dict(lens=None), INVALID), (dict(new=None), INVALID),
    (dict(new=P(16)), INVALID), (dict(kept=None), INVALID), (dict(w=None), INVALID),
    (dict(wo=None), INVALID), (dict(rows=0), INVALID), (dict(src=None), INVALID),
    (dict(row_bytes=0), INVALID), (dict(src_strides=I64(-320, 32, 16)), INVALID),
    (dict(row_bytes=6), UNSUPPORTED), (dict(src=(1 << 24) + 2), UNSUPPORTED),
    (dict(dst_strides=I64(192, 34, 16)), UNSUPPORTED), (dict(B=40000), UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(src_strides=I64(1 << 41, 32, 16)), UNSUPPORTED),
    (dict(dst=1 << 24), INVALID),                      # in place, but fewer rows
    (dict(dst=(1 << 24) + 320), INVALID),              # overlaps its source
    (dict(dst=1 << 20), INVALID),                      # overlaps the weights
    (dict(wo=P(1 << 20)), INVALID),                    # weights in place, but fewer rows
    (dict(n=2, dst=(1 << 25) + 1024), INVALID),        # two planes into the same rows
    (dict(n=2, dst=(1 << 25) + 1032), INVALID),
    (dict(B=0), OK)])
def test_evict(kw, code):
    assert evict(**kw) == code


def test_workspace_sizes():
    size = m.mea_decode_kv4_workspace_size
    r256 = lambda x: -(-x // 256) * 256  # noqa: E731
    assert size(64, 32, 8, 128, 0) == 0
    assert size(200, 8, 8, 64, 900) == 0            # one split each: nothing to join
    n = size(200, 8, 8, 64, 900, True)
    assert n == r256(1600 * 4) + r256(1600 * 900 * 4)
    assert size(1, 8, 8, 64, 1024) == r256(8 * 8 * 64 * 4) + r256(8 * 8 * 4)  # 128-row splits
    assert size(-1, 8, 8, 64, 10) == size(1, 7, 2, 64, 10) == 0


def test_binding_refuses_before_the_library():
    f16, i32 = torch.float16, torch.int32
    with pytest.raises(ValueError):
        m.mea_kv4_alloc(1, 8, 1, 96, f16, "cpu")
    with pytest.raises(ValueError):
        m.mea_kv4_alloc(1, 8, 1, 64, torch.float32, "cpu")
    good = m.mea_kv4_alloc(2, 8, 3, 64, f16, "cpu")
    x, lens = torch.zeros(2, 4, 3, 64, dtype=f16), torch.zeros(2, dtype=i32)
    for cache in (good,                                             # not on a GPU
                  good._replace(k_codes=good.k_codes.float()),
                  good._replace(v_codes=good.v_codes[:, :, :7]),
                  good._replace(k_params=good.k_params.float()),
                  good._replace(v_params=good.v_params.bfloat16()),
                  good._replace(k_codes=good.k_codes.transpose(1, 2)),
                  good._replace(v_params=good.v_params[:, :, :, :, :1])):
        with pytest.raises(ValueError):
            m.mea_kv4_append(x, x, cache, lens)
        with pytest.raises(ValueError):
            m.mea_kv4_read(cache, lens)
        with pytest.raises(ValueError):
            m.mea_decode_kv4(torch.zeros(2, 6, 64, dtype=f16), cache, lens, 8)
        with pytest.raises(ValueError):
            m.mea_cache_evict(cache, torch.zeros(2, 3, 8), lens, 4, 1)
    q, k, lse = torch.zeros(1, 4, 2, 64, dtype=f16), torch.zeros(1, 4, 1, 64, dtype=f16), \
        torch.zeros(1, 2, 4)
    for bad in ((q[0], k, lse), (q.float(), k.float(), lse), (q, k.bfloat16(), lse),
                (q, k[:, :, :, :32], lse), (q, k, lse.double()), (q, k, lse[:, :, :3]), (q, k, lse)):
        with pytest.raises(ValueError):
            m.mea_key_weights(*bad)
    with pytest.raises(ValueError):
        m.mea_key_weights(q, k, lse, q_seqlens=lens[:1])
    with pytest.raises(ValueError):
        m.mea_cache_evict((k, k[:, :3]), torch.zeros(1, 1, 4), lens[:1], 2, 1)
