"""The cache operators on a stream other than the current one: what a call allocates is
ordered by the stream it runs on, whatever the current stream still has to do."""
import types

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def mea():
    import memory_efficient_exact_mea_b200 as m

    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def outputs(mea, what):
    """A call of an operator on fixed inputs (of its stream), what it returns as a list, and
    the sizes of all that it allocates."""
    g = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randn(2, 600, 2, 128, generator=g, device=DEV).bfloat16()
    q = torch.randn(2, 200, 8, 128, generator=g, device=DEV).bfloat16()
    w = torch.rand(2, 2, 600, generator=g, device=DEV)
    cache = mea.mea_kv4_alloc(2, 600, 2, 128, device=DEV)
    mea.mea_kv4_append(k, k, cache, i32([0, 0]))
    n, q1, small = i32([600, 600]), q[:, 0].contiguous(), (k.clone(), k.clone())
    lse = torch.zeros(2, 8, 200, device=DEV)
    run = dict(
        read=lambda s: mea.mea_kv4_read(cache, n, stream=s),
        decode=lambda s: mea.mea_decode_kv4(q1, cache, n, 600, weights=w, return_weights=True,
                                            stream=s),
        weights=lambda s: [mea.mea_key_weights(q, k, lse, stream=s)],
        evict=lambda s: mea.mea_cache_evict((k, k), w, n, 64, 5, out=small, stream=s),
    )[what]
    want = [t.clone() for t in run(None)]
    torch.cuda.synchronize()
    sizes = {t.numel() * t.element_size() for t in want} | {
        mea.mea_decode_kv4_workspace_size(2, 8, 2, 128, 600, True)}
    return run, want, sizes


@pytest.mark.parametrize("what", ["read", "decode", "weights", "evict"])
def test_memory_in_use_on_the_current_stream_is_left_alone(mea, what):
    """Tensors of the outputs' sizes are freed with their last kernels still queued on the
    current stream; the call on another stream neither waits for nor meets them."""
    run, want, sizes = outputs(mea, what)
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    old = [torch.empty(s, dtype=torch.uint8, device=DEV) for s in sizes for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    for t in old:
        t.fill_(0x5A)
    used = {t.data_ptr() for t in old}
    del old, t
    got = run(side)
    assert not used & {t.data_ptr() for t in got}
    side.synchronize()
    early = [t.clone() for t in got]  # queued behind the kernels above
    torch.cuda.synchronize()
    for a, b, c in zip(got, want, early):
        assert torch.equal(a, b) and torch.equal(c, b)


def test_results_outlive_their_tensor_on_the_current_stream(mea):
    """A result read by work queued on the current stream keeps its memory until that work is
    done, although it was allocated on the other stream and its tensor is gone."""
    run, want, _ = outputs(mea, "weights")
    side = torch.cuda.Stream()
    got = run(side)[0]
    side.synchronize()
    torch.cuda._sleep(100_000_000)
    copy = torch.empty_like(got)
    copy.copy_(got)
    place = got.data_ptr()
    del got
    with torch.cuda.stream(side):
        again = [torch.full_like(copy, 7.0) for _ in range(4)]
    assert place not in {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert torch.equal(copy, want[0])


def test_a_stream_of_another_device_is_refused(mea):
    cache = mea.mea_kv4_alloc(1, 8, 1, 64, device="cuda:0")
    other = types.SimpleNamespace(device_index=1, cuda_stream=0)
    k = torch.zeros(1, 8, 1, 64, device="cuda:0").bfloat16()
    lse, w = torch.zeros(1, 1, 8, device="cuda:0"), torch.zeros(1, 1, 8, device="cuda:0")
    n = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    for call in (lambda: mea.mea_kv4_append(k, k, cache, n, stream=other),
                 lambda: mea.mea_kv4_read(cache, n, stream=other),
                 lambda: mea.mea_decode_kv4(k[:, 0], cache, n, 8, stream=other),
                 lambda: mea.mea_key_weights(k, k, lse, stream=other),
                 lambda: mea.mea_cache_evict(cache, w, n, 4, 1, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
