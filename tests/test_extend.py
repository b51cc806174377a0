"""PagedKVCache.extend when a call cannot be made: the allocator's state, and what the cache holds."""

import pytest
import torch

import paged_kv_cache_350_b200 as pa
from paged_kv_cache_350_b200 import binding as B

HQ, HKV, D, BS = 6, 2, 64, 8


def state(alloc, ids):
    return ([alloc.block_table(i) for i in ids], [alloc.refcount(b) for b in range(alloc.num_blocks)],
            alloc.free_list())


@pytest.mark.parametrize("have,n,shared", [(0, 0, False), (0, 9, False), (5, 3, False), (5, 3, True), (5, 30, True),
                                           (8, 17, True), (7, 1, True), (3, 0, True)])
def test_undo_append_restores_the_allocator(have, n, shared):
    a = pa.Allocator(12, BS, shuffle_seed=3)
    a.add_seq(1, have)
    ids = [1]
    if shared:
        a.fork(1, 2)
        ids = [1, 2]
    before = state(a, ids)
    _, pairs = a.append_tokens(1, n)
    assert bool(pairs) == (shared and n > 0 and have % BS != 0)
    a.undo_append(1, n, pairs[0] if pairs else None)
    assert state(a, ids) == before


def test_undo_append_refuses_what_no_append_did():
    a = pa.Allocator(12, BS)
    a.add_seq(1, 5)
    a.fork(1, 2)
    a.fork(1, 3)
    old = a.block_table(1)[0][0]
    _, ((src, dst),) = a.append_tokens(1, 20)
    after = state(a, [1, 2, 3])
    for sid, n, pair, status in ((9, 1, None, B.PA_ERR_NOT_FOUND), (1, 26, None, B.PA_ERR_INVALID_ARG),
                                 (1, -1, None, B.PA_ERR_INVALID_ARG), (1, 20, (src, src), B.PA_ERR_INVALID_ARG),
                                 (1, 20, (11, dst), B.PA_ERR_INVALID_ARG), (1, 20, (12, dst), B.PA_ERR_INVALID_ARG),
                                 (1, 20, (src, dst + 1), B.PA_ERR_INVALID_ARG), (1, 1, (src, dst), B.PA_ERR_INVALID_ARG),
                                 (1, 25, (src, dst), B.PA_ERR_INVALID_ARG), (2, 0, (dst, old), B.PA_ERR_INVALID_ARG)):
        with pytest.raises(pa.PAError) as e:
            a.undo_append(sid, n, pair)
        assert e.value.status == status and state(a, [1, 2, 3]) == after
    a.undo_append(1, 20, (src, dst))
    assert a.block_table(1) == ([old], 5) and a.refcount(old) == 3 and a.refcount(dst) == 0


@pytest.mark.parametrize("lens", [[1, 1, 1], [1, 9, 2], [1, 1, 1, 30], [2, 0, 1, 1]])
def test_tokens_of_a_batch_are_taken_back(lens):
    """Forks of one partial block: all but one copy it; a new sequence; the reverse order restores it all."""
    cache = pa.PagedKVCache(16, BS, HKV, D, device="cpu", shuffle_seed=7)
    cache.alloc.add_seq(0, 13)
    cache.alloc.fork(0, 1)
    cache.alloc.fork(0, 2)
    before = state(cache.alloc, [0, 1, 2])
    grown = []
    ids = list(range(len(lens)))
    slots, pairs = cache._append_tokens(ids, lens, grown)
    assert slots.size == sum(lens) and len(pairs) == min(2, sum(n > 0 for n in lens[:3]))
    cache._take_back(grown)
    assert state(cache.alloc, [0, 1, 2]) == before
    with pytest.raises(pa.PAError):
        cache.alloc.block_table(3)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1, 1], [1, 9]])
@pytest.mark.parametrize("broken", ["pa_copy_blocks", "pa_reshape_and_cache", "pa_attention"])
def test_a_step_that_fails_on_its_way_loses_nothing(monkeypatch, lens, broken):
    cache = pa.PagedKVCache(16, BS, HKV, D, dtype=torch.float32)
    mk = lambda T: (torch.randn(T, HQ, D, device="cuda"), torch.randn(T, HKV, D, device="cuda"),  # noqa: E731
                    torch.randn(T, HKV, D, device="cuda"))
    first = mk(13)
    cache.extend([0], [13], *first, 0.1)
    cache.fork(0, 1)
    before = state(cache.alloc, [0, 1])

    def fails(*a, **k):
        raise torch.OutOfMemoryError("no memory")
    more = mk(sum(lens))
    with monkeypatch.context() as m:
        m.setattr(B, broken, fails)
        with pytest.raises(torch.OutOfMemoryError):
            cache.extend([0, 1], lens, *more, 0.1)
    assert state(cache.alloc, [0, 1]) == before
    torch.cuda.synchronize()
    for sid in (0, 1):
        slots = torch.from_numpy(cache.alloc.seq_slots(sid)).cuda()
        assert torch.equal(cache.v_pool.view(-1, HKV, D)[slots], first[2])
        assert torch.equal(cache.k_pool.view(-1, HKV, D)[slots], first[1])
    # and the same step goes through afterwards
    cache.extend([0, 1], lens, *more, 0.1)
    torch.cuda.synchronize()
    t = 0
    for sid, n in zip((0, 1), lens):
        slots = torch.from_numpy(cache.alloc.seq_slots(sid)).cuda()
        assert torch.equal(cache.v_pool.view(-1, HKV, D)[slots], torch.cat([first[2], more[2][t:t + n]]))
        t += n
    cache.check_device_errors()


def steps(cache, data, gate=None, **kw):
    """A prompt, forks of it, and single tokens with a chunk among them; their outputs."""
    outs = [cache.extend([0], [13], *data[0], 0.1, **kw)]
    for i in (1, 2):
        cache.fork(0, i)
    if gate is not None:
        gate()
    for d in data[1:]:
        outs.append(cache.extend([0, 1, 2], [1, 1, d[0].shape[0] - 2], *d, 0.1, **kw))
    return outs


@pytest.mark.gpu
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("on_stream", [False, True])
def test_the_host_goes_on_while_the_gpu_works(rotated, on_stream):
    """32 steps are queued behind a kernel that still runs when the last call returns."""
    g = torch.Generator().manual_seed(2)
    data = [tuple(torch.randn(T, h, D, generator=g).cuda() for h in (HQ, HKV, HKV)) for T in [13] + [3, 8] * 16]
    inv = torch.from_numpy(pa.pa_rope_frequencies(D)[0]).cuda() if rotated else None
    stream = torch.cuda.Stream() if on_stream else torch.cuda.current_stream()
    kw = dict(inv_freq=inv, softcap=30.0, stream=stream)
    torch.cuda.synchronize()
    mk = lambda: pa.PagedKVCache(200, BS, HKV, D, dtype=torch.float32, shuffle_seed=9)  # noqa: E731
    want = steps(mk(), data, **kw)
    torch.cuda.synchronize()
    done = torch.cuda.Event()

    def gate():
        with torch.cuda.stream(stream):
            torch.cuda._sleep(1_000_000_000)   # (about half a second)
            done.record(stream)
    cache = mk()
    torch.cuda.synchronize()
    got = steps(cache, data, gate, **kw)
    assert not done.query()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    cache.check_device_errors()


@pytest.mark.gpu
def test_a_step_is_not_captured():
    cache = pa.PagedKVCache(16, BS, HKV, D, dtype=torch.float32)
    mk = lambda T: tuple(torch.randn(T, h, D, device="cuda") for h in (HQ, HKV, HKV))  # noqa: E731
    cache.extend([0], [5], *mk(5), 0.1)
    more, before = mk(1), state(cache.alloc, [0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captured"):
            cache.extend([0], [1], *more, 0.1)
        x += 1
    assert state(cache.alloc, [0]) == before
    graph.replay()
    torch.cuda.synchronize()
    assert x.tolist() == [1.0] * 4
