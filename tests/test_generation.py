"""A generation through PagedKVCache.extend and beam_step: prompts, chunks, forks and single
tokens with rotary positions, capped and masked scores, and beam search over the same cache,
against dense attention in 64 bits over the tokens that each sequence holds."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_350_b200 as pa
from paged_kv_cache_350_b200 import binding as B

HQ, HKV, D, BS = 6, 2, 64, 8


def turn(x, positions, inv_freq):
    a = x.double()
    half = len(inv_freq)
    angle = positions.double()[:, None] * torch.from_numpy(inv_freq)[None, :]
    z = torch.complex(a[..., :half], a[..., half:2 * half]) * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    return torch.cat([z.real, z.imag, a[..., 2 * half:]], -1)


class Dense:
    """Per sequence: rotated keys and values of all its tokens, 64 bits."""

    def __init__(self, inv_freq, scale, softcap, window):
        self.inv_freq, self.scale, self.softcap, self.window, self.seqs = inv_freq, scale, softcap, window, {}

    def extend(self, ids, lens, q, k, v):
        outs, tols, t = [], [], 0
        # rounding of the rotated q and k to the pool's type, of the weights and of the output, each
        # half a step; the scores' sums in 32 bits
        half = torch.finfo(q.dtype).eps / 2
        for sid, n in zip(ids, lens):
            K, V = self.seqs.get(sid, (torch.zeros(0, HKV, D).double(), torch.zeros(0, HKV, D).double()))
            pos = torch.arange(K.shape[0], K.shape[0] + n)
            qs = turn(q[t:t + n], pos, self.inv_freq)
            K = torch.cat([K, turn(k[t:t + n], pos, self.inv_freq)])
            V = torch.cat([V, v[t:t + n].double()])
            self.seqs[sid] = (K, V)
            key = torch.arange(K.shape[0])
            see = (key[None] <= pos[:, None]) & (key[None] > pos[:, None] - self.window)
            out = torch.zeros(n, HQ, D).double()
            tol = torch.zeros_like(out)
            for h in range(HQ):
                kk, vv = K[:, h // (HQ // HKV)], V[:, h // (HQ // HKV)]
                x = self.softcap * torch.tanh(qs[:, h] @ kk.T * self.scale / self.softcap)
                w = torch.softmax(x.masked_fill(~see, -math.inf), -1)
                out[:, h] = w @ vv
                mag = (qs[:, h].abs() @ kk.abs().T * self.scale).masked_fill(~see, 0.0).amax(-1, keepdim=True)
                dx = mag * (2 * half + D * 2.0 ** -22) + self.softcap * 1e-6
                tol[:, h] = (w @ vv.abs()) * (2 * torch.expm1(dx) + half + 2.0 ** -18) + out[:, h].abs() * half
            outs.append(out)
            tols.append(tol)
            t += n
        return torch.cat(outs), torch.cat(tols)


def close(got, ref):
    out, tol = ref
    assert bool(((got.cpu().double() - out).abs() <= tol).all()), float(((got.cpu().double() - out).abs() / tol).max())


@pytest.mark.parametrize("have,n,shared", [(0, 0, False), (0, 1, False), (5, 3, False), (5, 3, True), (8, 17, True),
                                           (7, 40, True), (3, 0, True)])
def test_append_tokens_is_append_slot_repeated(have, n, shared):
    one, many = pa.Allocator(12, 8, shuffle_seed=4), pa.Allocator(12, 8, shuffle_seed=4)
    for a in (one, many):
        a.add_seq(1, have)
        if shared:
            a.fork(1, 2)
    steps = [one.append_slot(1) for _ in range(n)]
    slots, pairs = many.append_tokens(1, n)
    assert slots.tolist() == [s for s, _, _ in steps]
    assert pairs == [(s, d) for _, s, d in steps if s >= 0]
    assert one.block_table(1) == many.block_table(1) and one.free_list() == many.free_list()
    before = many.block_table(1), many.free_list()
    for seq, count, status in ((1, 12 * 8 + 1, B.PA_ERR_OUT_OF_BLOCKS), (1, -1, B.PA_ERR_INVALID_ARG),
                               (9, 1, B.PA_ERR_NOT_FOUND)):
        with pytest.raises(pa.PAError) as e:
            many.append_tokens(seq, count)
        assert e.value.status == status
    assert (many.block_table(1), many.free_list()) == before


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompts_forks_chunks_and_single_tokens(dtype):
    g = torch.Generator().manual_seed(1)
    inv, _ = pa.pa_rope_frequencies(48)
    inv_d = torch.from_numpy(inv).cuda()
    cache = pa.PagedKVCache(64, BS, HKV, D, dtype=dtype, shuffle_seed=3)
    ref = Dense(inv, D ** -0.5, 8.0, 40)
    stream = torch.cuda.Stream()

    def both(ids, lens, on=None):
        T = sum(lens)
        qkv = torch.randn(T, (HQ + 2 * HKV) * D, generator=g).to(dtype)
        cut = lambda m: (m[:, :HQ * D].view(T, HQ, D), m[:, HQ * D:(HQ + HKV) * D].view(T, HKV, D),  # noqa: E731
                         m[:, (HQ + HKV) * D:].view(T, HKV, D))
        d = qkv.cuda()
        torch.cuda.synchronize()
        out = cache.extend(ids, lens, *cut(d), D ** -0.5, inv_freq=inv_d, softcap=8.0, window=40, stream=on)
        torch.cuda.synchronize()
        close(out, ref.extend(ids, lens, *cut(qkv)))
    both([0, 1], [21, 1])
    cache.fork(0, 2)
    ref.seqs[2] = ref.seqs[0]
    both([0, 2, 1], [1, 1, 1])                 # the shared partial block is copied before it is written
    both([1, 0, 3], [70, 2, 9], on=stream)     # a chunk, two tokens and a new prompt
    both([0, 1, 2, 3], [1, 1, 1, 1])
    cache.truncate(1, 60)
    ref.seqs[1] = tuple(x[:60] for x in ref.seqs[1])
    both([1], [5])
    cache.check_device_errors()
    for i in range(4):
        cache.retire(i)
    assert cache.alloc.num_free() == 64


@pytest.mark.gpu
def test_extend_is_all_or_nothing():
    cache = pa.PagedKVCache(6, BS, HKV, D, dtype=torch.float32)
    mk = lambda T: (torch.randn(T, HQ, D, device="cuda"), torch.randn(T, HKV, D, device="cuda"),  # noqa: E731
                    torch.randn(T, HKV, D, device="cuda"))
    first = mk(12)
    cache.extend([0], [12], *first, 0.1)
    cache.fork(0, 1)
    with pytest.raises(pa.PAError) as e:   # the fork's copied block fits, the new prompt does not
        cache.extend([1, 2], [1, 33], *mk(34), 0.1)
    assert e.value.status == B.PA_ERR_OUT_OF_BLOCKS
    assert cache.alloc.block_table(0)[1] == cache.alloc.block_table(1)[1] == 12
    with pytest.raises(pa.PAError):
        cache.alloc.block_table(2)
    torch.cuda.synchronize()
    for sid in (0, 1):   # both still hold the prompt's values
        slots = torch.from_numpy(cache.alloc.seq_slots(sid)).cuda()
        assert torch.equal(cache.v_pool.view(-1, HKV, D)[slots], first[2])
    free = cache.alloc.num_free()
    q, k, v = mk(3)
    for ids, lens in (([0, 0], [1, 2]), ([0], [2]), ([0, 1], [4, -1]), ([0], [1, 2])):
        with pytest.raises(ValueError):
            cache.extend(ids, lens, q, k, v, 0.1)
    with pytest.raises(ValueError):
        cache.extend([0], [3], q, k[:, :1], v[:, :1], 0.1)
    with pytest.raises(ValueError):
        cache.extend([0], [3], q.bfloat16(), k, v, 0.1)
    with pytest.raises(ValueError):
        cache.extend([0], [3], q, k, v, 0.1, inv_freq=torch.ones(40, dtype=torch.float64, device="cuda"))
    # refused by the calls themselves, after the tokens had their slots
    inv = torch.ones(16, dtype=torch.float64, device="cuda")
    for kw in (dict(window=-1), dict(softcap=-1.0), dict(alibi_slopes=torch.ones(HQ + 1, device="cuda")),
               dict(out=torch.empty(3, HQ + 1, D, device="cuda")), dict(inv_freq=inv, layout=7)):
        with pytest.raises((ValueError, pa.PAError)):
            cache.extend([0, 7], [2, 1], q, k, v, 0.1, **kw)
        assert cache.alloc.block_table(0)[1] == 12
        with pytest.raises(pa.PAError):
            cache.alloc.block_table(7)
    with pytest.raises(ValueError):
        cache.extend([0], [3], q, k.transpose(0, 1).contiguous().transpose(0, 1), v, 0.1, inv_freq=inv)
    assert cache.alloc.block_table(0)[1] == cache.alloc.block_table(1)[1] == 12
    assert cache.alloc.num_free() >= free - 1  # (a shared block may have become two)
    torch.cuda.synchronize()
    for sid in (0, 1):
        slots = torch.from_numpy(cache.alloc.seq_slots(sid)).cuda()
        assert torch.equal(cache.v_pool.view(-1, HKV, D)[slots], first[2])
    # queries that do not lie as the attention reads them are copied
    odd = torch.zeros(3 * HQ * D + 1, device="cuda")[1:].view(3, HQ, D).copy_(q)
    a = cache.extend([0], [3], odd, k, v, 0.1)
    cache.truncate(0, 12)
    b = cache.extend([0], [3], q, k, v, 0.1)
    assert torch.equal(a, b)
    cache.truncate(0, 12)
    assert cache.extend([0], [0], q[:0], k[:0], v[:0], 0.1).shape == (0, HQ, D)
    cache.check_device_errors()


@pytest.mark.gpu
def test_beam_search_over_the_cache():
    """Three beams of two requests: the selection against the definition, the re-pointed blocks
    against the histories, over steps that copy on write."""
    g = torch.Generator().manual_seed(5)
    N, W, V, dtype = 2, 3, 500, torch.bfloat16
    inv, _ = pa.pa_rope_frequencies(D)
    cache = pa.PagedKVCache(200, BS, HKV, D, dtype=dtype)
    ref = Dense(inv, D ** -0.5, 30.0, 1000)
    embed = torch.randn(V, (HQ + 2 * HKV) * D, generator=g).to(dtype)
    head = torch.randn(HQ * D, V, generator=g) * 0.2
    embed_d, head_d, inv_d = embed.cuda(), head.cuda(), torch.from_numpy(inv).cuda()

    def extend(ids, lens, toks):
        T = len(toks)
        cut = lambda m: (m[:, :HQ * D].view(T, HQ, D), m[:, HQ * D:(HQ + HKV) * D].view(T, HKV, D),  # noqa: E731
                         m[:, (HQ + HKV) * D:].view(T, HKV, D))
        rows = torch.tensor(toks)
        out = cache.extend(ids, lens, *cut(embed_d[rows.cuda()]), D ** -0.5, inv_freq=inv_d, softcap=30.0, window=1000)
        close(out, ref.extend(ids, lens, *cut(embed[rows])))
        return out
    ids = np.arange(N * W).reshape(N, W)
    prompts = [[int(t) for t in torch.randint(0, V, (n,), generator=g)] for n in (11, 16)]
    out = extend([int(ids[n, 0]) for n in range(N)], [len(x) for x in prompts], prompts[0] + prompts[1])
    last = out[[len(prompts[0]) - 1, len(prompts[0]) + len(prompts[1]) - 1]]
    logits = (last.flatten(1).float() @ head_d)[:, None].expand(N, W, V).contiguous()
    cum = torch.full((N, W), -math.inf, device="cuda")
    cum[:, 0] = 0.0
    history = torch.full((N, W, 8), -1, dtype=torch.int32, device="cuda")
    for n in range(N):
        for w in range(1, W):
            cache.fork(int(ids[n, 0]), int(ids[n, w]))
            ref.seqs[int(ids[n, w])] = ref.seqs[int(ids[n, 0])]
    texts = [[list(p) for _ in range(W)] for p in prompts]
    for step in range(5):
        x = torch.log_softmax(logits.double(), -1) + cum.double()[:, :, None]
        want = torch.sort(x.flatten(1), dim=-1, descending=True, stable=True)
        cum, parents, tokens, (history,) = cache.beam_step(ids, logits, cum, states=(history,))
        assert torch.equal(parents.long() * V + tokens.long(), want.indices[:, :W])
        # (32-bit exponentials and sums of 500 terms, one rounding of the score)
        assert bool(((cum.double() - want.values[:, :W]).abs() <= 2.0 ** -20 + cum.double().abs() * 2.0 ** -24).all())
        history[:, :, step] = tokens
        old = {i: ref.seqs[i] for i in ids.ravel().tolist()}
        for n in range(N):
            texts[n] = [texts[n][int(p)] + [int(t)] for p, t in zip(parents[n], tokens[n])]
            for w in range(W):
                ref.seqs[int(ids[n, w])] = old[int(ids[n, int(parents[n, w])])]
        for n in range(N):
            for w in range(W):
                assert history[n, w, :step + 1].tolist() == texts[n][w][len(prompts[n]):]
                assert cache.alloc.block_table(int(ids[n, w]))[1] == len(texts[n][w]) - 1
        flat = ids.ravel().tolist()
        out = extend(flat, [1] * (N * W), [texts[n][w][-1] for n in range(N) for w in range(W)])
        logits = (out.flatten(1).float() @ head_d).view(N, W, V)
    cache.check_device_errors()
    with pytest.raises(ValueError):
        cache.beam_step(ids[:, :2], logits, cum)
    with pytest.raises(pa.PAError):
        cache.beam_step(ids + 100, logits, cum)
