"""Attention of ragged query tokens over the paged cache (pa_attention) against the formula in
64 bits."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_350_b200 as pa
from paged_kv_cache_350_b200 import binding as B

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


class Case:
    """A ragged batch on the host: n query tokens of L cached ones per sequence, blocks in a
    shuffled pool; every slot that no sequence holds is NaN."""

    def __init__(self, dtype, n, L, Hq, Hkv, D, bs, softcap=0.0, bias=False, window=0, prefix=None, first=None,
                 seed=0, spread=1.0, extra=0, tail=0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.n, self.L, self.Hq, self.Hkv, self.D, self.bs = dtype, n, L, Hq, Hkv, D, bs
        self.softcap, self.window, self.extra, self.tail = softcap, window, extra, tail
        dt = DT[dtype]
        nblk = [-(-x // bs) for x in L]
        NB, MB = sum(nblk) + 2, max(max(nblk), 1) + 1
        order = torch.randperm(NB, generator=g).tolist()
        self.tables = torch.full((len(n), MB), -1, dtype=torch.int32)
        self.k_pool = torch.full((NB, bs, Hkv, D), NAN, dtype=dt)
        self.v_pool = torch.full((NB, bs, Hkv, D), NAN, dtype=dt)
        self.keys, self.values = [], []
        for b, (x, m) in enumerate(zip(L, nblk)):
            ids = [order.pop() for _ in range(m)]
            self.tables[b, :m] = torch.tensor(ids, dtype=torch.int32)
            k, v = (torch.randn(x, Hkv, D, generator=g).to(dt) for _ in range(2))
            self.keys.append(k.double())
            self.values.append(v.double())
            for i, blk in enumerate(ids):
                part = slice(i * bs, min(x, (i + 1) * bs))
                self.k_pool[blk, :part.stop - part.start] = k[part]
                self.v_pool[blk, :part.stop - part.start] = v[part]
        self.starts = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
        T = int(self.starts[-1])
        self.q = (torch.randn(T + tail, Hq, D, generator=g) * spread).to(dt)
        self.lens = torch.tensor(L, dtype=torch.int32)
        self.scale = D ** -0.5
        self.slopes = None
        if bias:
            self.slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)])
        self.prefix = None if prefix is None else torch.tensor(prefix, dtype=torch.int32)
        self.first = None if first is None else torch.tensor(first, dtype=torch.int32)

    def reference(self):
        """out, and for the tolerance: sum of weights * |v|, the largest score error per row."""
        T, G = int(self.starts[-1]), self.Hq // self.Hkv
        out = torch.zeros(T, self.Hq, self.D, dtype=torch.float64)
        size, dx = torch.zeros_like(out), torch.zeros(T, self.Hq, 1, dtype=torch.float64)
        for b in range(len(self.n)):
            t0, t1 = int(self.starts[b]), int(self.starts[b + 1])
            L = self.L[b]
            if t1 == t0 or L == 0:
                continue
            pos = torch.arange(L - (t1 - t0), L)[:, None]
            key = torch.arange(L)[None, :]
            see = key <= pos
            if self.prefix is not None:
                see |= key < int(self.prefix[b])
            if self.window:
                see &= key > pos - self.window
            if self.first is not None:
                see &= key >= self.first[t0:t1, None]
            see &= pos >= 0
            for h in range(self.Hq):
                q, k, v = self.q[t0:t1, h].double(), self.keys[b][:, h // G], self.values[b][:, h // G]
                x = q @ k.T * self.scale
                # Products summed over D in 32 bits (any order, 2^-22 a step for a tensor-core
                # sum that truncates): (D + 4) 2^-22 of the sum of magnitudes, then a few ulp of
                # the score from scale, cap (1e-6 of the cap) and bias.
                mag = q.abs() @ k.abs().T * self.scale
                if self.softcap:
                    x = self.softcap * torch.tanh(x / self.softcap)
                d = mag * (self.D + 4) * 2.0 ** -22 + x.abs() * 2.0 ** -21 + self.softcap * 1e-6
                if self.slopes is not None:
                    bias = float(self.slopes[h]) * (pos - key).abs().double()
                    x = x - bias
                    d = d + bias * 2.0 ** -22
                x = x.masked_fill(~see, -math.inf)
                w = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
                out[t0:t1, h] = w @ v
                size[t0:t1, h] = w @ v.abs()
                # only keys that carry weight count: e^(x - max) d, at most 1 * d there
                dx[t0:t1, h, 0] = (w * d).sum(-1) + (w * d).amax(-1)
        return out, size, dx

    def run(self, stream=None, graph=False, table_holes=False):
        T = int(self.starts[-1])
        dt = DT[self.dtype]
        row = self.Hq * self.D + self.extra
        buf = torch.full((T + self.tail, row), NAN, dtype=dt, device="cuda")
        q = buf[:, :self.Hq * self.D].view(T + self.tail, self.Hq, self.D)
        q.copy_(self.q)
        out = torch.full((T + self.tail, self.Hq, self.D), 7.0, dtype=dt, device="cuda")
        most = max(max(self.n), 1)
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        tables = self.tables.clone()
        if table_holes:  # blocks before every token's window
            for b, L in enumerate(self.L):
                lo = max(0, L - self.n[b] - self.window + 1)
                tables[b, :lo // self.bs] = -1
        args = [out, q, self.k_pool.cuda(), self.v_pool.cuda(), tables.cuda(), self.lens.cuda(), self.starts.cuda(),
                most, self.scale]
        size = pa.pa_attention_workspace_size(T + self.tail, len(self.n), most, self.Hq, self.Hkv, self.D, self.bs,
                                              self.tables.shape[1])
        ws = torch.full((max(size, 1),), 0xFF, dtype=torch.uint8, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = dict(softcap=self.softcap, alibi_slopes=dev(self.slopes), window=self.window, prefix_lens=dev(self.prefix),
                  first_keys=dev(self.first) if self.first is None or not self.tail else
                  torch.cat([self.first, torch.zeros(self.tail, dtype=torch.int32)]).cuda(),
                  workspace=ws, err_flag=err)
        torch.cuda.synchronize()
        pa.pa_attention(*args, stream=stream, **kw)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        if self.tail:  # rows behind the last sequence stay as they were
            assert bool((out[T:] == 7.0).all())
        return out[:T].cpu().double(), (args, kw)

    def close(self, got):
        ref, size, dx = self.reference()
        n = max(max(self.L), 1)
        if self.dtype == "bf16":
            # every weight rounded to bf16 on its way into the matrix product, and the output
            tol = size * 2.0 ** -8 + ref.abs() * 2.0 ** -8
        else:
            tol = size * 0
        # a weight is off by its score's error, the sums by 2^-24 a key; exponentials 2^-21
        tol = tol + size * (2 * dx + (n + 8) * 2.0 ** -24 + 2.0 ** -20) + 1e-30
        bad = ~((got - ref).abs() <= tol)
        assert not bool(bad.any()), (int(bad.sum()), float(((got - ref).abs() / tol).nan_to_num(1e9).max()),
                                     [int(i) for i in bad.nonzero()[0]])

    def check(self, **kw):
        got, call = self.run(**kw)
        self.close(got)
        return got, call


def docs_first(n, L, step):
    """First key of each query token's document, documents of `step` tokens."""
    return [p // step * step if p >= 0 else 0 for a, x in zip(n, L) for p in range(x - a, x)]


# ---- refusals --------------------------------------------------------------------------------

def test_workspace_size_and_refusals():
    ok = (16, 2, 8, 8, 2, 64, 16, 4)
    assert pa.pa_attention_workspace_size(*ok) > 0
    assert pa.pa_attention_workspace_size(0, 2, 8, 8, 2, 64, 16, 4) == 0
    for i, bad in ((0, -1), (1, -1), (2, -1), (3, 7), (3, 0), (4, 0), (5, 96), (6, 5), (7, 0)):
        a = list(ok)
        a[i] = bad
        with pytest.raises(pa.PAError):
            pa.pa_attention_workspace_size(*a)

    p = 0x10000

    def call(T=4, B_=2, most=2, Hq=4, Hkv=2, D=64, bs=16, MB=4, NB=8, stride=256, scale=0.125, mods=None, dt=B.PA_BF16,
             out=p, q=0x20000, ws=p, wbytes=1 << 40, tables=p):
        return B.lib.pa_attention(out, q, p, p, tables, p, p, T, B_, most, Hq, Hkv, D, bs, MB, NB, stride, scale,
                                  mods, dt, ws, wbytes, None, None)
    M = B.pa_attention_mods
    for bad in (dict(T=-1), dict(B_=-1), dict(most=-1), dict(Hq=5), dict(Hkv=0), dict(MB=0), dict(NB=0),
                dict(scale=NAN), dict(dt=5), dict(stride=255), dict(stride=260), dict(mods=M(-1.0)), dict(mods=M(NAN)),
                dict(mods=M(0.0, -1)), dict(out=None), dict(q=0x10008), dict(ws=0x10010), dict(ws=None),
                dict(tables=None), dict(mods=M(0.0, 0, 0x1002)), dict(mods=M(0.0, 0, None, 0x1002)),
                dict(mods=M(0.0, 0, None, None, 0x1002)), dict(scale=1e31), dict(mods=M(1e-31)), dict(mods=M(1e31)),
                dict(scale=10.0, mods=M(1e-30)), dict(out=0x20000), dict(out=0x207f0), dict(out=0x1f810)):
        assert call(**bad) == B.PA_ERR_INVALID_ARG, bad
    for bad in (dict(D=80, stride=320), dict(bs=64)):
        assert call(**bad) == B.PA_ERR_UNSUPPORTED, bad
    assert call(T=0) == B.PA_OK and call(B_=0) == B.PA_OK and call(most=0) == B.PA_OK


# ---- against the formula ---------------------------------------------------------------------

HEADS = [(8, 2, 128), (14, 2, 64), (4, 4, 64), (12, 1, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("bs", [4, 8, 16, 32])
def test_prompts_and_chunks(dtype, Hq, Hkv, D, bs):
    """Whole prompts, chunks behind cached tokens, sequences without query tokens or keys."""
    Case(dtype, [1, 70, 0, 129, 33, 0], [1, 70, 9, 300, 400, 0], Hq, Hkv, D, bs, seed=bs + Hq).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS + [(16, 1, 64), (32, 2, 128), (5, 5, 128), (17, 1, 128)])
@pytest.mark.parametrize("bs", [4, 16])
def test_single_tokens(dtype, Hq, Hkv, D, bs):
    L = [1, 2, 63, 64, 65, 127, 128, 129, 700, 0, 5, 2100]
    Case(dtype, [1] * len(L), L, Hq, Hkv, D, bs, seed=Hq).check()


MODS = {
    "cap": dict(softcap=5.0, spread=4.0),
    "cap_small": dict(softcap=50.0, spread=4.0),
    "cap_wide": dict(softcap=50.0, spread=60.0),
    "bias": dict(bias=True),
    "window": dict(window=37),
    "window_1": dict(window=1),
    "prefix": dict(prefix=[0, 50, 9, 300, 7]),
    "prefix_window": dict(prefix=[1, 64, 3, 130, 400], window=40, bias=True),
    "all": dict(softcap=8.0, spread=3.0, bias=True, window=100, prefix=[0, 20, 5, 10, 300]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", sorted(MODS))
@pytest.mark.parametrize("n", [[1, 70, 2, 129, 33], [1, 1, 1, 1, 1], [3, 1, 2, 0, 3]])
def test_modified_scores_and_masks(dtype, name, n):
    Case(dtype, n, [1, 70, 9, 300, 400], 8, 2, 64, 16, seed=len(name), **MODS[name]).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("step", [1, 16, 50])
def test_documents(dtype, step):
    n, L = [200, 1, 64, 5], [200, 77, 301, 5]
    Case(dtype, n, L, 6, 2, 128, 16, bias=True, first=docs_first(n, L, step), seed=step).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(dtype):
    """First keys past the token, more query tokens than keys, empty sequences: zero rows."""
    n, L = [40, 3, 5, 2], [40, 0, 2, 1]
    first = [0] * 50
    first[3], first[20], first[39] = 1000, 21, 40
    c = Case(dtype, n, L, 4, 2, 64, 16, first=first, seed=3, tail=3)
    got, _ = c.check()
    for t in (3, 20, 39, 40, 41, 42, 43, 44, 45, 48):
        assert bool((got[t] == 0).all()), t


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scattered_first_keys(dtype):
    g = torch.Generator().manual_seed(4)
    n, L = [150, 80], [400, 80]
    first = [int(torch.randint(0, max(p, 1), (1,), generator=g)) for a, x in zip(n, L) for p in range(x - a, x)]
    Case(dtype, n, L, 8, 4, 64, 32, first=first).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,L", [([1], [40000]), ([1, 1, 1], [9000, 20000, 3]), ([20], [30000]), ([1500], [1500]),
                                 ([700, 3], [5000, 9000])])
def test_long_axes_are_split_and_joined(dtype, n, L):
    if dtype == "f32" and max(n) > 100:
        L = [min(x, 2000) for x in L]
    Case(dtype, n, L, 8, 2, 128, 16, softcap=20.0, bias=True).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("extra,tail", [(0, 5), (8, 0), (512, 70)])
def test_strided_queries_and_a_padded_batch(dtype, extra, tail):
    Case(dtype, [17, 90], [50, 90], 4, 2, 64, 16, extra=extra, tail=tail).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [[1, 1], [40, 100]])
def test_freed_blocks_before_a_window_are_not_read(dtype, n):
    Case(dtype, n, [500, 333], 8, 2, 64, 16, window=60).check(table_holes=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores_and_equal_keys(dtype):
    c = Case(dtype, [65, 1], [200, 900], 4, 1, 128, 16, spread=200.0)
    c.check()
    c = Case(dtype, [5, 1], [300, 900], 4, 2, 64, 16, spread=0.0)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("mods", [{}, dict(softcap=30.0, spread=3.0), dict(bias=True, window=50)])
def test_many_short_units(mods):
    """More units than the ranges of one wave: they are taken one by one, empty ones skipped."""
    n = [33 if i % 7 else 0 for i in range(190)]
    L = [a + (i * 37) % 150 for i, a in enumerate(n)]
    Case("bf16", n, L, 16, 8, 64, 16, seed=2, **mods).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_sequences_than_the_token_kernel_scans(dtype):
    Case(dtype, [1] * 2100, [i % 40 for i in range(2100)], 2, 1, 64, 8, softcap=10.0).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wide_groups(dtype):
    """More query heads per KV head than a product's rows."""
    Case(dtype, [3, 1], [50, 200], 130, 1, 64, 16, bias=True).check()
    Case(dtype, [3, 1], [50, 200], 128, 1, 64, 16, window=30).check()
    Case(dtype, [9, 1], [50, 200], 33, 1, 64, 16, softcap=20.0).check()


@pytest.mark.gpu
def test_negative_and_zero_scales_and_extreme_caps():
    for scale, cap in ((-0.1, 0.0), (0.0, 0.0), (-0.1, 5.0), (0.1, 1e-3), (1e-6, 30.0), (0.1, 1e5)):
        for n in ([1, 1], [40, 3]):
            c = Case("bf16", n, [70, 300], 4, 2, 64, 16, softcap=cap)
            c.scale = scale
            c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0.5, 5.0, 30.0, 40.0, 50.0, 50.5, 60.0, 400.0])
@pytest.mark.parametrize("spread", [1.0, 40.0])
def test_caps_of_all_widths(cap, spread):
    for kw in ({}, dict(bias=True), dict(window=33)):
        Case("bf16", [70, 3, 150], [300, 200, 150], 4, 2, 64, 16, softcap=cap, spread=spread, **kw).check()


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [30.0, 50.0])
@pytest.mark.parametrize("size", [2.0 ** 50, 2.0 ** -15])
def test_capped_scores_with_large_and_small_values(cap, size):
    c = Case("bf16", [70, 3], [300, 200], 4, 2, 64, 16, softcap=cap, spread=40.0)
    c.v_pool *= size   # (a power of two: exact)
    c.values = [v * size for v in c.values]
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [[1, 1], [70, 1]])
def test_infinities_behind_a_mask_reach_nobody(dtype, n):
    """Slots past the lengths and before every window hold infinities of both signs."""
    c = Case(dtype, n, [100, 333], 8, 2, 64, 16, window=20)
    for pool in (c.k_pool, c.v_pool):
        pool[pool != pool] = math.inf
        pool[:, ::2][pool[:, ::2] == math.inf] = -math.inf
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [[1, 1], [40, 70]])
def test_blocks_past_32_bits(n):
    """The blocks lie behind 2^32 bytes (2^31 elements) of the pools."""
    c = Case("bf16", n, [100, 300], 8, 8, 128, 32)
    far = (1 << 31) // (32 * 8 * 128) + 5
    small = c.k_pool.shape[0]
    kd, vd = (torch.empty((far + small, 32, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kd[far:], vd[far:] = c.k_pool.cuda(), c.v_pool.cuda()
    _, (args, kw) = c.run()
    args[2], args[3] = kd, vd
    args[4] = torch.where(args[4] >= 0, args[4] + far, args[4])
    args[0].fill_(7.0)
    pa.pa_attention(*args, **kw)
    torch.cuda.synchronize()
    assert int(kw["err_flag"].item()) == 0
    c.close(args[0][:sum(n)].cpu().double())
    # the cache write reaches them as well
    T = 3
    q, k, v = (torch.randn(T, 8, 128, device="cuda").bfloat16() for _ in range(3))
    slots = torch.tensor([far * 32 + 1, (far + small) * 32 - 1, far * 32 + 40], device="cuda")
    inv = torch.zeros(64, dtype=torch.float64, device="cuda")   # no rotation: the rows themselves
    pa.pa_rope_and_cache(torch.empty_like(q), q, k, v, kd, vd, torch.zeros(T, dtype=torch.int32, device="cuda"), slots,
                         inv)
    assert torch.equal(kd.view(-1, 8, 128)[slots], k) and torch.equal(vd.view(-1, 8, 128)[slots], v)


@pytest.mark.gpu
def test_two_streams_with_a_workspace_each():
    cases = [Case("bf16", [64] * 4, [500, 64, 700, 90], 8, 2, 128, 16, seed=s, softcap=20.0) for s in (1, 2)]
    runs = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for (_, (args, _)) in runs:
        args[0].fill_(0)
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (_, (args, kw)) in zip(streams, runs):
            pa.pa_attention(*args, stream=s, **kw)
    torch.cuda.synchronize()
    for got, (args, _) in runs:
        assert torch.equal(args[0].cpu().double(), got)


@pytest.mark.gpu
def test_matches_pa_decode_on_single_tokens():
    c = Case("bf16", [1] * 20, [1 + 37 * i for i in range(20)], 32, 8, 128, 16)
    got, (args, _) = c.check()
    out, q, kp, vp, tables, lens = args[:6]
    other = torch.empty_like(out)
    ws = torch.empty(max(pa.pa_decode_workspace_size(20, 32, 8, 128, tables.shape[1] * 16, 16), 1), dtype=torch.uint8,
                     device="cuda")
    pa.pa_decode(other, q.contiguous(), kp, vp, tables, lens, c.scale, workspace=ws)
    c.close(other.cpu().double())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeated_calls_agree_bit_for_bit_and_in_a_graph(dtype):
    """The same call, twice on another stream and replayed: equal bits; then with other lengths."""
    c = Case(dtype, [1, 30, 1, 200], [900, 70, 5000, 260], 8, 2, 64, 16, softcap=10.0, window=800)
    first, (args, kw) = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args[0].fill_(0)
    torch.cuda.synchronize()
    pa.pa_attention(*args, stream=s, **kw)
    torch.cuda.synchronize()
    assert torch.equal(args[0].cpu().double(), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_attention(*args, **kw)
    args[0].fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(args[0].cpu().double(), first)
    c2 = Case(dtype, [1, 30, 1, 200], [900, 70, 5000, 260], 8, 2, 64, 16, softcap=10.0, window=800)
    c2.L, c2.n = [450, 70, 1, 200], c2.n
    c2.keys = [k[:x] for k, x in zip(c2.keys, c2.L)]
    c2.values = [v[:x] for v, x in zip(c2.values, c2.L)]
    args[5].copy_(torch.tensor(c2.L, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    c2.close(args[0].cpu().double())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_lengths_spans_and_blocks_are_flagged(dtype):
    c = Case(dtype, [4, 1, 30], [40, 64, 90], 4, 2, 64, 16)
    _, (args, kw) = c.run()

    def flag(change, most=None):
        a = [t.clone() if torch.is_tensor(t) and t.dtype == torch.int32 else t for t in args]
        change(a)
        if most is not None:
            a[7] = most
        kw["err_flag"].zero_()
        pa.pa_attention(*a, **kw)
        torch.cuda.synchronize()
        return int(kw["err_flag"].item())
    assert flag(lambda a: a[5].__setitem__(1, -3)) == B.PA_DEVERR_BAD_SEQ_LEN
    assert flag(lambda a: a[6].__setitem__(1, 60)) == B.PA_DEVERR_BAD_SEQ_LEN     # spans not in order
    assert flag(lambda a: a[6].__setitem__(3, 1000)) == B.PA_DEVERR_BAD_SEQ_LEN   # past the tokens
    assert flag(lambda a: None, most=29) == B.PA_DEVERR_BAD_SEQ_LEN               # longer than said
    assert flag(lambda a: a[4].__setitem__((0, 1), 10000)) == B.PA_DEVERR_BAD_BLOCK_ID
    assert flag(lambda a: a[4].__setitem__((2, 0), -1)) == B.PA_DEVERR_BAD_BLOCK_ID
    # a length past the table is cut to the table's
    assert flag(lambda a: (a[5].__setitem__(0, 1 << 20), a[4].clamp_(min=0))) == B.PA_DEVERR_BAD_SEQ_LEN
    assert flag(lambda a: None) == 0


@pytest.mark.gpu
def test_binding_refusals():
    c = Case("bf16", [4, 1], [40, 64], 4, 2, 64, 16)
    _, (args, kw) = c.run()
    out, q, kp, vp, tables, lens, starts, most, scale = args
    for i, bad in [(0, out[:, :, :32]), (1, q.float()), (1, q.transpose(0, 1)), (2, kp[:, :8]), (4, tables.long()),
                   (5, lens[:1]), (6, starts[:2]), (5, lens.cpu())]:
        a = list(args)
        a[i] = bad
        with pytest.raises(ValueError):
            pa.pa_attention(*a, **kw)
    for bad in (dict(alibi_slopes=torch.ones(3, device="cuda")), dict(prefix_lens=lens.float()),
                dict(first_keys=lens)):
        with pytest.raises(ValueError):
            pa.pa_attention(*args, **{**kw, **bad})
    with pytest.raises(pa.PAError):
        pa.pa_attention(*args, **{**kw, "workspace": kw["workspace"][:256]})
    with pytest.raises(pa.PAError):
        pa.pa_attention(*args, **{**kw, "workspace": None})
