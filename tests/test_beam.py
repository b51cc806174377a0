"""Beam search's selection and the reordering of states (pa_beam_topk, pa_beam_gather)."""

import numpy as np
import pytest
import torch

import paged_kv_cache_350_b200 as pa
from paged_kv_cache_350_b200 import binding as B


def reference(logits, cum, k, finished=None, eos=0):
    """Scores (64 bits), parents and tokens, from the definition; NumPy on the host."""
    N, W, V = logits.shape
    x = logits.double().numpy()
    scores, parents, tokens = (np.zeros((N, k)) for _ in range(3))
    for n in range(N):
        s = np.full((W, V), -np.inf)
        for w in range(W):
            c = float(cum[n, w])
            if finished is not None and finished[n, w]:
                s[w, eos] = c if np.isfinite(c) else -np.inf
                continue
            with np.errstate(all="ignore"):
                m = x[n, w].max()
                lse = m + np.log(np.exp(x[n, w] - m).sum())
            if np.isfinite(lse) and np.isfinite(c):
                s[w] = c + (x[n, w] - lse)
        flat = s.ravel()
        order = np.lexsort((np.arange(flat.size), -flat))[:k]
        scores[n], parents[n], tokens[n] = flat[order], order // V, order % V
    return torch.from_numpy(scores), torch.from_numpy(parents).int(), torch.from_numpy(tokens).int()


def select(logits, cum, k, finished=None, eos=0):
    N, W, V = logits.shape
    ws = torch.empty(max(pa.pa_beam_topk_workspace_size(N, W, V, k), 1), dtype=torch.uint8, device="cuda").fill_(0xFF)
    s = torch.full((N, k), float("nan"), device="cuda")
    p, t = (torch.full((N, k), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    pa.pa_beam_topk(s, p, t, logits, cum, finished=finished, eos_token=eos, workspace=ws)
    return s.cpu(), p.cpu(), t.cpu()


def lse_error(V):
    # Each exponential is off by 2^-22 and each of a lane's at most V / 256 + 1 additions by
    # 2^-24 of the sum; the scores are 64-bit from there on and rounded once (2^-24 of the score).
    return 2.0 ** -22 * 2 + (V / 256 + 2) * 2.0 ** -24


def check(logits, cum, k, finished=None, eos=0, device_logits=None):
    rs, rp, rt = reference(logits, cum, k, finished, eos)
    d = device_logits if device_logits is not None else logits.cuda()
    s, p, t = select(d, cum.cuda(), k, None if finished is None else finished.cuda(), eos)
    assert torch.equal(p, rp) and torch.equal(t, rt)
    inf = torch.isinf(rs)
    assert torch.equal(torch.isinf(s), inf)
    tol = lse_error(logits.shape[-1]) + rs.abs() * 2.0 ** -24
    assert bool(((s.double() - rs).abs()[~inf] <= tol[~inf]).all())


def random_case(N, W, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, W, V, generator=g) * spread).to(dtype)
    return x, -torch.rand(N, W, generator=g) * 6


def test_sizes_and_refusals():
    for a in ((-1, 1, 10, 1), (1, 0, 10, 1), (1, 1, 0, 1), (1, 1, 10, 0), (1, 1, 10, 11), (1, 2, 100, 33),
              (1, 1 << 16, 1 << 15, 1), (1, 1, (1 << 30) + 1, 1)):
        with pytest.raises(pa.PAError):
            pa.pa_beam_topk_workspace_size(*a)
    assert pa.pa_beam_topk_workspace_size(0, 4, 100, 4) == 0
    assert pa.pa_beam_topk_workspace_size(64, 16, 131072, 32) > 0

    p = 0x1000

    def call(N=2, W=2, V=64, k=2, stride=64, dt=B.PA_F32, ws=1 << 20, eos=0, fin=None, wsp=p, x=p, cum=0x8000):
        return B.lib.pa_beam_topk(p, p, p, x, cum, fin, eos, N, W, V, k, stride, dt, wsp, ws, None)
    for bad in (dict(N=-1), dict(W=0), dict(V=0), dict(k=0), dict(k=129), dict(stride=63), dict(dt=9), dict(ws=10),
                dict(wsp=None), dict(wsp=0x1010), dict(x=0x1002), dict(fin=p, eos=64), dict(fin=p, eos=-1),
                dict(cum=p, k=3), dict(cum=p + 4), dict(cum=p - 12)):
        assert call(**bad) == B.PA_ERR_INVALID_ARG, bad
    assert call(k=33) == B.PA_ERR_UNSUPPORTED
    assert call(N=0) == B.PA_OK

    def gather(N=1, W=2, k=2, row=8, dst=0x1000, src=0x9000, par=p):
        return B.lib.pa_beam_gather(dst, src, par, N, W, k, row, None, None)
    for bad in (dict(N=-1), dict(W=0), dict(k=0), dict(row=-1), dict(dst=None), dict(src=0x1008), dict(par=0x1002),
                dict(src=0xff8)):
        assert gather(**bad) == B.PA_ERR_INVALID_ARG, bad
    assert gather(N=0) == B.PA_OK and gather(row=0) == B.PA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,W,V,k", [(1, 1, 1, 1), (1, 4, 32000, 4), (3, 2, 100, 4), (2, 5, 777, 10), (7, 3, 50257, 3),
                                     (2, 16, 1000, 32), (1, 9, 33, 32), (5, 1, 4099, 1), (1, 40, 65, 32),
                                     (64, 4, 2048, 4)])
def test_topk_matches_definition(dtype, N, W, V, k):
    check(*random_case(N, W, V, dtype, N + W + V + k), k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_topk_ties_go_to_the_lowest_index(dtype):
    x = torch.zeros(2, 3, 5000, dtype=dtype)
    check(x, torch.zeros(2, 3), 32)            # every candidate equal
    x[:, :, 4000:4040] = 2.0                   # a run across lanes and batches
    check(x, torch.zeros(2, 3), 32)
    check(x, torch.tensor([[0.0, 0.0, -1.0], [-2.0, 0.0, 0.0]]), 20)


@pytest.mark.gpu
def test_topk_sorted_rows():
    """Ascending logits move the list at every step; descending ones never."""
    x = torch.arange(6000, dtype=torch.float32).view(1, 1, -1).repeat(1, 2, 1) * 0.01
    x[0, 1] = x[0, 1].flip(0)
    # The two rows hold the same values in another order, so their exact sums are equal and every
    # score comes twice; each row's sum is off by at most lse_error, which decides the order of
    # such a pair (the oracle's sums round as well).  Within a beam the order is that of the
    # logits whatever the sum is.
    rs, _, _ = reference(x, torch.zeros(1, 2), 32)
    s, p, t = select(x.cuda(), torch.zeros(1, 2).cuda(), 32)
    assert bool(((s.double() - rs).abs() <= lse_error(6000) + rs.abs() * 2.0 ** -24).all())
    for w, best in ((0, torch.arange(5999, 5983, -1)), (1, torch.arange(16))):
        assert torch.equal(t[p == w].long(), best)


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1, 5, 32])
@pytest.mark.parametrize("eos", [0, 3, 31, 32, 99])
def test_topk_finished_beams(k, eos):
    x, cum = random_case(3, 5, 100, torch.float32, k)
    fin = torch.tensor([[1, 0, 1, 0, 0], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0]], dtype=torch.bool)
    check(x, cum, k, fin, eos)
    check(x, cum * 100, k, fin.to(torch.uint8) * 3, eos)


@pytest.mark.gpu
def test_topk_beams_without_candidates():
    x, cum = random_case(4, 4, 300, torch.float32, 1)
    inf = float("inf")
    cum[0] = torch.tensor([0.0, -inf, -inf, -inf])   # the first step: one beam in use
    cum[1] = -inf
    x[2, 0, 7], x[2, 1, 5] = inf, float("nan")       # not finite: the beam is out
    x[2, 2] = -inf
    x[3, :, 10:] = -inf                              # tokens that are not allowed
    check(x, cum, 4)
    check(x, cum, 32)
    check(x.bfloat16(), cum, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_topk_extreme_logits(dtype):
    x, cum = random_case(2, 2, 3000, dtype, 3, spread=0.01)
    x[0, 0, 77] = 3e38
    x[0, 1] = -3e38
    x[1, 0] += 500
    check(x, cum, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("stride,offset", [(1003, 0), (1008, 0), (1008, 3), (2000, 8)])
def test_topk_strided_rows(dtype, stride, offset):
    x, cum = random_case(3, 4, 1003, dtype, stride)
    buf = torch.full((offset + 12 * stride,), float("nan"), dtype=dtype, device="cuda")
    d = buf[offset:offset + 12 * stride].view(3, 4, stride)[:, :, :1003]
    d.copy_(x)
    check(x, cum, 8, device_logits=d)


@pytest.mark.gpu
def test_topk_identical_beams_and_a_repeated_call():
    """The first step of a search whose beams are all alike: every tie goes to beam 0; twice the same."""
    x, cum = random_case(3, 1, 4000, torch.bfloat16, 8)
    x, cum = x.expand(3, 4, 4000).contiguous(), cum.expand(3, 4).contiguous()
    check(x, cum, 8)
    assert all(torch.equal(a, b) for a, b in zip(select(x.cuda(), cum.cuda(), 8), select(x.cuda(), cum.cuda(), 8)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_topk_rows_past_32_bits(dtype):
    """Rows that lie behind 2^31 elements of the logits."""
    N, W, V = 2, 2, 3000
    stride = (1 << 30) + 24
    buf = torch.empty(3 * stride + V, dtype=dtype, device="cuda")
    x, cum = random_case(N, W, V, dtype, 4)
    d = torch.as_strided(buf, (N, W, V), (2 * stride, stride, 1))
    d.copy_(x)
    check(x, cum, 4, device_logits=d)


@pytest.mark.gpu
@pytest.mark.parametrize("shape,dtype", [((7,), torch.int32), ((8, 16), torch.float32), ((3,), torch.uint8),
                                         ((5, 1, 3), torch.bfloat16), ((100003,), torch.int16)])
def test_gather(shape, dtype):
    N, W, k = 3, 4, 6
    src = torch.randint(0, 100, (N, W, *shape)).to(dtype).cuda()
    par = torch.randint(0, W, (N, k), dtype=torch.int32, device="cuda")
    dst = torch.empty(N, k, *shape, dtype=dtype, device="cuda")
    pa.pa_beam_gather(dst, src, par)
    assert torch.equal(dst, torch.stack([src[i][par[i].long()] for i in range(N)]))


@pytest.mark.gpu
def test_gather_bad_parent_and_empty():
    src = torch.arange(24, dtype=torch.float32, device="cuda").view(1, 4, 6)
    dst = torch.full((1, 3, 6), -1.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_beam_gather(dst, src, torch.tensor([[3, 4, -1]], dtype=torch.int32, device="cuda"), err_flag=err)
    assert int(err.item()) == B.PA_DEVERR_BAD_PARENT
    assert pa.pa_status_from_device_flag(int(err.item())) == B.PA_ERR_BAD_PARENT
    assert torch.equal(dst[0, 0], src[0, 3]) and bool((dst[0, 1:] == -1).all())
    pa.pa_beam_gather(torch.empty(0, 3, 6, device="cuda"), torch.empty(0, 4, 6, device="cuda"),
                      torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    pa.pa_beam_gather(torch.empty(1, 3, 0, device="cuda"), torch.empty(1, 4, 0, device="cuda"),
                      torch.zeros(1, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(pa.PAError):
        pa.pa_beam_gather(src, src, torch.zeros(1, 4, dtype=torch.int32, device="cuda"))


@pytest.mark.gpu
def test_topk_in_a_graph_follows_its_inputs():
    x, cum = random_case(4, 4, 5000, torch.bfloat16, 9)
    d, c = x.cuda(), cum.cuda()
    ws = torch.empty(pa.pa_beam_topk_workspace_size(4, 4, 5000, 4), dtype=torch.uint8, device="cuda")
    s = torch.empty(4, 4, device="cuda")
    p, t = (torch.empty(4, 4, dtype=torch.int32, device="cuda") for _ in range(2))
    pa.pa_beam_topk(s, p, t, d, c, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_beam_topk(s, p, t, d, c, workspace=ws)
    for seed in (10, 11):
        y, cum2 = random_case(4, 4, 5000, torch.bfloat16, seed)
        d.copy_(y)
        c.copy_(cum2)
        graph.replay()
        torch.cuda.synchronize()
        _, rp, rt = reference(y, cum2, 4)
        assert torch.equal(p.cpu(), rp) and torch.equal(t.cpu(), rt)


@pytest.mark.gpu
def test_topk_writes_over_the_scores_so_far():
    x, cum = random_case(5, 3, 9000, torch.float32, 12)
    d, c = x.cuda(), cum.cuda()
    ws = torch.empty(pa.pa_beam_topk_workspace_size(5, 3, 9000, 3), dtype=torch.uint8, device="cuda")
    s = torch.empty(5, 3, device="cuda")
    p, t, p2, t2 = (torch.empty(5, 3, dtype=torch.int32, device="cuda") for _ in range(4))
    pa.pa_beam_topk(s, p, t, d, c, workspace=ws)
    pa.pa_beam_topk(c, p2, t2, d, c, workspace=ws)
    assert torch.equal(s, c) and torch.equal(p, p2) and torch.equal(t, t2)
