"""Attention with caps over their whole range and with far positions, against the formula in 64
bits: tolerances grow neither with the cap nor with the position."""

import math

import pytest
import torch

import paged_kv_cache_350_b200 as pa
from test_attention import Case

ULP = 2.0 ** -24   # half a step of 32 bits


class Capped(Case):
    """A causal batch whose tokens' queries have spreads of their own."""

    def __init__(self, *a, spreads=(1.0,), **kw):
        super().__init__(*a, **kw)
        for t in range(self.q.shape[0]):
            self.q[t] *= spreads[t % len(spreads)]

    def score_error(self, x):
        """How far a capped score may be from c tanh(x / c), beside the error of x itself (tanh does
        not enlarge that).  fp32: the constants scale / c and c, and two products, are four half
        steps, tanhf at most 2 ulp, four more.  bf16: the same constants and products; up to 64 the
        formulas' errors are absolute, below 1e-6 of the cap; past it relative: a series
        truncated at 2.4e-7, at most 4 half steps, or 1 - 2 / (1 + e^2t) from t = 0.35 on, where
        exponential, reciprocal and sum are 5.4 half steps of the cap, 16 of tanh(0.35)."""
        rel = x.abs() * 8 * ULP
        if self.softcap == 0 or self.dtype == "f32":
            return rel
        return rel + (self.softcap * 1e-6 if self.softcap <= 64 else x.abs() * 16 * ULP)

    def reference(self):
        T, G = int(self.starts[-1]), self.Hq // self.Hkv
        out = torch.zeros(T, self.Hq, self.D, dtype=torch.float64)
        size, dx = torch.zeros_like(out), torch.zeros(T, self.Hq, 1, dtype=torch.float64)
        for b, n in enumerate(self.n):
            t0, L = int(self.starts[b]), self.L[b]
            if n == 0:
                continue
            pos, key = torch.arange(L - n, L)[:, None], torch.arange(L)[None, :]
            for h in range(self.Hq):
                q, k, v = self.q[t0:t0 + n, h].double(), self.keys[b][:, h // G], self.values[b][:, h // G]
                x = q @ k.T * self.scale
                # sums over D in 32 bits in any order, 2^-22 a step
                d = q.abs() @ k.abs().T * abs(self.scale) * (self.D + 4) * 2.0 ** -22
                if self.softcap:
                    x = self.softcap * torch.tanh(x / self.softcap)
                d = d + self.score_error(x)
                if self.slopes is not None:
                    bias = float(self.slopes[h]) * (pos - key).abs().double()
                    x, d = x - bias, d + (bias + x.abs()) * 4 * ULP
                w = torch.softmax(x.masked_fill(key > pos, -math.inf), -1)
                out[t0:t0 + n, h], size[t0:t0 + n, h] = w @ v, w @ v.abs()
                # (close doubles it) the weights' errors e^d - 1, those of the sum among them
                dx[t0:t0 + n, h, 0] = torch.expm1((w * d).sum(-1) + (w * d).amax(-1))
        return out, size, dx


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [50.0, 64.0, 65.0, 1e3, 1e5, 1e6, 1e8, 1e30])
@pytest.mark.parametrize("n", [[8, 1], [9, 3, 150]])   # 16 rows, the most of the kernels for few, and 18
def test_caps_up_to_no_cap(dtype, cap, n):
    L = [300, 77, 200][:len(n)]
    for D, spreads, bias in ((64, (1.0,), False), (128, (1.0, 300.0, 0.01), False), (64, (4.0, 2e4), True)):
        Capped(dtype, n, L, 4, 2, D, 16, softcap=cap, spreads=spreads, bias=bias, seed=D).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [[1, 1], [40, 1]])
def test_a_cap_past_all_scores_is_no_cap(dtype, n):
    plain = Capped(dtype, n, [300, 90], 8, 2, 128, 16)
    got, (args, kw) = Capped(dtype, n, [300, 90], 8, 2, 128, 16, softcap=1e30).run()
    plain.close(got)
    c = Capped(dtype, n, [300, 90], 8, 2, 128, 16, softcap=1e4)
    c.scale = -c.scale
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,Hq", [(1, 4), (3, 4), (20, 4)])
def test_a_bias_past_2_24_positions(dtype, n, Hq):
    """A sequence of 2^25 keys over a table that goes round a few blocks: neighbouring keys are told
    apart by their distances."""
    bs, D, blocks, tail = 32, 64, 5, 4096
    L = (1 << 25) + 77
    g = torch.Generator().manual_seed(n)
    kp, vp = (torch.randn(blocks, bs, 1, D, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(n, Hq, D, generator=g).to(dtype)
    slopes = torch.tensor([1.0, 0.5, 0.25, 0.125][:Hq])
    MB = -(-L // bs)
    table = (torch.arange(MB, dtype=torch.int32) % blocks)[None]
    out = torch.empty(n, Hq, D, dtype=dtype, device="cuda")
    ws = torch.empty(pa.pa_attention_workspace_size(n, 1, n, Hq, 1, D, bs, MB), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_attention(out, q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), torch.tensor([L], dtype=torch.int32).cuda(),
                    torch.tensor([0, n], dtype=torch.int32).cuda(), n, D ** -0.5, alibi_slopes=slopes.cuda(),
                    workspace=ws, err_flag=err)
    got = out.cpu().double()
    assert int(err.item()) == 0
    # keys before the last `tail` weigh less than e^(largest score difference - slope * tail) each
    key = torch.arange(L - tail, L)
    rows = key // bs % blocks * bs + key % bs
    k, v = kp.view(-1, D)[rows].double(), vp.view(-1, D)[rows].double()
    pos = torch.arange(L - n, L)[:, None]
    for h in range(Hq):
        x = q[:, h].double() @ k.T * D ** -0.5
        assert L * math.exp(2 * float(x.abs().max()) - 0.125 * (tail - n)) < 1e-100
        bias = float(slopes[h]) * (pos - key).abs().double()
        d = q[:, h].double().abs() @ k.abs().T * D ** -0.5 * (D + 4) * 2.0 ** -22 + (x.abs() + 2 * bias) * 4 * ULP
        w = torch.softmax((x - bias).masked_fill(key > pos, -math.inf), -1)
        ref, size = w @ v, w @ v.abs()
        off = torch.expm1((w * d).sum(-1, keepdim=True) + (w * d).amax(-1, keepdim=True))
        half = torch.finfo(dtype).eps / 2
        # weights rounded to bf16 for their product, the output; sums over the keys that have a weight
        tol = size * (2 * off + (tail + 8) * ULP + 2.0 ** -20 + (half if dtype == torch.bfloat16 else 0)) + ref.abs() * half
        assert bool(((got[:, h] - ref).abs() <= tol).all()), float(((got[:, h] - ref).abs() / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [1e3, 1e6, 1e30])
def test_wide_caps_of_wide_groups_and_of_large_batches(cap):
    """The CUDA-core kernel: more than 128 heads a group, and fp32 batches of more sequences than are scanned."""
    Capped("bf16", [3, 1], [50, 200], 130, 1, 64, 16, softcap=cap, spreads=(1.0, 300.0)).check()
    Capped("f32", [1] * 2100, [1 + i % 40 for i in range(2100)], 2, 1, 64, 8, softcap=cap).check()
    # and the tensor cores, where units are taken one by one
    n = [33 if i % 7 else 0 for i in range(190)]
    Capped("bf16", n, [a + (i * 37) % 150 for i, a in enumerate(n)], 16, 8, 64, 16, softcap=cap,
           spreads=(1.0, 300.0)).check()
