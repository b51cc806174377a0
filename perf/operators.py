"""The operators that stand around the paged cache in a serving step: rotary positions with
the cache write, attention with capped, biased or masked scores for prompts and for single
tokens, and beam search's selection with the reordering of its states.

`listed()` and `draw()` describe cases, `prepare()` makes a case's inputs on the GPU, `run()`
makes one pass (elementary torch operations, or the library's calls where `own` is true),
`work()` counts what a pass cannot do without and `exact()` gives the results in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 256 sequences, whole heads rotated (the batch of the decode benchmark)
        dict(name="rope_step_256", op="rope", dtype="bf16", T=256, Hq=32, Hkv=8, D=128, bs=16, R=128,
             layout="half", scaling="none", far=4096, pad=0),
        # prompts' tokens of a few requests, half of the head rotated in interleaved pairs, context
        # stretched by the ramp; the tail of the token buffer is padding
        dict(name="rope_prompts_part", op="rope", dtype="bf16", T=16384, Hq=32, Hkv=8, D=128, bs=16,
             R=64, layout="interleaved", scaling="ramp", far=131072, pad=37),
        # a small fp32 model, odd token count, blocks of 4
        dict(name="rope_f32_odd", op="rope", dtype="f32", T=1023, Hq=6, Hkv=2, D=64, bs=4, R=48,
             layout="half", scaling="bands", far=32768, pad=5),

        # one sequence, one token: the latency of a single request's step
        dict(name="token_one_capped", op="attention", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, bs=16,
             n_lo=1, n_hi=1, c_lo=1000, c_hi=1000, softcap=50.0, bias=False, window=0, prefix=False,
             docs=False, shape_seed=1),
        # the decode benchmark's batch with capped scores and a sliding window
        dict(name="tokens_capped_window", op="attention", dtype="bf16", B=256, Hq=32, Hkv=8, D=128,
             bs=16, n_lo=1, n_hi=1, c_lo=63, c_hi=4095, softcap=50.0, bias=False, window=1024,
             prefix=False, docs=False, shape_seed=2),
        # the long-context batch with a distance bias
        dict(name="tokens_long_biased", op="attention", dtype="bf16", B=8, Hq=64, Hkv=8, D=128, bs=16,
             n_lo=1, n_hi=1, c_lo=32767, c_hi=131071, softcap=0.0, bias=True, window=0, prefix=False,
             docs=False, shape_seed=3),
        # prompts of equal length, capped scores
        dict(name="prompts_capped", op="attention", dtype="bf16", B=8, Hq=32, Hkv=8, D=128, bs=16,
             n_lo=2048, n_hi=2048, c_lo=0, c_hi=0, softcap=30.0, bias=False, window=0, prefix=False,
             docs=False, shape_seed=4),
        # one long prompt in which a prefix is seen by all and the rest through a window
        dict(name="prompt_long_prefix", op="attention", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, bs=16,
             n_lo=8192, n_hi=8192, c_lo=0, c_hi=0, softcap=0.0, bias=False, window=0, prefix=True,
             docs=False, shape_seed=5),
        # ragged chunks behind cached context, packed documents, distance bias, odd group of heads
        dict(name="chunks_documents", op="attention", dtype="bf16", B=6, Hq=14, Hkv=2, D=64, bs=32,
             n_lo=1, n_hi=700, c_lo=0, c_hi=3000, softcap=0.0, bias=True, window=0, prefix=False,
             docs=True, shape_seed=6),

        # one request with four beams
        dict(name="beam_one", op="beam", dtype="bf16", N=1, W=4, V=32000, k=4, finished=False, hist=128),
        # a batch of requests, scores in fp32
        dict(name="beam_batch", op="beam", dtype="f32", N=64, W=4, V=131072, k=4, finished=False,
             hist=1024),
        # odd vocabulary and beam count, some beams finished, twice as many candidates as beams
        dict(name="beam_odd_finished", op="beam", dtype="bf16", N=7, W=5, V=50257, k=10, finished=True,
             hist=77),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attention", "attention", "beam"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        D = rng.choice([64, 128])
        G, Hkv = rng.choice([1, 2, 3, 4, 7, 8]), rng.choice([1, 2, 4, 8])
        T = _log(rng, 1, 16384)
        return dict(op=op, dtype=dtype, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, bs=rng.choice([4, 8, 16, 32]),
                    R=rng.choice([D, D // 2, 16, 2 * rng.randint(1, D // 2)]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "ramp", "bands"]),
                    far=_log(rng, 128, 1 << 20), pad=rng.choice([0, 0, rng.randint(0, T // 8)]))
    if op == "beam":
        W = rng.choice([1, 2, 3, 4, 5, 8, 16])
        V = _log(rng, 100, 131072)
        N = _log(rng, 1, 64)
        while N * W * V > 64 * 4 * 131072:
            N = max(1, N // 2)
        return dict(op=op, dtype=dtype, N=N, W=W, V=V, k=rng.choice([W, W, min(2 * W, 32)]),
                    finished=rng.random() < 0.4, hist=_log(rng, 1, 1024))
    D = rng.choice([64, 128])
    G, Hkv = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]), rng.choice([1, 2, 4, 8])
    Hq = G * Hkv
    if rng.random() < 0.5:   # single tokens (now and then a few speculative ones)
        n_hi = rng.choice([1, 1, 1, 5])
        n_lo, c_hi = 1, _log(rng, 4, 131072)
        c_lo = rng.randint(0, c_hi)
        B = _log(rng, 1, 256)
        while B * (c_hi + n_hi) * Hkv * D > 8 * 131072 * 8 * 128 // 2:
            B = max(1, B // 2)
    else:
        n_hi = _log(rng, 2, 4096)
        n_lo, c_hi = rng.choice([n_hi, 1, 0]), rng.choice([0, 0, _log(rng, 1, 8192)])
        c_lo = rng.randint(0, c_hi)
        B = _log(rng, 1, 16)
        cap = (1 << 29) if dtype == "bf16" else (1 << 27)
        while B > 1 and B * Hq * n_hi * (c_hi + n_hi) > cap:
            B //= 2
        while n_hi > 2 and B * Hq * n_hi * (c_hi + n_hi) > cap:
            n_hi, c_hi = n_hi // 2, c_hi // 2
            n_lo, c_lo = min(n_lo, n_hi), min(c_lo, c_hi)
    mask = rng.choice(["causal", "causal", "window", "prefix", "docs"])
    score = rng.choice(["plain", "cap", "bias", "bias"])
    return dict(op=op, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, D=D, bs=rng.choice([4, 8, 16, 16, 32]),
                n_lo=n_lo, n_hi=n_hi, c_lo=c_lo, c_hi=c_hi,
                softcap=rng.choice([20.0, 30.0, 50.0]) if score == "cap" else 0.0,
                bias=score == "bias", window=_log(rng, 1, 4096) if mask == "window" else 0,
                prefix=mask == "prefix", docs=mask == "docs", shape_seed=rng.randrange(1 << 30))


# ---------------------------------------------------------------------------------------------
# shapes that follow from a case alone
# ---------------------------------------------------------------------------------------------

def _shape(case):
    """Per sequence: query tokens, length, prefix length; per query token: position, first visible key."""
    rng = random.Random(case["shape_seed"])
    B = case["B"]

    def pick(lo, hi):
        return lo if lo == hi else (rng.randint(0, 3) if lo == 0 and rng.random() < 0.1
                                    else min(hi, max(lo, _log(rng, max(lo, 1), hi))))
    n = [pick(case["n_lo"], case["n_hi"]) for _ in range(B)]
    if sum(n) == 0:
        n[0] = 1
    L = [a + pick(case["c_lo"], case["c_hi"]) for a in n]
    pre = [rng.randint(0, x) if case["prefix"] else 0 for x in L]
    first = []
    for a, x in zip(n, L):
        f = np.zeros(a, np.int64)
        if case["docs"]:
            start, starts = 0, []
            while start < x:
                starts.append(start)
                start += max(1, _log(rng, 1, 1500))
            pos = np.arange(x - a, x)
            f = np.asarray(starts, np.int64)[np.searchsorted(np.asarray(starts), pos, side="right") - 1]
        first.append(f)
    return n, L, pre, first


def _visible(case):
    """(sum over query tokens of visible keys, sum over sequences of keys that any of them sees)."""
    n, L, pre, first = _shape(case)
    rows = keys = 0
    for a, x, pr, f in zip(n, L, pre, first):
        if not a:
            continue
        pos = np.arange(x - a, x)
        hi = np.minimum(np.maximum(pos + 1, pr), x)
        lo = np.maximum(f, np.maximum(0, pos + 1 - case["window"]) if case["window"] else 0)
        rows += int(np.maximum(hi - lo, 0).sum())
        seen = np.zeros(x + 1, np.int64)
        np.add.at(seen, lo, 1)
        np.add.at(seen, np.maximum(hi, lo), -1)
        keys += int((np.cumsum(seen)[:x] > 0).sum())
    return rows, keys


def work(case):
    e = ESIZE[case["dtype"]]
    if case["op"] == "rope":
        T, row = case["T"], (case["Hq"] + 2 * case["Hkv"]) * case["D"] * e
        live = T - case["pad"]
        moved = T * (row + 12) + T * case["Hq"] * case["D"] * e + live * 2 * case["Hkv"] * case["D"] * e
        return {"bytes": moved, "flops": live * (case["Hq"] + case["Hkv"]) * case["R"] * 3}
    if case["op"] == "beam":
        N, W, V, k = case["N"], case["W"], case["V"], case["k"]
        return {"bytes": N * W * V * e + N * W * 4 + N * k * 12 + 2 * N * k * case["hist"] * 4,
                "flops": 4 * N * W * V}
    rows, keys = _visible(case)
    n, L, _, _ = _shape(case)
    T, D = sum(n), case["D"]
    tables = sum((x + case["bs"] - 1) // case["bs"] for x in L) * 4
    return {"bytes": 2 * T * case["Hq"] * D * e + keys * case["Hkv"] * D * 2 * e + tables + 8 * case["B"],
            "flops": 4 * D * case["Hq"] * rows}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _frequencies(case):
    """Angle per position of each rotated pair (64 bits, host) and the factor on cos and sin."""
    R, base, s, old = case["R"], 10000.0, 8.0, 4096.0
    i = np.arange(R // 2, dtype=np.float64)
    f = base ** (-2.0 * i / R)
    kind = case["scaling"]
    if kind == "linear":          # positions interpolated
        return f / s, 1.0
    if kind == "base":            # the base stretched so that the slowest pair is interpolated by s
        return (base * s ** (R / max(R - 2, 1))) ** (-2.0 * i / R), 1.0
    turns = old * f / (2 * math.pi)
    if kind == "ramp":            # pairs with many turns kept, with few interpolated, a ramp between
        dim = lambda b: R * math.log(old / (b * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), R - 1)
        keep = 1.0 - np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / s * (1 - keep) + f * keep, 0.1 * math.log(s) + 1.0
    if kind == "bands":           # the same by bands of wavelength: 1 turn and 4 turns in the old length
        smooth = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return f / s * (1 - smooth) + f * smooth, 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, dev = DT[case["dtype"]], "cuda"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    st = {"case": dict(case)}
    if case["op"] == "rope":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        NB = (T + case["bs"] - 1) // case["bs"] + 3
        # the projection's output: q, k and v of a token side by side
        qkv = normal(T, (Hq + 2 * Hkv) * D)
        st["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        st["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        st["k_pool"], st["v_pool"] = normal(NB, case["bs"], Hkv, D), normal(NB, case["bs"], Hkv, D)
        st["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=dev, dtype=torch.int32)
        slots = torch.randperm(NB * case["bs"], generator=g, device=dev)[:T].contiguous()
        slots[T - case["pad"]:] = -1
        st["slots"] = slots
        st["live"] = T - case["pad"]
        f, st["factor"] = _frequencies(case)
        st["inv_freq"] = torch.from_numpy(np.ascontiguousarray(f)).to(dev)
        st["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
        st["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
        return st
    if case["op"] == "beam":
        N, W, V = case["N"], case["W"], case["V"]
        # a model's logits: a spread of a few units, one shared part per request
        x = torch.randn(N, 1, V, generator=g, device=dev) * 1.5 + torch.randn(N, W, V, generator=g, device=dev) * 2.0
        st["logits"] = x.to(dt)
        st["cum"] = -torch.rand(N, W, generator=g, device=dev) * 8.0 - 4.0
        st["eos"] = V // 2
        st["finished"] = None
        if case["finished"]:
            st["finished"] = torch.rand(N, W, generator=g, device=dev) < 0.3
        st["history"] = torch.randint(0, V, (N, W, case["hist"]), generator=g, device=dev, dtype=torch.int32)
        return st
    n, L, pre, first = _shape(case)
    B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
    T = sum(n)
    nblk = [(x + bs - 1) // bs for x in L]
    NB = sum(nblk) + max(1, sum(nblk) // 10)
    MB = max(max(nblk), 1)
    ids = torch.randperm(NB, generator=g, device=dev).to(torch.int32)
    tables = np.full((B, MB), -1, np.int64)
    at = 0
    for b, m in enumerate(nblk):
        tables[b, :m] = np.arange(at, at + m)
        at += m
    tab = torch.from_numpy(tables).to(dev)
    st["tables"] = torch.where(tab >= 0, ids[tab.clamp_min(0)], tab.to(torch.int32)).contiguous()
    st["k_pool"], st["v_pool"] = normal(NB, bs, Hkv, D), normal(NB, bs, Hkv, D)
    # scores of a unit's spread, four where a cap is to matter
    st["q"] = normal(T, Hq, D) * (4.0 if case["softcap"] else 1.0)
    st["out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
    st["scale"] = 1.0 / math.sqrt(D)
    st["lens"] = torch.tensor(L, dtype=torch.int32, device=dev)
    st["starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(dev)
    st["n"], st["L"] = n, L
    st["slopes"] = None
    if case["bias"]:
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32,
                                    device=dev)
    st["prefix"] = torch.tensor(pre, dtype=torch.int32, device=dev) if case["prefix"] else None
    st["first"] = torch.from_numpy(np.concatenate(first).astype(np.int32)).to(dev) if case["docs"] else None
    st["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return st


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _plain_rope(st):
    c = st["case"]
    R, D = c["R"], c["D"]
    t = st["positions"].to(torch.float64)[:, None] * st["inv_freq"][None, :]
    t = torch.remainder(t, 2 * math.pi)
    cos = (torch.cos(t) * st["factor"]).to(torch.float32)[:, None, :]
    sin = (torch.sin(t) * st["factor"]).to(torch.float32)[:, None, :]

    def turn(x):
        y = x.to(torch.float32).clone()
        a, b = ((y[..., 0:R:2], y[..., 1:R:2]) if c["layout"] == "interleaved"
                else (y[..., :R // 2], y[..., R // 2:R]))
        na, nb = a * cos - b * sin, a * sin + b * cos
        if c["layout"] == "interleaved":
            y[..., 0:R:2], y[..., 1:R:2] = na, nb
        else:
            y[..., :R // 2], y[..., R // 2:R] = na, nb
        return y.to(x.dtype)
    st["q_out"].copy_(turn(st["q"]))
    live = st["live"]   # the padded tokens come last
    slots = st["slots"][:live]
    st["k_pool"].view(-1, c["Hkv"], D)[slots] = turn(st["k"])[:live]
    st["v_pool"].view(-1, c["Hkv"], D)[slots] = st["v"][:live]
    return st["q_out"], st["k_pool"], st["v_pool"]


def _plain_attention(st):
    c = st["case"]
    B, Hq, Hkv, D, bs = c["B"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    G, dev = Hq // Hkv, st["q"].device
    nmax, Lmax = max(st["n"]), max(max(st["L"]), 1)
    lens, starts = st["lens"].long(), st["starts"].long()
    count = starts[1:] - starts[:-1]
    # keys and values of every sequence side by side, padded
    j = torch.arange(Lmax, device=dev)
    have = j[None, :] < lens[:, None]
    block = st["tables"].long()[:, (j // bs).clamp_max(st["tables"].shape[1] - 1)]
    slot = torch.where(have, block * bs + j % bs, 0)
    K = st["k_pool"].view(-1, Hkv, D)[slot].to(torch.float32)
    V = torch.where(have[:, :, None, None], st["v_pool"].view(-1, Hkv, D)[slot].to(torch.float32), 0.0)
    # query tokens, padded; i runs over a sequence's own
    i = torch.arange(nmax, device=dev)
    real = i[None, :] < count[:, None]
    token = torch.where(real, starts[:-1, None] + i[None, :], 0)
    pos = (lens - count)[:, None] + i[None, :]
    Q = st["q"][token].to(torch.float32).view(B, nmax, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nmax, D)
    x = torch.matmul(Q * st["scale"], K.permute(0, 2, 3, 1)).view(B, Hkv, G, nmax, Lmax)
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    dist = pos[:, :, None] - j[None, None, :]
    if st["slopes"] is not None:
        x = x - st["slopes"].view(1, Hkv, G, 1, 1) * dist.abs()[:, None, None].to(torch.float32)
    see = dist >= 0
    if st["prefix"] is not None:
        see = see | (j[None, None, :] < st["prefix"].long()[:, None, None])
    if c["window"]:
        see = see & (dist < c["window"])
    if st["first"] is not None:
        see = see & (j[None, None, :] >= st["first"].long()[token][:, :, None])
    see = see & have[:, None, :] & real[:, :, None] & (pos >= 0)[:, :, None]
    x = x.masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    del x
    total = p.sum(-1).view(B, Hkv, G * nmax, 1)
    o = torch.matmul(p.view(B, Hkv, G * nmax, Lmax), V.permute(0, 2, 1, 3))
    o = torch.where(total > 0, o / total.clamp_min(1e-37), 0.0)
    o = o.view(B, Hkv, G, nmax, D).permute(0, 3, 1, 2, 4).reshape(B * nmax, Hq, D)
    # a padded token's row goes to a spare one behind the last
    T = st["q"].shape[0]
    to = torch.where(real, token, T).view(-1)
    out = torch.empty(T + 1, Hq, D, dtype=st["q"].dtype, device=dev)
    out[to] = o.to(out.dtype)
    return out[:T]


def _plain_beam(st):
    c = st["case"]
    N, W, V, k = c["N"], c["W"], c["V"], c["k"]
    x = st["logits"].to(torch.float64)   # neighbours on the border differ by less than 32 bits hold
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    s = st["cum"].to(torch.float64)[:, :, None] + (x - lse)
    if st["finished"] is not None:
        done = st["finished"][:, :, None]
        keep = torch.arange(V, device=x.device)[None, None, :] == st["eos"]
        s = torch.where(done, torch.where(keep, st["cum"].to(torch.float64)[:, :, None], -math.inf), s)
    s, at = torch.sort(s.view(N, W * V), dim=-1, descending=True, stable=True)
    s, at = s[:, :k], at[:, :k]
    parent = at // V
    history = torch.gather(st["history"], 1, parent[:, :, None].expand(N, k, c["hist"]))
    return s.to(torch.float32), parent.to(torch.int32), (at % V).to(torch.int32), history


def _own(st):
    import paged_kv_cache_350_b200 as pa
    c = st["case"]
    if c["op"] == "rope":
        layout = pa.PA_ROPE_INTERLEAVED if c["layout"] == "interleaved" else pa.PA_ROPE_HALF
        pa.pa_rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["k_pool"], st["v_pool"],
                             st["positions"], st["slots"], st["inv_freq"], layout=layout,
                             attn_factor=st["factor"], err_flag=st["err"])
        return st["q_out"], st["k_pool"], st["v_pool"]
    if c["op"] == "attention":
        most = max(st["n"])
        if "ws" not in st:   # kept, as a serving program keeps its workspace
            size = pa.pa_attention_workspace_size(st["q"].shape[0], c["B"], most, c["Hq"], c["Hkv"], c["D"],
                                                  c["bs"], st["tables"].shape[1])
            st["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device=st["q"].device)
        pa.pa_attention(st["out"], st["q"], st["k_pool"], st["v_pool"], st["tables"], st["lens"],
                        st["starts"], most, st["scale"], softcap=c["softcap"], alibi_slopes=st["slopes"],
                        window=c["window"], prefix_lens=st["prefix"], first_keys=st["first"],
                        workspace=st["ws"], err_flag=st["err"])
        return st["out"]
    N, k = c["N"], c["k"]
    if "ws" not in st:
        dev = st["logits"].device
        size = pa.pa_beam_topk_workspace_size(N, c["W"], c["V"], k)
        st["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
        st["best"] = (torch.empty(N, k, dtype=torch.float32, device=dev),
                      torch.empty(N, k, dtype=torch.int32, device=dev),
                      torch.empty(N, k, dtype=torch.int32, device=dev))
        st["moved"] = torch.empty(N, k, c["hist"], dtype=torch.int32, device=dev)
    scores, parents, tokens = st["best"]
    pa.pa_beam_topk(scores, parents, tokens, st["logits"], st["cum"], finished=st["finished"],
                    eos_token=st["eos"], workspace=st["ws"])
    pa.pa_beam_gather(st["moved"], st["history"], parents)
    return scores, parents, tokens, st["moved"]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "attention": _plain_attention, "beam": _plain_beam}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_rope(st):
    c = st["case"]
    D, half = c["D"], c["R"] // 2
    # the rotation as a complex product per pair
    first = [2 * i if c["layout"] == "interleaved" else i for i in range(half)]
    second = [2 * i + 1 if c["layout"] == "interleaved" else i + half for i in range(half)]
    angle = torch.outer(st["positions"].double(), st["inv_freq"])
    unit = torch.polar(torch.full_like(angle, st["factor"]), angle)

    def turn(x):
        y = x.double().clone()
        z = torch.complex(y[:, :, first], y[:, :, second]) * unit[:, None, :]
        y[:, :, first], y[:, :, second] = z.real, z.imag
        return y
    kp, vp = st["k_pool"].double(), st["v_pool"].double()
    live = c["T"] - c["pad"]
    s = st["slots"][:live]
    kp[s // c["bs"], s % c["bs"]] = turn(st["k"])[:live]
    vp[s // c["bs"], s % c["bs"]] = st["v"].double()[:live]
    return turn(st["q"]), kp, vp


def _exact_attention(st):
    c = st["case"]
    G, bs = c["Hq"] // c["Hkv"], c["bs"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    t0 = 0
    pre = st["prefix"].tolist() if st["prefix"] is not None else None
    for b, (n, L) in enumerate(zip(st["n"], st["L"])):
        if n and L:
            blocks = st["tables"][b, :(L + bs - 1) // bs].long()
            for h in range(c["Hkv"]):
                k = st["k_pool"][blocks, :, h].double().flatten(0, 1)[:L]
                v = st["v_pool"][blocks, :, h].double().flatten(0, 1)[:L]
                for r0 in range(0, n, 1024):
                    r1 = min(n, r0 + 1024)
                    at = torch.arange(L - n + r0, L - n + r1, device="cuda")[:, None]
                    key = torch.arange(L, device="cuda")[None, :]
                    hidden = key > at
                    if pre:
                        hidden = hidden & (key >= pre[b])
                    if c["window"]:
                        hidden = hidden | (key <= at - c["window"])
                    if st["first"] is not None:
                        hidden = hidden | (key < st["first"][t0 + r0:t0 + r1].long()[:, None])
                    for e in range(h * G, h * G + G):
                        s = (st["q"][t0 + r0:t0 + r1, e].double() @ k.T) * st["scale"]
                        if c["softcap"]:
                            s = torch.tanh(s / c["softcap"]) * c["softcap"]
                        if st["slopes"] is not None:
                            s = s - float(st["slopes"][e]) * (at - key).abs().double()
                        s[hidden] = -math.inf
                        w = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
                        out[t0 + r0:t0 + r1, e] = w @ v
        t0 += n
    return out


def _exact_beam(st):
    c = st["case"]
    scores, parents, tokens = [], [], []
    for i in range(c["N"]):
        logp = torch.log_softmax(st["logits"][i].double(), -1)
        if st["finished"] is not None:
            for w in torch.nonzero(st["finished"][i]).flatten().tolist():
                logp[w] = -math.inf
                logp[w, st["eos"]] = 0.0
        s = (logp + st["cum"][i].double()[:, None]).flatten()
        top = torch.topk(s, min(s.numel(), 4 * c["k"])).values.min()
        near = torch.nonzero(s >= top).flatten().tolist()
        value = s[near].tolist() if near else []
        best = sorted(zip(value, near), key=lambda p: (-p[0], p[1]))[:c["k"]]
        scores.append([p[0] for p in best])
        parents.append([p[1] // c["V"] for p in best])
        tokens.append([p[1] % c["V"] for p in best])
    par = torch.tensor(parents, dtype=torch.int32, device="cuda")
    moved = torch.stack([st["history"][i][par[i].long()] for i in range(c["N"])])
    return (torch.tensor(scores, dtype=torch.float64, device="cuda"), par,
            torch.tensor(tokens, dtype=torch.int32, device="cuda"), moved)


def exact(case, seed):
    with torch.no_grad():
        return {"rope": _exact_rope, "attention": _exact_attention, "beam": _exact_beam}[case["op"]](
            prepare(case, seed))
