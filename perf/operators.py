"""The operators around the router that the framework's users call next to
routing, as measurable cases: the norm that makes the router's input (with the
residual's addition and an 8-bit output for the experts) and its gradient, the
balance loss with its per-expert counts and gradient, and the expert layer on
8-bit operands.

``own = False``: the plain forms, elementary torch operations in 32 bits (64
for long sums).  ``own = True``: the framework's calls on the same inputs.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
GROUP = 128          # columns per 8-bit scale; weight blocks are GROUP x GROUP
E4M3_MAX = 448.0
AMAX_MIN = 1e-30     # a smaller group maximum counts as this
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a decode step: latency only
        dict(name="norm_decode_1", op="norm", N=1, d=2560, x="bf16", res="bf16", y=True, fp8=True),
        # a prefill of 16384 tokens before the router and the 8-bit experts
        dict(name="norm_prefill_16384", op="norm", N=16384, d=2560, x="bf16", res="bf16", y=True, fp8=True),
        # a training batch of the narrower model, fp32 residual stream, bf16 output only
        dict(name="norm_train_65536", op="norm", N=65536, d=2048, x="bf16", res="f32", y=True, fp8=False),
        # backward of a microbatch, the residual's gradient added
        dict(name="norm_grad_16384", op="norm_grad", N=16384, d=2560, h="bf16", gy="bf16", gres=True),
        # a short ragged batch with fp32 streams
        dict(name="norm_grad_ragged_333", op="norm_grad", N=333, d=2048, h="f32", gy="f32", gres=False),
        # a small batch as one sequence: loss and gradient in one call
        dict(name="balance_256", op="balance", N=256, E=384, K=6, S=1, score="sigmoid", fused=True, pad=0),
        # packed documents of uneven lengths with padding behind them, softmax scores; the gradient in the backward pass
        dict(name="balance_packed_65536", op="balance", N=65536, E=128, K=8, S=61, score="softmax", fused=False, pad=117),
        # the million-token batch as one sequence
        dict(name="balance_1m", op="balance", N=1 << 20, E=384, K=6, S=1, score="sigmoid", fused=True, pad=0),
        # decode: one token through seven experts
        dict(name="experts_decode_1", op="experts", N=1, d=2560, F=512, E=384, K=6, shared=True),
        # decode of 64 requests: about one row per expert, the weights are what is read
        dict(name="experts_decode_64", op="experts", N=64, d=2560, F=512, E=384, K=6, shared=True),
        # a prefill chunk on the narrower shape without a shared expert, odd token count
        dict(name="experts_chunk_2049", op="experts", N=2049, d=2048, F=512, E=128, K=8, shared=False),
        # a prefill microbatch of the full layer
        dict(name="experts_prefill_16384", op="experts", N=16384, d=2560, F=512, E=384, K=6, shared=True),
    ]


def _spread(rng, lo, hi):
    """An integer in [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "balance", "experts"])
    if op == "norm":
        d = 8 * _spread(rng, 64, 512)
        fp8 = rng.random() < 0.7
        return dict(op=op, N=_spread(rng, 1, 40_000_000 // d), d=d, x=rng.choice(["bf16", "f32"]),
                    res=rng.choice(["none", "bf16", "f32"]), y=not fp8 or rng.random() < 0.7, fp8=fp8)
    if op == "norm_grad":
        d = 8 * _spread(rng, 64, 512)
        return dict(op=op, N=_spread(rng, 1, 20_000_000 // d), d=d, h=rng.choice(["bf16", "f32"]),
                    gy=rng.choice(["bf16", "f32"]), gres=rng.random() < 0.5)
    if op == "balance":
        E = 4 * _spread(rng, 2, 128)
        N = _spread(rng, 1, 400000)
        return dict(op=op, N=N, E=E, K=rng.randint(1, min(8, E - 1)), S=_spread(rng, 1, min(100, N)),
                    score=rng.choice(["sigmoid", "softmax"]), fused=rng.random() < 0.5, pad=rng.choice([0, 0, 5, 300]))
    return dict(op=op, N=_spread(rng, 1, 12000), d=256 * rng.randint(2, 10), F=128 * rng.randint(2, 6), E=32 * rng.randint(1, 8),
                K=rng.randint(1, 8), shared=rng.random() < 0.6)


# ---------------------------------------------------------------- inputs

def _quantise_blocks(w):
    """[..., r, c] -> e4m3 values and one scale per GROUP x GROUP block."""
    *lead, r, c = w.shape
    v = w.view(*lead, r // GROUP, GROUP, c // GROUP, GROUP)
    s = v.abs().amax(dim=(-3, -1)).float().clamp_min(AMAX_MIN) / E4M3_MAX
    return (v / s[..., :, None, :, None].to(w.dtype)).clamp(-E4M3_MAX, E4M3_MAX).to(F8).view(w.shape), s.contiguous()


def _quantise_rows(x):
    n, c = x.shape
    v = x.float().view(n, c // GROUP, GROUP)
    s = v.abs().amax(-1).clamp_min(AMAX_MIN) / E4M3_MAX
    return (v / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8).view(n, c), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    st = dict(case)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device=dev, dtype=dtype)

    op = case["op"]
    if op == "norm":
        N, d = case["N"], case["d"]
        # the residual stream is wider than a layer's output, and some channels are much wider
        wide = torch.exp(randn(d) * 0.7)
        st["x"] = randn(N, d).to(TYPES[case["x"]])
        st["r"] = None if case["res"] == "none" else (randn(N, d) * wide * 2.0).to(TYPES[case["res"]])
        st["g"] = (1.0 + 0.2 * randn(d)).to(torch.bfloat16)
        st["res_out"] = None if st["r"] is None else torch.empty_like(st["r"])
        st["out"] = empty(N, d, dtype=torch.bfloat16) if case["y"] else None
        st["out8"] = empty(N, d, dtype=F8) if case["fp8"] else None
        st["scales"] = empty(N, -(-d // GROUP)) if case["fp8"] else None
    elif op == "norm_grad":
        N, d = case["N"], case["d"]
        wide = torch.exp(randn(d) * 0.7)
        st["hid"] = (randn(N, d) * wide * 2.0).to(TYPES[case["h"]])
        st["dy"] = (randn(N, d) * 0.01).to(TYPES[case["gy"]])
        st["dres"] = (randn(N, d) * 0.01).to(TYPES[case["h"]]) if case["gres"] else None
        st["g"] = (1.0 + 0.2 * randn(d)).to(torch.bfloat16)
        st["gx"] = torch.empty_like(st["hid"])
        st["gg"] = empty(d)
    elif op == "balance":
        N, E, K, S = case["N"], case["E"], case["K"], case["S"]
        z = randn(N, E) + 0.7 * randn(E)          # some experts are liked more: uneven loads
        st["z"] = z
        st["ids"] = torch.topk(z + 0.3 * randn(E), K, dim=1).indices.to(torch.int32)
        used = max(N - case["pad"], S)
        cuts = torch.sort(torch.randint(0, used + 1, (S - 1,), generator=g, device=dev)).values
        ends = torch.tensor([0, used], device=dev)
        st["seq"] = torch.cat([ends[:1], cuts, ends[1:]])[: S + 1].to(torch.int64).contiguous()
        st["lam"] = 1e-3
        st["up"] = (0.5 + torch.rand(S, generator=g, device=dev))       # dL_total / dL_s
        st["gz"] = empty(N, E)
        st["loss"], st["counts"], st["prob"] = empty(S), empty(S, E, dtype=torch.int32), empty(S, E)
    else:
        N, d, F, E, K = (case[k] for k in ("N", "d", "F", "E", "K"))
        st["x8"], st["xs"] = _quantise_rows(randn(N, d))
        score = randn(N, E) + 0.15 * randn(E)
        top = torch.topk(score, K, dim=1)
        ids = top.indices
        st["gates"] = torch.sigmoid(top.values).contiguous()
        flat = ids.reshape(-1)
        perm = torch.argsort(flat, stable=True)
        inv = torch.empty_like(perm)
        inv[perm] = torch.arange(N * K, device=dev)
        counts = torch.bincount(flat, minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int64, device=dev)
        offsets[1:] = torch.cumsum(counts, 0)
        st["ids"], st["perm"], st["inv"], st["offsets"] = ids.contiguous(), perm.to(torch.int32), inv.to(torch.int32), offsets
        st["most"] = int(counts.max())
        st["wgu"], st["sgu"] = _quantise_blocks(randn(E, 2 * F, d, dtype=torch.bfloat16) * d ** -0.5)
        st["wd"], st["sd"] = _quantise_blocks(randn(E, d, F, dtype=torch.bfloat16) * F ** -0.5)
        if case["shared"]:
            st["wgu_s"], st["sgu_s"] = _quantise_blocks(randn(2 * F, d, dtype=torch.bfloat16) * d ** -0.5)
            st["wd_s"], st["sd_s"] = _quantise_blocks(randn(d, F, dtype=torch.bfloat16) * F ** -0.5)
        else:
            st["wgu_s"] = st["sgu_s"] = st["wd_s"] = st["sd_s"] = None
        st["y"] = empty(N, d, dtype=torch.bfloat16)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    return {"norm": _norm, "norm_grad": _norm_grad, "balance": _balance, "experts": _experts}[state["op"]](state)


def _norm(st):
    if own:
        from expert_load_balancing_b200 import binding as B
        res_out, y, y8, scales = B.kolibri_rms_norm(
            st["x"], st["g"], EPS, res=st["r"], res_out=st["res_out"], y=st["out"], y8=st["out8"], scales=st["scales"],
            want_y=st["out"] is not None, want_fp8=st["out8"] is not None)
        return dict(res=res_out, y=y, y8=y8, scales=scales)
    h = st["x"].float()
    if st["r"] is not None:
        h = h + st["r"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["g"].float()
    out = dict(res=None if st["r"] is None else h.to(st["r"].dtype), y=y.to(torch.bfloat16) if st["out"] is not None else None,
               y8=None, scales=None)
    if st["out8"] is not None:
        N, d = y.shape
        v = torch.nn.functional.pad(y, (0, -d % GROUP)).view(N, -1, GROUP)
        s = v.abs().amax(-1).clamp_min(AMAX_MIN) / E4M3_MAX
        out["scales"] = s
        out["y8"] = (v / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(N, -1)[:, :d].to(F8)
    return out


def _norm_grad(st):
    if own:
        from expert_load_balancing_b200 import binding as B
        gx, gg = B.kolibri_rms_norm_grad(st["dy"], st["hid"], st["g"], EPS, gres=st["dres"], gx=st["gx"], gweight=st["gg"])
        return dict(gx=gx, gg=gg)
    h, dy, g = st["hid"].float(), st["dy"].float(), st["g"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    xh = h * r
    t = dy * g
    gx = r * (t - xh * (t * xh).mean(-1, keepdim=True))
    if st["dres"] is not None:
        gx = gx + st["dres"].float()
    return dict(gx=gx.to(st["hid"].dtype), gg=(dy * xh).sum(0, dtype=torch.float64).float())


def _balance(st):
    N, E, K, S = st["N"], st["E"], st["K"], st["S"]
    if own:
        from expert_load_balancing_b200 import binding as B
        score = B.KOLIBRI_SCORE_SOFTMAX if st["score"] == "softmax" else B.KOLIBRI_SCORE_SIGMOID
        if st["fused"]:
            loss, counts, prob, gz = B.kolibri_balance_loss(
                st["z"], st["ids"], st["lam"], seq_offsets=st["seq"], score=score, grad_loss=st["up"], gz=st["gz"],
                want_gz=True, loss=st["loss"], counts=st["counts"], prob=st["prob"])
        else:
            loss, counts, prob, _ = B.kolibri_balance_loss(
                st["z"], st["ids"], st["lam"], seq_offsets=st["seq"], score=score, loss=st["loss"], counts=st["counts"],
                prob=st["prob"])
            gz = B.kolibri_balance_loss_grad(st["z"], counts, K, st["lam"], seq_offsets=st["seq"], score=score,
                                             grad_loss=st["up"], gz=st["gz"])
        return dict(loss=loss, counts=counts, prob=prob, gz=gz)
    z, seq = st["z"], st["seq"]
    length = seq[1:] - seq[:-1]
    row = torch.arange(N, device=z.device)
    of = torch.searchsorted(seq, row, right=True) - 1                   # the row's sequence; S behind the last
    inside = (of >= 0) & (of < S)
    of = torch.where(inside, of, S)
    if st["score"] == "softmax":
        s = torch.exp(z - z.amax(-1, keepdim=True))
        slope = None
    else:
        s = 1.0 / (1.0 + torch.exp(-z))
        slope = 1.0 / (1.0 + torch.exp(z))
    p = s / s.sum(-1, keepdim=True)
    hot = (of[None, :] == torch.arange(S, device=z.device)[:, None]).double()
    mean = (hot @ p.double()) / length.clamp_min(1)[:, None]
    slot = of[:, None] * E + st["ids"].long()
    counts = torch.zeros((S + 1) * E, dtype=torch.int64, device=z.device).scatter_add_(0, slot.view(-1), torch.ones_like(slot).view(-1))
    counts = counts.view(S + 1, E)[:S]
    f = counts.double() * E / (K * length.clamp_min(1))[:, None]
    loss = st["lam"] * (f * mean).sum(-1)
    # sum_j p_j = 1, so f may be taken relative to 1, its mean
    rel = torch.cat([f - 1.0, f.new_zeros(1, E)]).float()[of]
    scale = torch.cat([st["up"].double() * st["lam"] / length.clamp_min(1), f.new_zeros(1)]).float()[of]
    gz = scale[:, None] * p * (rel - (rel * p).sum(-1, keepdim=True))
    if slope is not None:
        gz = gz * slope
    gz = torch.where(inside[:, None], gz, torch.zeros_like(gz))
    return dict(loss=loss.float(), counts=counts.to(torch.int32), prob=mean.float(), gz=gz)


def _dequantise(w, s):
    *lead, r, c = w.shape
    return (w.float().view(*lead, r // GROUP, GROUP, c // GROUP, GROUP) * s[..., :, None, :, None]).view(w.shape)


def _swiglu(a, wgu, wd):
    """The two projections of a (batch of) expert(s), h held in 8 bits with a scale per GROUP units."""
    gu = a @ wgu.transpose(-1, -2)
    g, u = gu.chunk(2, dim=-1)
    h = g / (1.0 + torch.exp(-g)) * u
    v = h.view(*h.shape[:-1], -1, GROUP)
    s = v.abs().amax(-1, keepdim=True).clamp_min(AMAX_MIN) / E4M3_MAX
    q = (v / s).clamp(-E4M3_MAX, E4M3_MAX).to(F8).float() * s
    return q.view(h.shape) @ wd.transpose(-1, -2)


def _experts(st):
    if own:
        from expert_load_balancing_b200 import binding as B
        return B.kolibri_expert_ffn_fp8(
            st["x8"], st["xs"], st["perm"], st["offsets"], st["inv"], st["gates"], st["wgu"], st["sgu"], st["wd"], st["sd"],
            st["wgu_s"], st["sgu_s"], st["wd_s"], st["sd_s"], y=st["y"])
    N, d, E, K = st["N"], st["d"], st["E"], st["K"]
    x = (st["x8"].float().view(N, -1, GROUP) * st["xs"][..., None]).view(N, d)
    if N * K < E:       # few slots: the weights of each slot's expert
        e = st["ids"].view(-1)
        a = x.repeat_interleave(K, 0)[:, None, :]
        slots = _swiglu(a, _dequantise(_take(st["wgu"], e), st["sgu"][e]), _dequantise(_take(st["wd"], e), st["sd"][e]))[:, 0]
    else:               # every expert's rows, padded to the longest
        perm = st["perm"].long()
        e = st["ids"].view(-1)[perm]
        at = e * st["most"] + torch.arange(N * K, device=x.device) - st["offsets"][e]
        a = x.new_zeros(E * st["most"], d)
        a[at] = x[perm // K]
        rows = _swiglu(a.view(E, -1, d), _dequantise(st["wgu"], st["sgu"]), _dequantise(st["wd"], st["sd"])).view(-1, d)[at]
        slots = rows[st["inv"].long()]
    y = (slots.view(N, K, d) * st["gates"][..., None]).sum(1)
    if st["wgu_s"] is not None:
        y = y + _swiglu(x, _dequantise(st["wgu_s"], st["sgu_s"]), _dequantise(st["wd_s"], st["sd_s"]))
    return y.to(torch.bfloat16)


def _take(w, e):
    return w.view(torch.uint8)[e].view(F8)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    size = {"none": 0, "bf16": 2, "f32": 4}
    if op == "norm":
        N, d = case["N"], case["d"]
        per = size[case["x"]] + 2 * size[case["res"]] + (2 if case["y"] else 0) + (1 if case["fp8"] else 0)
        return dict(bytes=N * d * per + 2 * d + (4 * N * -(-d // GROUP) if case["fp8"] else 0), flops=6 * N * d)
    if op == "norm_grad":
        N, d = case["N"], case["d"]
        per = size[case["h"]] * (3 if case["gres"] else 2) + size[case["gy"]]
        return dict(bytes=N * d * per + 6 * d, flops=11 * N * d)
    if op == "balance":
        N, E, K, S = case["N"], case["E"], case["K"], case["S"]
        return dict(bytes=8 * N * E + 4 * N * K + S * (8 * E + 16), flops=12 * N * E)
    N, d, F, E, K = (case[k] for k in ("N", "d", "F", "E", "K"))
    active = E * (1.0 - (1.0 - K / E) ** N)          # experts that have rows, expected
    weights = (active + (1 if case["shared"] else 0)) * 3 * d * F * (1 + 4 / GROUP ** 2)
    rows = N * K + (N if case["shared"] else 0)
    return dict(bytes=weights + N * d * (1 + 4 / GROUP + 2) + 12 * N * K + 8 * E, flops=6 * rows * d * F)


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "norm":
        d = case["d"]
        h = st["x"].to(f64)
        res = None
        if st["r"] is not None:
            h = h + st["r"].to(f64)
            res = h.clone()
        y = h / torch.sqrt(torch.sum(h.square(), 1) / d + EPS).unsqueeze(1) * st["g"].to(f64)
        if not case["fp8"]:
            return dict(res=res, y=y, y8=None, scales=None)
        groups = -(-d // GROUP)
        full = y.new_zeros(case["N"], groups * GROUP)
        full[:, :d] = y
        top = full.abs().reshape(-1, GROUP).max(1).values.reshape(-1, groups)
        s = torch.maximum(top, torch.full_like(top, AMAX_MIN)) / E4M3_MAX
        return dict(res=res, y=y if case["y"] else None, y8=y / s.repeat_interleave(GROUP, 1)[:, :d], scales=s)
    if op == "norm_grad":
        d = case["d"]
        h, dy = st["hid"].to(f64), st["dy"].to(f64)
        w = dy * st["g"].to(f64)
        q = torch.sum(h.square(), 1, keepdim=True) / d + EPS
        gx = w / q.sqrt() - h * torch.sum(w * h, 1, keepdim=True) / (d * q * q.sqrt())
        if st["dres"] is not None:
            gx += st["dres"].to(f64)
        return dict(gx=gx, gg=torch.sum(dy * h / q.sqrt(), 0))
    if op == "balance":
        E, K, S = case["E"], case["K"], case["S"]
        cut = st["seq"].tolist()
        loss, prob, gz = [], [], torch.zeros(case["N"], E, dtype=f64, device=st["z"].device)
        for s in range(S):
            a, b = cut[s], cut[s + 1]
            if a == b:
                loss.append(gz.new_zeros(()))
                prob.append(gz.new_zeros(E))
                continue
            z = st["z"][a:b].to(f64)
            load = torch.bincount(st["ids"][a:b].reshape(-1).long(), minlength=E).to(f64) * E / (K * (b - a))
            q = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z) / torch.sigmoid(z).sum(1, keepdim=True)
            prob.append(q.mean(0))
            loss.append(st["lam"] * torch.dot(load, prob[-1]))
            part = q * (load - (q @ load)[:, None]) * (st["lam"] * st["up"][s].to(f64) / (b - a))
            gz[a:b] = part if case["score"] == "softmax" else part * torch.sigmoid(-z)
        return dict(loss=torch.stack(loss), counts=None, prob=torch.stack(prob), gz=gz)
    N, d, F, E, K = (case[k] for k in ("N", "d", "F", "E", "K"))

    def wide(w, s):
        return w.to(f64) * s.to(f64).repeat_interleave(GROUP, -2).repeat_interleave(GROUP, -1)

    def layer(a, gate_up, gate_up_s, down, down_s):
        both = a @ wide(gate_up, gate_up_s).T
        h = both[:, :F] * torch.sigmoid(both[:, :F]) * both[:, F:]
        s = h.abs().reshape(-1, F // GROUP, GROUP).amax(2).clamp(min=AMAX_MIN) / E4M3_MAX
        s = s.repeat_interleave(GROUP, 1)
        held = (h / s).to(torch.float32).clamp(-E4M3_MAX, E4M3_MAX).to(F8).to(f64) * s
        return held @ wide(down, down_s).T

    x = st["x8"].to(f64) * st["xs"].to(f64).repeat_interleave(GROUP, 1)
    y = layer(x, st["wgu_s"], st["sgu_s"], st["wd_s"], st["sd_s"]) if case["shared"] else x.new_zeros(N, d)
    cut, perm = st["offsets"].tolist(), st["perm"].long()
    gates = st["gates"].to(f64).reshape(-1)
    for e in range(E):
        slots = perm[cut[e]:cut[e + 1]]
        if slots.numel():
            part = layer(x[slots // K], st["wgu"][e], st["sgu"][e], st["wd"][e], st["sd"][e])
            y.index_add_(0, slots // K, part * gates[slots][:, None])
    return y
