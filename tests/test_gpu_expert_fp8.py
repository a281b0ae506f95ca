"""The expert layer on 8-bit operands against the formulas in 64 bits, in two
steps: the hidden units that the call leaves at the front of its workspace
(h8 [rows, F] e4m3, then from the next multiple of 256 bytes hs [F/128, ld]
fp32, ld = rows rounded up to 4 and at least 132) against SiLU(g) u, and y against the down projection of those very h.

Bars.  Half a rounding step is 2^-4 (e4m3; 2^-10 absolute below 2^-6) and 2^-8
(bf16).  A sum of n fp32 products is within n 2^-24 of the sum of their
magnitudes A, so g and u carry d 2^-24 (Ag, Au), and with |SiLU'| < 1.1
  |dh| <= d 2^-24 (1.1 |u| Ag + |SiLU(g)| Au) + 2^-19 |h|
(the fast exponential and division: under 32 units of 2^-24).  The scale of a
group moves with its largest |h|: by max |dh| / 448 and two roundings.  Then y:
an expert's o carries F 2^-24 of the magnitudes and, kept in fp16 with its
group's largest in [2^14, 2^15), 2^-11 |o| or, where that is below the normal
numbers, 2^-25 of 2^-14 of the group's largest; the sum over K + 1 of them (K + 1)
2^-24 and y itself 2^-8 |y|."""
import math

import pytest
import torch

from expert_load_balancing_b200 import binding as B

from gpu_helpers import check_status

pytestmark = pytest.mark.gpu
F8, BF = torch.float8_e4m3fn, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(kolibri_lib):
    return kolibri_lib


def _f8(g, *shape):
    return (torch.randn(*shape, generator=g, device="cuda") * 60).clamp(-448, 448).to(F8)


def _scale(g, *shape, mean):
    return torch.exp(0.5 * torch.randn(*shape, generator=g, device="cuda")) * mean


def _group(ids, E):
    flat = ids.reshape(-1).long()
    perm = torch.argsort(flat, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(flat.numel(), device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    off[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    return perm.to(torch.int32), off, inv.to(torch.int32)


def _case(N, d, F, E, K, shared, seed, skew=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    like = torch.randn(N, E, generator=g, device="cuda")
    if skew:                       # expert 1 in every token, the upper half of the experts in none
        like[:, 1] += 100.0
        like[:, E // 2:] -= 100.0
    ids = torch.topk(like, K, dim=1).indices.to(torch.int32)
    c = dict(x8=_f8(g, N, d), xs=_scale(g, N, d // 128, mean=1 / 60), gates=torch.rand(N, K, generator=g, device="cuda"),
             wgu=_f8(g, E, 2 * F, d), sgu=_scale(g, E, 2 * F // 128, d // 128, mean=d ** -0.5 / 60),
             wd=_f8(g, E, d, F), sd=_scale(g, E, d // 128, F // 128, mean=F ** -0.5 / 60), ids=ids)
    c["perm"], c["off"], c["inv"] = _group(ids, E)
    if shared:
        c |= dict(wgu_s=_f8(g, 2 * F, d), sgu_s=_scale(g, 2 * F // 128, d // 128, mean=d ** -0.5 / 60),
                  wd_s=_f8(g, d, F), sd_s=_scale(g, d // 128, F // 128, mean=F ** -0.5 / 60))
    else:
        c |= dict(wgu_s=None, sgu_s=None, wd_s=None, sd_s=None)
    return c


def _call(c, **kw):
    return B.kolibri_expert_ffn_fp8(c["x8"], c["xs"], c["perm"], c["off"], c["inv"], c["gates"], c["wgu"], c["sgu"],
                                    c["wd"], c["sd"], c["wgu_s"], c["sgu_s"], c["wd_s"], c["sd_s"], **kw)


def _wide(w, s):
    return w.double() * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)


DECODE_ROWS = 64      # up to this many rows h stays in fp32 and is put into e4m3 where it is read


def _hidden(ws, rows, F):
    if rows <= DECODE_ROWS:
        h = ws[:rows * F * 4].view(torch.float32).view(rows, F // 128, 128)
        amax = h.abs().amax(2).clamp_min(1e-30)
        q = (h * (448.0 / amax)[..., None]).clamp(-448, 448).to(F8)          # the same fp32 operations, the same bits
        return q.view(rows, F), amax / 448.0
    h8 = ws[:rows * F].view(F8).view(rows, F)
    at = (rows * F + 255) // 256 * 256
    ld = max((rows + 3) // 4 * 4, 132)
    return h8, ws[at:at + ld * (F // 128) * 4].view(torch.float32).view(F // 128, ld)[:, :rows].t()


def _check(c, y, ws):
    N, d = c["x8"].shape
    K = c["gates"].shape[1]
    E, F2, _ = c["wgu"].shape
    F = F2 // 2
    shared = c["wgu_s"] is not None
    NK = N * K
    rows = NK + (N if shared else 0)
    h8, hs = _hidden(ws, rows, F)
    x = c["x8"].double() * c["xs"].double().repeat_interleave(128, 1)
    off = c["off"].tolist() + ([rows] if shared else [])
    perm = torch.cat([c["perm"].long() // K, torch.arange(N, device="cuda")])
    o = torch.zeros(rows, d, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(o)
    for e in range(E + shared):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        wgu = _wide(c["wgu"][e], c["sgu"][e]) if e < E else _wide(c["wgu_s"], c["sgu_s"])
        wd = _wide(c["wd"][e], c["sd"][e]) if e < E else _wide(c["wd_s"], c["sd_s"])
        xe = x[perm[a:b]]
        gu, agu = xe @ wgu.T, xe.abs() @ wgu.abs().T
        g, u, ag, au = gu[:, :F], gu[:, F:], agu[:, :F], agu[:, F:]
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = d * 2.0 ** -24 * (1.1 * u.abs() * ag + silu.abs() * au) + 2.0 ** -19 * h.abs()
        s = hs[a:b].double()
        group = lambda t: t.view(b - a, F // 128, 128).amax(2)  # noqa: E731
        want_s = group(h.abs()).clamp_min(1e-30) / 448
        assert ((s - want_s).abs() <= group(dh) / 448 + 2.0 ** -22 * want_s).all(), "scales"
        sw = s.repeat_interleave(128, 1)
        hq = h8[a:b].double() * sw
        v = h.abs() / sw
        step = torch.maximum(2.0 ** -4 * v, torch.full_like(v, 2.0 ** -10)) * (1 + 2.0 ** -10) * sw
        err = ((hq - h).abs() / (step + dh * (1 + 2.0 ** -3) + 1e-300)).max()
        assert float(err) <= 1.0, ("h", e, float(err))
        o[a:b] = hq @ wd.T
        mag[a:b] = hq.abs() @ wd.abs().T
    top = o.abs().view(rows, d // 128, 128).amax(2).repeat_interleave(128, 1)
    do = F * 2.0 ** -24 * mag
    do = do + 2.0 ** -11 * (o.abs() + do) + 2.0 ** -39 * (top + do)
    gates = c["gates"].double()
    at = c["inv"].long().view(N, K)
    want = (o[at] * gates[..., None]).sum(1)
    bound = (do[at] * gates[..., None]).sum(1)
    size = (o[at].abs() * gates[..., None]).sum(1)
    if shared:
        want, bound, size = want + o[NK:], bound + do[NK:], size + o[NK:].abs()
    bound = bound + (K + 1) * 2.0 ** -24 * size
    bound = bound + 2.0 ** -8 * (want.abs() + bound)
    worst = float(((y.double() - want).abs() / bound.clamp_min(1e-300)).max())
    assert torch.isfinite(y.float()).all() and worst <= 1.0, ("y", worst)


CASES = [
    # N, d, F, E, K, shared, skew
    (1, 256, 128, 4, 1, False, False), (1, 2560, 512, 16, 6, True, False), (2, 512, 256, 8, 3, True, False),
    (5, 768, 384, 12, 8, False, False), (17, 1024, 128, 3, 1, True, False), (64, 2560, 512, 96, 6, True, False),
    (130, 512, 256, 2, 1, False, False), (129, 256, 128, 4, 3, True, True), (700, 1280, 256, 8, 2, True, True),
    (1500, 256, 512, 32, 16, False, False), (333, 2048, 512, 128, 8, False, False), (2000, 512, 128, 512, 6, True, False),
    (3001, 768, 256, 5, 2, True, False),
    (1, 8192, 128, 4, 2, True, False), (1, 256, 8192, 4, 1, True, False), (260, 4352, 128, 4, 1, False, False), (150, 256, 4224, 4, 1, True, False),
    # a few rows per expert, some of them with many
    (64, 2560, 512, 384, 6, True, False), (100, 512, 256, 128, 4, True, True), (65, 256, 128, 512, 1, True, False),
    (500, 768, 384, 64, 1, True, False), (12, 8192, 128, 64, 8, False, False), (12, 256, 8192, 64, 8, True, False),
    (33, 256, 128, 1, 1, True, False), (300, 256, 128, 1, 1, False, False),
    # several tiles per block: every barrier goes round many times
    (20000, 256, 512, 6, 2, True, False), (4000, 2048, 256, 4, 2, False, False), (9000, 1024, 384, 3, 1, True, True),
]


@pytest.mark.parametrize("N,d,F,E,K,shared,skew", CASES)
def test_layer(N, d, F, E, K, shared, skew):
    c = _case(N, d, F, E, K, shared, N + d + E, skew)
    ws = B.expert_ffn_fp8_workspace(N, d, F, K, shared)
    ws.fill_(255)                                  # NaN bytes: nothing may be read before it is written
    y = torch.full((N + 2, d), 7.0, device="cuda", dtype=BF)
    _call(c, y=y[:N], ws=ws)
    check_status()
    assert (y[N:] == 7.0).all()
    _check(c, y[:N], ws)
    again = _call(c)                               # the same bits, from a workspace of its own
    assert torch.equal(again, y[:N])


def test_exact_values():
    """Powers of two throughout: every product, sum and rounding is exact, and so is y.

    x = 1, gate rows sum to 64 (SiLU(64) = 64 to fp32), up rows to 2 u: h = 128 u, and the down rows pick units."""
    N, d, F, E, K = 40, 256, 128, 4, 2
    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    x8 = one(N, d).to(F8)
    u = 2.0 ** torch.arange(-3, 1, device="cuda").float().repeat(F // 4)
    wgu = torch.zeros(E, 2 * F, d, device="cuda")
    wgu[:, :F] = 0.25
    wgu[:, F:, :2] = u[None, :, None]
    wd = torch.zeros(E, d, F, device="cuda")
    for col in range(d):
        wd[:, col, col % F] = 1.0
    ids = torch.stack([torch.arange(N, device="cuda") % E, (torch.arange(N, device="cuda") + 1) % E], 1).to(torch.int32)
    perm, off, inv = _group(ids, E)
    sgu, sd = one(E, 2, 2), one(E, 2, 1) * 3.5
    gates = one(N, K)
    gates[:, 1] = 0.5
    y = B.kolibri_expert_ffn_fp8(x8, one(N, 2), perm, off, inv, gates, wgu.to(F8), sgu, wd.to(F8), sd)
    check_status()
    # amax = 128: hs = 128 / 448 = 2^-1.807..., h8 = 448 u exactly; o = fp32(448 u hs 3.5) = 448 u within one rounding
    want = (1.5 * 448.0 * u).repeat(d // F).expand(N, d)
    assert ((y.float() - want).abs() <= 2.0 ** -8 * want).all()
    assert torch.equal(y.float(), want.to(BF).float())


def test_zero_rows_and_empty_experts():
    c = _case(50, 512, 128, 16, 2, True, 3, skew=True)
    c["x8"][7] = torch.zeros(512, device="cuda").to(F8)
    ws = B.expert_ffn_fp8_workspace(50, 512, 128, 2, True)
    y = _call(c, ws=ws)
    check_status()
    assert not y[7].any()
    _check(c, y, ws)


def test_gates_of_zero_and_a_shared_expert_alone():
    c = _case(33, 512, 256, 8, 2, True, 4)
    c["gates"].zero_()
    ws = B.expert_ffn_fp8_workspace(33, 512, 256, 2, True)
    y = _call(c, ws=ws)
    _check(c, y, ws)
    check_status()


def test_bad_entries_are_reported():
    """Out-of-range perm and inv entries and broken offsets set the status word; every access stays in the arrays."""
    for E in (8, 128):
        for key, bad in (("perm", -1), ("perm", 1 << 30), ("inv", -7), ("inv", 300 * 2)):
            c = _case(300, 256, 128, E, 2, True, 5)
            c[key][13] = bad
            _call(c)
            assert B.kolibri_device_status() == B.KOLIBRI_ERR_DEVICE, (E, key, bad)
        for i, v in ((0, 1), (E, 599), (E, 1 << 40), (4, -1), (4, 1 << 35)):
            c = _case(300, 256, 128, E, 2, False, 5)
            c["off"][i] = v
            _call(c)
            assert B.kolibri_device_status() == B.KOLIBRI_ERR_DEVICE, (E, i, v)
    check_status()


def test_bad_entries_are_reported_for_a_few_tokens():
    for bad in (-7, 8 * 2):
        c = _case(8, 256, 128, 8, 2, True, 5)
        c["inv"][13] = bad
        _call(c)
        assert B.kolibri_device_status() == B.KOLIBRI_ERR_DEVICE, bad
    for i, v in ((0, 1), (8, 15), (8, 1 << 40), (4, -1), (4, 1 << 35)):
        c = _case(8, 256, 128, 8, 2, False, 5)
        c["off"][i] = v
        _call(c)
        assert B.kolibri_device_status() == B.KOLIBRI_ERR_DEVICE, (i, v)
    check_status()


@pytest.mark.parametrize("N,K,shared", [(9, 6, True), (10, 6, True), (64, 1, False), (65, 1, False), (4, 16, False), (3, 16, True)])
def test_both_sides_of_the_choice_of_kernels(N, K, shared):
    """Up to 64 rows the layer streams each row's weights, above it runs in tiles."""
    c = _case(N, 512, 384, 20, K, shared, 40 + N)
    ws = B.expert_ffn_fp8_workspace(N, 512, 384, K, shared)
    ws.fill_(255)
    _check(c, _call(c, ws=ws), ws)
    check_status()


def test_refusals():
    c = _case(8, 256, 128, 4, 2, True, 6)
    for kw in (dict(x8=c["x8"].view(torch.uint8)), dict(xs=c["xs"][:, :1]), dict(gates=c["gates"].double()),
               dict(perm=c["perm"].long()), dict(off=c["off"][:-1]), dict(inv=c["inv"][:3]), dict(sgu=c["sgu"][:, :1]),
               dict(wd=c["wd"][:, :128]), dict(sd=c["sd"].to(BF)), dict(wgu_s=None), dict(sd_s=None),
               dict(wd_s=c["wd_s"].t()), dict(xs=c["xs"].cpu())):
        with pytest.raises(ValueError):
            _call(c | kw)
    with pytest.raises(ValueError):
        _call(c, y=torch.empty(8, 256, device="cuda"))
    with pytest.raises(B.KolibriError):
        _call(c, ws=torch.empty(256, device="cuda", dtype=torch.uint8))
    odd = _case(4, 384, 128, 4, 2, False, 6)       # d % 256
    with pytest.raises(B.KolibriError):
        _call(odd, ws=torch.empty(1 << 20, device="cuda", dtype=torch.uint8))


def test_other_stream_and_graph():
    for N in (1, 30, 400):
        c = _case(N, 1280, 256, 16, 4, True, 7)
        want = _call(c)
        torch.cuda.synchronize()
        ws = B.expert_ffn_fp8_workspace(N, 1280, 256, 4, True)
        y = torch.zeros_like(want)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        _call(c, y=y, ws=ws, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _call(c, y=y, ws=ws)
        y.zero_()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    check_status()


def test_rows_behind_32_bit_offsets():
    """2.4e9 bytes of gathered rows, 4.8e9 of expert outputs: the last tokens come out as in a call of their own."""
    N, d, F, E, K, tail = 155_000, 2560, 128, 16, 6, 40
    c = _case(N, d, F, E, K, True, 9)
    y = _call(c)
    check_status()
    t = dict(c)
    for k in ("x8", "xs", "gates", "ids"):
        t[k] = c[k].view(torch.uint8)[-tail:].view(F8).contiguous() if k == "x8" else c[k][-tail:].contiguous()
    t["perm"], t["off"], t["inv"] = _group(t["ids"], E)
    small = _call(t)
    assert torch.equal(y[-tail:], small)
    check_status()
