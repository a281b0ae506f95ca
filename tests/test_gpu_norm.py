"""The norm in front of the router and its gradient against the formulas in
64 bits.

Bars.  Half a rounding step is 2^-8 (bf16), 2^-24 (fp32), 2^-4 (e4m3, and
2^-10 below its smallest normal number 2^-6).
- h = x + res is one fp32 addition (2^-24), the sum of squares of d <= 16384
  terms in fp32 is a chain of at most 16 + 5 + 32 additions, each 2^-24, all
  terms positive; the square root halves it; r, the two products and the
  reciprocal add under ten more roundings.  So y before its last rounding is
  within 64 * 2^-24 = 2^-18 of the formula, relative.
- gx = r t - h r^3 mean(t h): both parts carry that error relative to the sum
  of their terms' magnitudes: 2^-17 (|r t| + |h| r^3 mean|t h|).
- gweight sums N terms in fp32: (N + 64) 2^-24 + 2^-17 of the sum of magnitudes."""
import math
import threading

import pytest
import torch

from expert_load_balancing_b200 import binding as B

from gpu_helpers import check_status

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, FP = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib(kolibri_lib):
    return kolibri_lib


def _randn(g, *shape, dtype=FP, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _inputs(N, d, xt, rt, wt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = torch.exp(torch.randn(d, generator=g, device="cuda"))
    x = _randn(g, N, d, dtype=xt)
    res = None if rt is None else (_randn(g, N, d) * wide).to(rt)
    w = (1.0 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(wt)
    return x, res, w


def _within(got, want, bound, what):
    err = (got.double() - want).abs()
    assert torch.isfinite(got.float()).all(), what
    worst = float((err / bound.clamp_min(1e-300)).max())
    assert worst <= 1.0, (what, worst)


def _check_forward(x, res, w, eps, out, y8=True):
    res_out, y, q, s = out
    N, d = x.shape
    h = x.double() + (0 if res is None else res.double())
    want = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.double()
    if res is not None:
        _within(res_out, h, (HALF[res.dtype] + 2.0 ** -24) * h.abs() + 1e-38, "res_out")
    if y is not None:
        _within(y, want, (HALF[BF] + 2.0 ** -18) * want.abs() + 1e-38, "y")
    if q is not None:
        G = -(-d // 128)
        pad = want.new_zeros(N, G * 128)
        pad[:, :d] = want
        amax = pad.abs().view(N, G, 128).amax(2).clamp_min(1e-30)
        _within(s, amax / 448, 2.0 ** -17 * amax / 448, "scales")
        sc = s.double().repeat_interleave(128, 1)[:, :d]
        v = (want / sc).abs()
        half = torch.maximum(2.0 ** -4 * v, torch.full_like(v, 2.0 ** -10)) * (1 + 2.0 ** -10) + 2.0 ** -16 * v
        _within(q.double() * sc, want, half * sc, "y8")


@pytest.mark.parametrize("N,d,xt,rt,wt", [
    (1, 2560, BF, BF, BF), (1, 8, BF, None, BF), (3, 16, FP, BF, FP), (7, 128, BF, FP, BF),
    (5, 136, BF, BF, FP), (33, 1000, FP, FP, BF), (257, 2048, BF, BF, BF), (1500, 2560, BF, BF, BF),
    (2049, 2560, FP, BF, BF), (1200, 640, BF, None, BF), (64, 4104, BF, BF, BF), (9, 8200, FP, FP, FP),
    (5, 16384, BF, BF, BF), (1100, 16384, BF, FP, FP), (20000, 512, BF, FP, BF), (40000, 64, FP, None, FP)])
def test_forward(N, d, xt, rt, wt):
    x, res, w = _inputs(N, d, xt, rt, wt, 11 + N + d)
    keep = x.clone(), None if res is None else res.clone()
    out = B.kolibri_rms_norm(x, w, EPS, res=res, want_fp8=True)
    torch.cuda.synchronize()
    assert torch.equal(x, keep[0]) and (res is None or torch.equal(res, keep[1]))
    _check_forward(x, res, w, EPS, out)
    # each output alone gives the same bits
    a = B.kolibri_rms_norm(x, w, EPS, res=res, want_fp8=False)
    assert torch.equal(a[1], out[1]) and a[2] is None and a[3] is None
    b = B.kolibri_rms_norm(x, w, EPS, res=res, want_y=False, want_fp8=True)
    assert b[1] is None and torch.equal(b[2].view(torch.uint8), out[2].view(torch.uint8)) and torch.equal(b[3], out[3])


@pytest.mark.parametrize("scale", [1e-18, 1e-3, 1e3, 1e15])
def test_forward_of_small_and_large_values(scale):
    x, res, w = _inputs(37, 2560, FP, FP, BF, 5)
    x, res = x * scale, res * scale
    out = B.kolibri_rms_norm(x, w, 0.0, res=res, want_fp8=True)
    _check_forward(x, res, w, 0.0, out)


def test_zero_rows_and_zero_groups():
    x = torch.zeros(5, 512, device="cuda")
    x[1] = torch.randn(512, device="cuda")
    x[1, 128:256] = 0.0
    w = torch.ones(512, device="cuda", dtype=BF)
    _, y, q, s = B.kolibri_rms_norm(x, w, EPS, want_fp8=True)
    assert not y[0].any() and not y[2:].any() and not q.float()[0].any()
    assert torch.isfinite(s).all() and (s > 0).all()
    assert not (q.float() * s.repeat_interleave(128, 1))[1, 128:256].any()
    _check_forward(x, None, w, EPS, (None, y, q, s))


def test_residual_that_cancels():
    x, _, w = _inputs(9, 2048, BF, None, BF, 3)
    res = -x
    res[:, ::7] += 1.0
    out = B.kolibri_rms_norm(x, w, EPS, res=res.contiguous(), want_fp8=True)
    _check_forward(x, res, w, EPS, out)


@pytest.mark.parametrize("wt", [FP, BF])
def test_eight_bit_values_are_those_of_the_quotient(wt):
    """h = 1 and eps = 0, so y is the weight itself: y8 has to be e4m3(y / scale), scale = amax / 448, each one rounding.

    The weights stand at the midpoints between e4m3 values times the group's scale and just beside them, where any other
    order of the roundings is off by a whole step."""
    d = 16384
    g = torch.Generator().manual_seed(17)
    top = torch.exp(3.0 * torch.randn(d // 128, 1, generator=g)).to(wt).float()
    s = top / 448.0
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()       # the values 0 .. 448
    mid = (grid[:-1] + grid[1:]) / 2
    v = s * mid[torch.randint(0, 126, (d // 128, 128), generator=g)] * torch.where(torch.rand(d // 128, 128, generator=g) < 0.5, -1.0, 1.0)
    v = torch.where(torch.rand(v.shape, generator=g) < 0.3, torch.nextafter(v, 2 * v), v)
    v[:, :1] = top
    v[:, 1], v[:, 2] = 0.0, -0.0
    w = v.reshape(d).to(wt)
    v = w.float().view(-1, 128)
    assert torch.equal(v.abs().amax(1, keepdim=True), top)
    want = (v / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(d)
    x = torch.ones(3, d, device="cuda")
    _, y, y8, scales = B.kolibri_rms_norm(x, w.cuda(), 0.0, want_fp8=True)
    for row in range(3):
        assert torch.equal(y[row].cpu(), w.to(BF))                    # so y is the weight
        assert torch.equal(scales[row].cpu(), s.view(-1))
        assert torch.equal(y8[row].cpu().view(torch.uint8), want.view(torch.uint8))
    # an infinite value: its group's scale is infinite, the others' quotients are 0; the groups beside it are as before
    w[130] = torch.inf
    _, _, y8, scales = B.kolibri_rms_norm(x, w.cuda(), 0.0, want_fp8=True)
    q = y8[0].float().cpu()
    assert scales[0, 1].isinf() and q[130].isnan() and not q[128:130].any() and not q[131:256].any()
    q = y8[0].cpu().view(torch.uint8)
    assert torch.equal(q[:128], want.view(torch.uint8)[:128]) and torch.equal(q[256:], want.view(torch.uint8)[256:])


@pytest.mark.parametrize("N", [1, 3000])
def test_in_place(N):
    x, res, w = _inputs(N, 2560, BF, BF, BF, 8)
    want = B.kolibri_rms_norm(x, w, EPS, res=res, want_fp8=True)
    r1 = res.clone()
    got = B.kolibri_rms_norm(x, w, EPS, res=r1, res_out=r1, want_fp8=True)
    assert got[0].data_ptr() == r1.data_ptr() and torch.equal(r1, want[0]) and torch.equal(got[1], want[1])
    x1, x2 = x.clone(), x.clone()
    B.kolibri_rms_norm(x1, w, EPS, res=res, res_out=x1)
    assert torch.equal(x1, want[0])
    B.kolibri_rms_norm(x2, w, EPS, res=res, y=x2)
    assert torch.equal(x2, want[1])


def test_rows_behind_the_outputs_stay():
    x, res, w = _inputs(100, 640, BF, BF, BF, 4)
    y = torch.full((103, 640), 7.0, device="cuda", dtype=BF)
    s = torch.full((103, 5), 7.0, device="cuda")
    B.kolibri_rms_norm(x, w, EPS, res=res, y=y[:100], y8=torch.empty(100, 640, device="cuda", dtype=torch.float8_e4m3fn),
                       scales=s[:100])
    assert (y[100:] == 7.0).all() and (s[100:] == 7.0).all()


def test_refusals():
    x, res, w = _inputs(8, 64, BF, BF, BF, 1)
    bad = [dict(x=x.half()), dict(x=x[:, ::2]), dict(w=w[:32]), dict(w=w.double()), dict(res=res[:4]), dict(res=res.half()),
           dict(res=None, res_out=res), dict(res_out=res.float()), dict(y=x.float()), dict(y8=torch.empty(8, 64, device="cuda")),
           dict(scales=torch.empty(8, 2, device="cuda"), want_fp8=True), dict(w=w.cpu())]
    for kw in bad:
        a = dict(x=x, w=w, res=res) | kw
        xx, ww = a.pop("x"), a.pop("w")
        with pytest.raises(ValueError):
            B.kolibri_rms_norm(xx, ww, EPS, **a)
    for kw in (dict(d=12), dict(eps=-1.0), dict(none=True)):
        d = kw.get("d", 64)
        xx = torch.zeros(4, d, device="cuda", dtype=BF)
        with pytest.raises(B.KolibriError):
            B.kolibri_rms_norm(xx, torch.ones(d, device="cuda", dtype=BF), kw.get("eps", EPS), want_y="none" not in kw)
    with pytest.raises(B.KolibriError):
        B.kolibri_rms_norm(x[:0], w, EPS)


# ---------------------------------------------------------------- gradient

def _grad64(gy, h, w, eps, gres):
    h, gy, w = h.double(), gy.double(), w.double()
    d = h.shape[1]
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    t = gy * w
    gx = r * t - h * r ** 3 * (t * h).mean(1, keepdim=True)
    mag = (r * t).abs() + h.abs() * r ** 3 * (t * h).abs().mean(1, keepdim=True)
    if gres is not None:
        gx = gx + gres.double()
    return gx, mag, (gy * h * r).sum(0), (gy * h * r).abs().sum(0)


def _check_grad(gy, h, w, eps, gres, gx, gg):
    want, mag, wg, wmag = _grad64(gy, h, w, eps, gres)
    _within(gx, want, HALF[h.dtype] * want.abs() + 2.0 ** -17 * mag + 2.0 ** -22 * want.abs() + 1e-38, "gx")
    if gg is not None:
        _within(gg, wg, ((h.shape[0] + 64) * 2.0 ** -24 + 2.0 ** -17) * wmag + 1e-38, "gweight")


@pytest.mark.parametrize("N,d,ht,gt,wt,gres", [
    (1, 2560, BF, BF, BF, True), (1, 8, FP, FP, FP, False), (3, 24, BF, FP, BF, True), (333, 2048, FP, FP, BF, False),
    (1500, 2560, BF, BF, BF, True), (2049, 640, BF, FP, FP, False), (64, 4104, FP, BF, BF, True),
    (7, 8200, BF, BF, BF, False), (1030, 16384, FP, FP, FP, True), (5, 16384, BF, FP, BF, True), (30000, 128, BF, BF, BF, False)])
def test_gradient(N, d, ht, gt, wt, gres):
    h, _, w = _inputs(N, d, ht, None, wt, 21 + N)
    g = torch.Generator(device="cuda").manual_seed(N + d)
    gy = _randn(g, N, d, dtype=gt, scale=0.01)
    gr = _randn(g, N, d, dtype=ht, scale=0.02) if gres else None
    gx, gg = B.kolibri_rms_norm_grad(gy, h, w, EPS, gres=gr)
    _check_grad(gy, h, w, EPS, gr, gx, gg)
    # the same bits again, without the weight's gradient, and in place over gres and h
    gx2, gg2 = B.kolibri_rms_norm_grad(gy, h, w, EPS, gres=gr)
    assert torch.equal(gx, gx2) and torch.equal(gg, gg2)
    gx3, none = B.kolibri_rms_norm_grad(gy, h, w, EPS, gres=gr, want_gweight=False)
    assert none is None and torch.equal(gx, gx3)
    if gr is not None:
        B.kolibri_rms_norm_grad(gy, h, w, EPS, gres=gr, gx=gr)
        assert torch.equal(gr, gx)
    if gt == ht:
        y1 = gy.clone()
        B.kolibri_rms_norm_grad(y1, h, w, EPS, gres=None, gx=y1)
        assert torch.equal(y1, B.kolibri_rms_norm_grad(gy, h, w, EPS)[0])
    h1 = h.clone()
    B.kolibri_rms_norm_grad(gy, h1, w, EPS, gres=None, gx=h1)
    assert torch.equal(h1, B.kolibri_rms_norm_grad(gy, h, w, EPS)[0])


@pytest.mark.parametrize("scale", [1e-18, 1e-3, 1e3, 1e15])
@pytest.mark.parametrize("N,d,ht,gt,gres", [(37, 2560, FP, FP, False), (37, 2560, BF, BF, True), (1500, 2560, FP, BF, True), (9, 16384, FP, FP, False)])
def test_gradient_of_small_and_large_values(N, d, ht, gt, gres, scale):
    """The scales of the forward's test: gx is about gy / |h|, and both of its terms are of that size."""
    h, _, w = _inputs(N, d, FP, None, BF, 31 + N)
    h = (h * scale).to(ht)
    g = torch.Generator(device="cuda").manual_seed(N)
    gy = _randn(g, N, d, dtype=gt)
    gr = _randn(g, N, d, dtype=ht, scale=1 / scale) if gres else None
    gx, gg = B.kolibri_rms_norm_grad(gy, h, w, 0.0, gres=gr)
    _check_grad(gy, h, w, 0.0, gr, gx, gg)


@pytest.mark.parametrize("N", [5, 1500])
def test_gradient_of_zero_rows_with_a_tiny_eps(N):
    """h = 0: gx = gy weight / sqrt(eps), and nothing for the weight's gradient."""
    h, _, w = _inputs(N, 512, FP, None, BF, 41)
    h[3] = 0.0
    gy = _randn(torch.Generator(device="cuda").manual_seed(2), N, 512)
    gx, gg = B.kolibri_rms_norm_grad(gy, h, w, 1e-30)
    _check_grad(gy, h, w, 1e-30, None, gx, gg)


def test_gradient_against_differences():
    """L = sum y c: <gx, v> and <gweight, u> against central differences of the formula in 64 bits."""
    h, _, w = _inputs(6, 264, FP, None, FP, 2)
    g = torch.Generator(device="cuda").manual_seed(9)
    c, v, u = _randn(g, 6, 264), _randn(g, 6, 264), _randn(g, 264)
    gx, gg = B.kolibri_rms_norm_grad(c, h, w, EPS)

    def loss(hh, ww):
        return (hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + EPS) * ww * c.double()).sum()

    e = 1e-6
    for got, a, b in ((gx, (e * v.double(), 0), v), (gg, (0, e * u.double()), u)):
        plus = loss(h.double() + a[0], w.double() + a[1])
        minus = loss(h.double() - a[0], w.double() - a[1])
        diff = float((plus - minus) / (2 * e))
        terms = (got.double() * b.double())
        # differences: e^2 times a third derivative of order one, and 2^-52 |L| / e
        assert abs(float(terms.sum()) - diff) <= 2.0 ** -16 * float(terms.abs().sum()) + 1e-5


def test_gradient_refusals():
    h, _, w = _inputs(8, 64, BF, None, BF, 1)
    for kw in (dict(gy=h[:4]), dict(gres=h.float()), dict(gx=h.float()), dict(gweight=w), dict(w=w[:8]), dict(gy=h.half()),
               dict(ws=torch.empty(1 << 20, device="cuda"))):
        a = dict(gy=h, w=w) | kw
        gy, ww = a.pop("gy"), a.pop("w")
        with pytest.raises(ValueError):
            B.kolibri_rms_norm_grad(gy, h, ww, EPS, **a)
    with pytest.raises(B.KolibriError):
        B.kolibri_rms_norm_grad(h, h, w, EPS, ws=torch.empty(16, device="cuda", dtype=torch.uint8))


def test_other_stream_and_graph():
    x, res, w = _inputs(700, 2560, BF, BF, BF, 6)
    want = B.kolibri_rms_norm(x, w, EPS, res=res, want_fp8=True)
    gwant = B.kolibri_rms_norm_grad(want[1], want[0], w, EPS)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = [torch.empty_like(t) for t in want]
    gx, gg = torch.empty_like(want[0]), torch.empty(2560, device="cuda")
    ws = torch.empty(B.load().kolibri_rms_norm_grad_workspace_size(700, 2560), device="cuda", dtype=torch.uint8)

    def run(stream=None):
        B.kolibri_rms_norm(x, w, EPS, res=res, res_out=out[0], y=out[1], y8=out[2], scales=out[3], stream=stream)
        B.kolibri_rms_norm_grad(out[1], out[0], w, EPS, gx=gx, gweight=gg, ws=ws, stream=stream)

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, want))
        assert torch.equal(gx, gwant[0]) and torch.equal(gg, gwant[1])

    run(stream=st)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for t in out + [gx, gg]:
        t.view(torch.uint8).fill_(0)
    for _ in range(2):
        graph.replay()
    same()
    check_status()


def test_gradient_from_several_host_threads():
    """Four threads, a stream and buffers each, on sizes that no test before has launched: the bits of calls one by one."""
    shapes = [(1200, 328), (1200, 2456), (1200, 3352), (700, 4632), (1100, 6536), (1100, 12296)]
    cases = []
    for i, (N, d) in enumerate(shapes):
        h, _, w = _inputs(N, d, FP, None, BF, 60 + i)
        cases.append((_randn(torch.Generator(device="cuda").manual_seed(i), N, d), h, w))
    torch.cuda.synchronize()
    got, wrong = {}, []
    start = threading.Barrier(4)

    def work(t):
        try:
            st = torch.cuda.Stream()
            start.wait()
            for i, (gy, h, w) in enumerate(cases):
                got[t, i] = B.kolibri_rms_norm_grad(gy, h, w, EPS, stream=st)
            st.synchronize()
        except Exception as e:                      # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    torch.cuda.synchronize()
    for i, (gy, h, w) in enumerate(cases):
        gx, gg = B.kolibri_rms_norm_grad(gy, h, w, EPS)
        _check_grad(gy, h, w, EPS, None, gx, gg)
        for t in range(4):
            assert torch.equal(got[t, i][0], gx) and torch.equal(got[t, i][1], gg), (t, i)
    check_status()


def test_rows_behind_32_bit_offsets():
    """2.2e9 elements: the last rows come out as in a call of their own."""
    N, d = 860_000, 2560
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty(N, d, device="cuda", dtype=BF).normal_(generator=g)
    w = torch.ones(d, device="cuda", dtype=BF)
    out = B.kolibri_rms_norm(x, w, EPS, res=x, want_fp8=True)
    t = x[-5:].contiguous()
    for a, b in zip(out, B.kolibri_rms_norm(t, w, EPS, res=t, want_fp8=True)):
        assert torch.equal(a[-5:].view(torch.uint8), b.view(torch.uint8))
    gx, _ = B.kolibri_rms_norm_grad(out[1], out[0], w, EPS, gres=x)
    small, _ = B.kolibri_rms_norm_grad(out[1][-5:].contiguous(), out[0][-5:].contiguous(), w, EPS, gres=t)
    # another block size sums a row in another order: fp32 sums of 2560 terms, then one bf16 rounding
    assert ((gx[-5:].float() - small.float()).abs() <= 2.0 ** -7 * small.float().abs() + 1e-6).all()
    check_status()
