"""The norm, the router, the grouping, the 8-bit experts and the balance loss as
a layer runs them one after the other, forward and backward.

Bars.  Serving: the experts get the very y8, scales and routing that the calls
before them wrote, so y is off by what the layer's own test allows; here an h
may also fall on the other side of a rounding border (one step, 2^-3 of itself),
which is held against the products' magnitudes.  Training: the gradients go
through four calls, each within 2^-13 of its terms' magnitudes (the balance
loss's 2^-15, the fp32 products' E 2^-24 and d 2^-24, the norm's 2^-17), and gx
is rounded to bf16 once, within 2^-8 of each value: 2^-8 + 2^-10 in the 2-norm."""
import pytest
import torch

from expert_load_balancing_b200 import binding as B

from gpu_helpers import check_status

pytestmark = pytest.mark.gpu
F8, BF = torch.float8_e4m3fn, torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib(kolibri_lib):
    return kolibri_lib


def _blocks(w):
    """w [..., r, c] in e4m3 with one scale per 128 x 128 block."""
    *lead, r, c = w.shape
    v = w.view(*lead, r // 128, 128, c // 128, 128)
    s = v.abs().amax(dim=(-3, -1)) / 448
    return (v / s[..., :, None, :, None]).clamp(-448, 448).to(F8).view(w.shape), s.contiguous()


def _wide(w, s):
    return w.double() * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)


class Layer:
    def __init__(self, d, F, E, K, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.d, self.F, self.E, self.K = d, F, E, K
        self.norm = (1 + 0.2 * rnd(d)).to(BF)
        self.norm2 = (1 + 0.2 * rnd(d)).to(BF)
        self.router = (rnd(E, d) / d ** 0.5).to(BF)
        self.bias = 0.3 * rnd(E)
        self.gu, self.sgu = _blocks(rnd(E, 2 * F, d) / d ** 0.5)
        self.dn, self.sdn = _blocks(rnd(E, d, F) / F ** 0.5)
        self.gus, self.sgus = _blocks(rnd(2 * F, d) / d ** 0.5)
        self.dns, self.sdns = _blocks(rnd(d, F) / F ** 0.5)
        self.rnd = rnd

    def forward(self, x, res, ws, fws, out):
        """One layer and the next one's norm; every buffer is the caller's."""
        B.kolibri_rms_norm(x, self.norm, EPS, res=res, res_out=out["res"], y=out["y"], y8=out["y8"], scales=out["s"])
        B.kolibri_router_forward_permute(out["y"], self.router, self.bias, self.K, z=out["z"], ids=out["ids"],
                                         gates=out["gates"], alpha=out["alpha"], counts=out["counts"],
                                         offsets=out["offsets"], perm=out["perm"], inv=out["inv"], ws=ws)
        B.kolibri_expert_ffn_fp8(out["y8"], out["s"], out["perm"], out["offsets"], out["inv"], out["gates"], self.gu,
                                 self.sgu, self.dn, self.sdn, self.gus, self.sgus, self.dns, self.sdns, y=out["ffn"], ws=fws)
        B.kolibri_rms_norm(out["ffn"], self.norm2, EPS, res=out["res"], res_out=out["res2"], y=out["y2"])

    def buffers(self, N):
        d, E, K = self.d, self.E, self.K
        e = lambda *s, t=torch.float32: torch.empty(*s, device="cuda", dtype=t)  # noqa: E731
        return dict(res=e(N, d, t=BF), y=e(N, d, t=BF), y8=e(N, d, t=F8), s=e(N, d // 128), z=e(N, E), ids=e(N, K, t=torch.int32),
                    gates=e(N, K), alpha=e(N), counts=e(E, t=torch.int32), offsets=e(E + 1, t=torch.int64),
                    perm=e(N * K, t=torch.int32), inv=e(N * K, t=torch.int32), ffn=e(N, d, t=BF), res2=e(N, d, t=BF),
                    y2=e(N, d, t=BF))


def _experts64(L, out):
    """The layer on the y8, scales, ids and gates that the calls wrote, in 64 bits, with the magnitudes of its products."""
    x = out["y8"].double() * out["s"].double().repeat_interleave(128, 1)

    def one(a, gu, dn):
        both = a @ gu.T
        g, u = both[:, :L.F], both[:, L.F:]
        h = g * torch.sigmoid(g) * u
        s = h.abs().view(-1, L.F // 128, 128).amax(2).clamp_min(1e-30).repeat_interleave(128, 1) / 448
        q = (h / s).float().clamp(-448, 448).to(F8).double() * s
        return q @ dn.T, q.abs() @ dn.abs().T

    y, mag = one(x, _wide(L.gus, L.sgus), _wide(L.dns, L.sdns))
    ids, gates = out["ids"].long(), out["gates"].double()
    for e in range(L.E):
        t, k = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            o, m = one(x[t], _wide(L.gu[e], L.sgu[e]), _wide(L.dn[e], L.sdn[e]))
            y.index_add_(0, t, o * gates[t, k][:, None])
            mag.index_add_(0, t, m * gates[t, k][:, None])
    return y, mag


@pytest.mark.parametrize("N", [1, 9, 70, 1000])
def test_serving_block(N):
    L = Layer(512, 256, 128, 4, N)
    x, res = L.rnd(N, 512).to(BF), (2 * L.rnd(N, 512)).to(BF)
    out = L.buffers(N)
    ws = B.workspace(B.KOLIBRI_OP_PERMUTE, N, L.E, L.K)
    fws = B.expert_ffn_fp8_workspace(N, 512, 256, 4, True)
    L.forward(x, res, ws, fws, out)
    check_status()
    y, mag = _experts64(L, out)
    assert ((out["ffn"].double() - y).abs() <= 2.0 ** -3 * mag + 2.0 ** -8 * y.abs() + 1e-30).all()
    rel = float((out["ffn"].double() - y).norm() / y.norm())
    assert rel <= 2.0 ** -8, rel
    h = out["ffn"].double() + out["res"].double()
    want = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * L.norm2.double()
    assert ((out["y2"].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want.abs() + 1e-38).all()
    # captured and replayed on other inputs, and run again directly: the same bits
    x2, res2 = L.rnd(N, 512).to(BF), (2 * L.rnd(N, 512)).to(BF)
    fresh = L.buffers(N)
    L.forward(x2, res2, ws, fws, fresh)
    torch.cuda.synchronize()
    xin, rin, graph = x.clone(), res.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward(xin, rin, ws, fws, out)
    for a, b in ((x2, res2), (x, res), (x2, res2)):
        xin.copy_(a)
        rin.copy_(b)
        graph.replay()
    torch.cuda.synchronize()
    for k in out:
        assert torch.equal(out[k].view(torch.uint8), fresh[k].view(torch.uint8)), k
    check_status()


@pytest.mark.parametrize("score", [B.KOLIBRI_SCORE_SIGMOID, B.KOLIBRI_SCORE_SOFTMAX])
def test_router_training_step(score):
    """The gradient of sum gs sigma(z) + sum up L(z) back to the residual stream and the norm's weight."""
    N, d, E, K = 600, 512, 128, 4
    L = Layer(d, 256, E, K, 77)
    x, res = L.rnd(N, d).to(BF), (2 * L.rnd(N, d)).to(BF)
    h, y, _, _ = B.kolibri_rms_norm(x, L.norm, EPS, res=res)
    z, ids, gates, alpha = B.kolibri_router_forward(y, L.router, L.bias, K)
    seq = torch.tensor([0, 250, 600], device="cuda")
    up = torch.tensor([0.7, 1.3], device="cuda") * 30
    gs = L.rnd(N, E) * 1e-3
    gz = B.kolibri_score_grad_to_logits(z, gs)
    B.kolibri_balance_loss(z, ids, 0.5, seq_offsets=seq, score=score, grad_loss=up, gz=gz, accumulate=True)
    gy = gz @ L.router.float()
    gres = (L.rnd(N, d) * 1e-3).to(BF)
    gx, gw = B.kolibri_rms_norm_grad(gy, h, L.norm, EPS, gres=gres)
    check_status()

    hh = h.double().requires_grad_()
    w = L.norm.double().requires_grad_()
    y64 = hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + EPS) * w
    zz = (y64 + (y.double() - y64).detach()) @ L.router.double().T          # bf16 y, its gradient straight through
    total = (gs.double() * torch.sigmoid(zz)).sum() + (hh * gres.double()).sum()
    for s, (a, b) in enumerate(((0, 250), (250, 600))):
        f = torch.bincount(ids[a:b].reshape(-1).long(), minlength=E).double() * E / (K * (b - a))
        q = torch.softmax(zz[a:b], 1) if score == B.KOLIBRI_SCORE_SOFTMAX else torch.sigmoid(zz[a:b])
        total = total + float(up[s]) * 0.5 * (f * (q / q.sum(1, keepdim=True)).mean(0)).sum()
    total.backward()
    assert float((gx.double() - hh.grad).norm() / hh.grad.norm()) <= 2.0 ** -8 + 2.0 ** -10
    assert float((gw.double() - w.grad).norm() / w.grad.norm()) <= 2.0 ** -10


def test_calls_on_a_stream_of_their_own_with_buffers_of_theirs():
    """Two streams at once, each call allocating what it needs: the memory of one is not handed to the other."""
    L = Layer(512, 256, 64, 2, 5)
    N = 300
    xs = [L.rnd(N, 512).to(BF) for _ in range(2)]
    bufs = [L.buffers(N) for _ in range(2)]
    for b, x in zip(bufs, xs):
        L.forward(x, x, B.workspace(B.KOLIBRI_OP_PERMUTE, N, L.E, L.K), B.expert_ffn_fp8_workspace(N, 512, 256, 2, True), b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            b = bufs[i]
            y = B.kolibri_expert_ffn_fp8(b["y8"], b["s"], b["perm"], b["offsets"], b["inv"], b["gates"], L.gu, L.sgu, L.dn,
                                         L.sdn, L.gus, L.sgus, L.dns, L.sdns, stream=st)
            loss = B.kolibri_balance_loss(b["z"], b["ids"], 0.1, want_gz=True, stream=st)
            gx, gw = B.kolibri_rms_norm_grad(b["y"], b["res"], L.norm, EPS, stream=st)
            got[i].append((y, *loss, gx, gw))
    torch.cuda.synchronize()
    for i in range(2):
        for row in got[i]:
            assert torch.equal(row[0], bufs[i]["ffn"])
            assert all(torch.equal(a, b) for a, b in zip(row, got[i][0]))
    check_status()


@pytest.mark.parametrize("which", ["norm", "norm_grad", "balance", "balance_grad", "experts"])
def test_memory_of_a_call_on_another_stream(which):
    """A call on a busy stream that allocates what it needs.  What the current stream allocates meanwhile is not the
    call's workspace, and memory that the current stream has still to read is not given to the call."""
    L = Layer(512, 256, 64, 2, 6)
    N = 1100                                  # the loss has a workspace from 1025 rows on
    x = L.rnd(N, 512).to(BF)
    b = L.buffers(N)
    L.forward(x, x, B.workspace(B.KOLIBRI_OP_PERMUTE, N, L.E, L.K), B.expert_ffn_fp8_workspace(N, 512, 256, 2, True), b)
    counts = torch.bincount(b["ids"].reshape(-1).long(), minlength=L.E).to(torch.int32).view(1, L.E)
    lib = B.load()
    call, ws_bytes = {
        "norm": (lambda st: B.kolibri_rms_norm(x, L.norm, EPS, res=x, want_fp8=True, stream=st), 4),
        "norm_grad": (lambda st: B.kolibri_rms_norm_grad(b["y"], b["res"], L.norm, EPS, stream=st),
                      lib.kolibri_rms_norm_grad_workspace_size(N, 512)),
        "balance": (lambda st: B.kolibri_balance_loss(b["z"], b["ids"], 0.1, want_gz=True, stream=st),
                    lib.kolibri_balance_loss_workspace_size(N, L.E, 1)),
        "balance_grad": (lambda st: (B.kolibri_balance_loss_grad(b["z"], counts, 2, 0.1, stream=st),), 4),
        "experts": (lambda st: (B.kolibri_expert_ffn_fp8(b["y8"], b["s"], b["perm"], b["offsets"], b["inv"], b["gates"],
                                                         L.gu, L.sgu, L.dn, L.sdn, L.gus, L.sgus, L.dns, L.sdns, stream=st),),
                    lib.kolibri_expert_ffn_fp8_workspace_size(N, 512, 256, 2, 1)),
    }[which]
    want = call(None)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(40_000_000)
    got = call(st)
    mine = [torch.full((ws_bytes,), 3, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all((m == 3).all() for m in mine)
    assert all(torch.equal(a.view(torch.uint8), w.view(torch.uint8)) for a, w in zip(got, want))
    held = [torch.full((w.numel() * w.element_size(),), 5, dtype=torch.uint8, device="cuda") for w in want for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)
    copies = [h.clone() for h in held]
    del held
    got = call(st)
    torch.cuda.synchronize()
    assert all((c == 5).all() for c in copies)
    assert all(torch.equal(a.view(torch.uint8), w.view(torch.uint8)) for a, w in zip(got, want))
    check_status()


def test_two_graphs_with_one_workspace():
    """Two batches captured apart on the same workspaces, replayed in turn: each leaves its own results."""
    L = Layer(512, 256, 64, 2, 8)
    sizes = (700, 90)
    fws = B.expert_ffn_fp8_workspace(max(sizes), 512, 256, 2, True).fill_(255)
    pws = [B.workspace(B.KOLIBRI_OP_PERMUTE, n, L.E, L.K) for n in sizes]
    nbytes = max(max(B.load().kolibri_balance_loss_workspace_size(n, L.E, 1), B.load().kolibri_rms_norm_grad_workspace_size(n, 512))
                 for n in sizes)
    lws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    runs = []
    for n, pw in zip(sizes, pws):
        x, b = L.rnd(n, 512).to(BF), L.buffers(n)
        o = dict(loss=torch.zeros(1, device="cuda"), counts=torch.zeros(1, L.E, dtype=torch.int32, device="cuda"),
                 prob=torch.zeros(1, L.E, device="cuda"), gz=torch.zeros(n, L.E, device="cuda"),
                 gx=torch.zeros(n, 512, dtype=BF, device="cuda"), gw=torch.zeros(512, device="cuda"))

        def call(x=x, b=b, o=o, pw=pw):
            L.forward(x, x, pw, fws, b)
            B.kolibri_balance_loss(b["z"], b["ids"], 0.1, gz=o["gz"], loss=o["loss"], counts=o["counts"], prob=o["prob"],
                                   ws=lws)
            B.kolibri_rms_norm_grad(b["y"], b["res"], L.norm, EPS, gx=o["gx"], gweight=o["gw"], ws=lws)

        call()
        torch.cuda.synchronize()
        out = [b["ffn"], *o.values()]
        want = [t.clone() for t in out]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for t in out:
            t.fill_(1)
        runs.append((graph, out, want, call))          # call holds the arrays that the graph reads
    for i in (0, 1, 1, 0, 1, 0, 0):
        runs[i][0].replay()
    torch.cuda.synchronize()
    for _, out, want, _ in runs:
        assert all(torch.equal(a, w) for a, w in zip(out, want))
    check_status()
