"""The balance loss, its counts and its gradient against the formulas in 64
bits.

Bars.  The fast exponential is within 2 + 1.2 |x| units of 2^-23 (CUDA's
stated bound), 2^-18.5 for |x| <= 16; p = q / sum q carries it twice, with 25
additions and two divisions of 2^-22: p is within 2^-17 relative, and so is P
and 1 - sigma, plus (rows per warp) 2^-24 for P's sum: at most 64 rows here.
With D = |f_e - 1| + sum_j |f_j - 1| p_j, the bracket f_e - sum f p is within
2^-16 D, so gz within 2^-15 of scale p D slope.  L = lambda (1 + mean dot):
within 2^-16 lambda (1 + mean_t sum_j |f_j - 1| p_j)."""
import pytest
import torch

from expert_load_balancing_b200 import binding as B

from gpu_helpers import check_status

pytestmark = pytest.mark.gpu

SCORES = [B.KOLIBRI_SCORE_SIGMOID, B.KOLIBRI_SCORE_SOFTMAX]


@pytest.fixture(scope="module", autouse=True)
def _lib(kolibri_lib):
    return kolibri_lib


def _plain(z, ids, lam, cut, score, up):
    """Loss, counts, P, gz and the bars of the last three, from the formulas."""
    N, E = z.shape
    K = ids.shape[1]
    z = z.double()
    out = dict(loss=[], counts=[], prob=[], gz=z.new_zeros(N, E), gbar=z.new_zeros(N, E), lbar=[])
    for s in range(len(cut) - 1):
        a, b = cut[s], cut[s + 1]
        T = b - a
        if T == 0:
            out["loss"].append(z.new_zeros(()))
            out["lbar"].append(z.new_zeros(()))
            out["counts"].append(torch.zeros(E, dtype=torch.int64, device=z.device))
            out["prob"].append(z.new_zeros(E))
            continue
        c = torch.zeros(E, dtype=torch.int64, device=z.device)
        c.index_add_(0, ids[a:b].reshape(-1).long(), torch.ones(T * K, dtype=torch.int64, device=z.device))
        f = c.double() * E / (K * T)
        zz = z[a:b]
        logq = zz if score == B.KOLIBRI_SCORE_SOFTMAX else torch.nn.functional.logsigmoid(zz)
        none = (zz == -torch.inf).all(1, keepdim=True)
        p = torch.softmax(torch.where(none, 0.0, logq), 1) * ~none
        slope = torch.ones_like(p) if score == B.KOLIBRI_SCORE_SOFTMAX else torch.sigmoid(-zz)
        k = lam * float(up[s]) / T
        out["gz"][a:b] = k * p * (f - (p * f).sum(1, keepdim=True)) * slope
        D = (f - 1).abs() + (p * (f - 1).abs()).sum(1, keepdim=True)
        out["gbar"][a:b] = 2.0 ** -15 * abs(k) * p * D * slope + 1e-37
        out["counts"].append(c)
        out["prob"].append(p.mean(0))
        out["loss"].append(lam * (f * out["prob"][-1]).sum())
        out["lbar"].append(2.0 ** -16 * abs(lam) * (1 + (p * (f - 1).abs()).sum(1).mean()))
    for n in ("loss", "counts", "prob", "lbar"):
        out[n] = torch.stack(out[n])
    return out


def _check(got, want):
    loss, counts, prob, gz = got
    assert torch.equal(counts.long(), want["counts"])
    assert ((loss.double() - want["loss"]).abs() <= want["lbar"] + 1e-30).all()
    assert ((prob.double() - want["prob"]).abs() <= 2.0 ** -16 * want["prob"] + 1e-37).all()
    if gz is not None:
        err = (gz.double() - want["gz"]).abs()
        assert torch.isfinite(gz).all()
        assert (err <= want["gbar"]).all(), float((err / want["gbar"].clamp_min(1e-300)).max())


def _inputs(N, E, K, cut, seed, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(N, E, generator=g, device="cuda") * spread + torch.randn(E, generator=g, device="cuda")
    ids = torch.topk(z + 0.2 * torch.randn(E, generator=g, device="cuda"), K, dim=1).indices.to(torch.int32)
    S = len(cut) - 1
    up = torch.rand(S, generator=g, device="cuda") * 2 - 0.5
    return z, ids, torch.tensor(cut, dtype=torch.int64, device="cuda"), up


CASES = [
    # either side of the small form, with few slots and with many
    (682, 384, 6, [0, 682]), (683, 384, 6, [0, 683]), (683, 384, 5, [3, 680]), (512, 512, 9, [0, 512]), (512, 512, 3, [20, 500]),
    (1024, 256, 16, [0, 1024]), (1024, 256, 4, [1, 1024]), (1024, 256, 3, [700, 1024]),
    (1, 4, 1, [0, 1]), (1024, 384, 6, [0, 1024]), (1024, 512, 3, [100, 900]), (1025, 384, 6, [0, 1025]), (1000, 64, 8, [0, 0]), (513, 200, 2, [7, 513]), (900, 128, 4, [0, 3]), (1, 384, 6, [0, 1]), (2, 8, 3, [0, 1, 2]), (5, 132, 8, [0, 0, 5, 5]), (7, 128, 8, [0, 7]),
    (256, 384, 6, [0, 256]), (257, 260, 2, [0, 100, 100, 257]), (1000, 512, 16, [0, 1, 2, 3, 500, 1000]),
    (4096, 384, 6, [0, 4096]), (5003, 128, 8, [0, 17, 4000, 4000, 4001, 5003]), (700, 64, 1, list(range(0, 701))),
    (6000, 12, 5, [0, 2999, 6000]), (40001, 256, 4, [0, 12345, 40001]),
    # more sequences than a block keeps boundaries of, most of them empty
    (1500, 64, 2, [0] * 400 + sorted((7 * i) % 1501 for i in range(1501)) + [1500] * 9),
]


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("N,E,K,cut", CASES)
def test_loss_counts_and_gradient(N, E, K, cut, score):
    z, ids, seq, up = _inputs(N, E, K, cut, N + E)
    want = _plain(z, ids, 1e-3, cut, score, up)
    one = cut == [0, N]
    got = B.kolibri_balance_loss(z, ids, 1e-3, seq_offsets=seq, score=score, grad_loss=up, want_gz=True)
    _check(got, want)
    # forward alone, the gradient alone, and again: the same bits
    loss, counts, prob, none = B.kolibri_balance_loss(z, ids, 1e-3, seq_offsets=None if one else seq, score=score)
    assert none is None and torch.equal(loss, got[0]) and torch.equal(counts, got[1]) and torch.equal(prob, got[2])
    gz = B.kolibri_balance_loss_grad(z, counts, K, 1e-3, seq_offsets=seq, score=score, grad_loss=up)
    _check((loss, counts, prob, gz), want)
    assert torch.equal(gz, got[3])
    # added to what is there: one fp32 addition more
    base = torch.randn_like(z) * 1e-6
    acc = base.clone()
    B.kolibri_balance_loss_grad(z, counts, K, 1e-3, seq_offsets=seq, score=score, grad_loss=up, gz=acc, accumulate=True)
    total = base.double() + want["gz"]
    assert ((acc.double() - total).abs() <= want["gbar"] + 2.0 ** -23 * (base.double().abs() + total.abs())).all()
    acc2 = base.clone()
    B.kolibri_balance_loss(z, ids, 1e-3, seq_offsets=seq, score=score, grad_loss=up, gz=acc2, accumulate=True)
    assert torch.equal(acc, acc2)
    check_status()


@pytest.mark.parametrize("score", SCORES)
def test_padding_is_not_read(score):
    """Rows before the first and behind the last sequence hold NaN logits and ids of nowhere."""
    N, E, K, cut = 900, 384, 6, [37, 400, 400, 811]
    z, ids, seq, up = _inputs(N, E, K, cut, 3)
    want = _plain(z, ids, 0.5, cut, score, up)
    outside = torch.ones(N, dtype=torch.bool, device="cuda")
    outside[37:811] = False
    z[outside] = float("nan")
    ids[outside] = 1 << 30
    got = B.kolibri_balance_loss(z, ids, 0.5, seq_offsets=seq, score=score, grad_loss=up, want_gz=True)
    _check(got, want)
    assert not got[3][outside].any()
    kept = torch.full((N, E), 3.0, device="cuda")
    B.kolibri_balance_loss_grad(z, got[1], K, 0.5, seq_offsets=seq, score=score, grad_loss=up, gz=kept, accumulate=True)
    assert (kept[outside] == 3.0).all()
    check_status()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("N", [64, 1100])
def test_extreme_logits(score, N):
    """-infinity for some experts and for a whole row, rows far below zero, far above, the type's lowest value."""
    E, K = 128, 4
    z, ids, seq, up = _inputs(N, E, K, [0, N], 5)
    z[:, 5] = -torch.inf
    z[3] = -torch.inf
    z[7] -= 300.0
    z[9] -= 3000.0
    z[11] += 80.0
    z[13, ::2] = torch.finfo(torch.float32).min
    want = _plain(z, ids, 1.0, [0, N], score, up)
    got = B.kolibri_balance_loss(z, ids, 1.0, seq_offsets=seq, score=score, grad_loss=up, want_gz=True)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[2]).all() and torch.isfinite(got[3]).all()
    assert not got[3][3].any() and not got[3][:, 5].any()
    assert ((got[0].double() - want["loss"]).abs() <= 4 * want["lbar"]).all()       # P is held to four times its bar below
    alone = B.kolibri_balance_loss(z, ids, 1.0, seq_offsets=seq, score=score)
    assert torch.equal(alone[0], got[0]) and torch.equal(alone[2], got[2])
    # logits of this size enter the exponential unreduced: their rows are held to the units it is then off by
    big = torch.zeros(N, 1, dtype=torch.float64, device="cuda")
    big[[7, 9, 11]] = 1.0
    slack = want["gbar"] * (1 + 64 * big)
    assert ((got[3].double() - want["gz"]).abs() <= slack).all()
    assert ((got[2].double() - want["prob"]).abs() <= 2.0 ** -14 * want["prob"] + 1e-37).all()
    check_status()


def test_bad_ids_and_offsets_are_reported():
    N, E, K = 300, 64, 4
    z, ids, seq, up = _inputs(N, E, K, [0, 100, N], 6)
    for bad in (-1, E, 1 << 30):
        broken = ids.clone()
        broken[17, 2] = bad
        _, counts, _, _ = B.kolibri_balance_loss(z, broken, 1e-3, seq_offsets=seq)
        assert B.kolibri_device_status() == B.KOLIBRI_ERR_DEVICE
        assert int(counts.sum()) == N * K - 1          # the others are counted
    twice = ids.clone()
    twice[:, 1] = twice[:, 0]
    _, counts, _, _ = B.kolibri_balance_loss(z, twice, 1e-3)
    assert int(counts.sum()) == N * K
    assert torch.equal(counts[0].long(), torch.bincount(twice.reshape(-1).long(), minlength=E))
    for cut in ([0, 200, 100], [-5, 100, N], [0, 100, N + 1], [300, 0, 300], [0, N + 1], [200, 100], [-1, N]):
        B.kolibri_balance_loss(z, ids, 1e-3, seq_offsets=torch.tensor(cut, device="cuda"), want_gz=True)
        assert B.kolibri_device_status() == B.KOLIBRI_ERR_DEVICE
    check_status()


@pytest.mark.parametrize("score", SCORES)
def test_gradient_reports_bad_offsets(score):
    """The gradient alone checks its boundaries as the loss does, in whichever part of them the fault is."""
    N, E, K = 300, 64, 4
    z, ids, seq, up = _inputs(N, E, K, [0, 100, N], 6)
    counts = B.kolibri_balance_loss(z, ids, 1e-3, seq_offsets=seq)[1]
    B.kolibri_balance_loss_grad(z, counts, K, 1e-3, seq_offsets=seq, score=score)
    check_status()
    for cut in ([0, 200, 100], [-5, 100, N], [0, 100, N + 1], [300, 0, 300], [0, N + 1], [200, 100], [-1, N]):
        S = len(cut) - 1
        B.kolibri_balance_loss_grad(z, counts[:1].expand(S, E).contiguous(), K, 1e-3, seq_offsets=torch.tensor(cut, device="cuda"), score=score)
        assert B.kolibri_device_status() == B.KOLIBRI_ERR_DEVICE, cut
    # more boundaries than a block keeps, the fault behind them
    many = torch.arange(5001, device="cuda").clamp(max=N)
    one = torch.ones(5000, E, device="cuda", dtype=torch.int32)
    B.kolibri_balance_loss_grad(z, one, K, 1e-3, seq_offsets=many, score=score)
    check_status()
    for at, v in ((0, -1), (2500, N - 1), (4999, 0), (5000, N + 1)):
        bad = many.clone()
        bad[at] = v
        B.kolibri_balance_loss_grad(z, one, K, 1e-3, seq_offsets=bad, score=score)
        assert B.kolibri_device_status() == B.KOLIBRI_ERR_DEVICE, (at, v)
    check_status()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("E", [64, 68, 128, 132, 384, 388])
def test_a_row_that_is_not_a_number_shows(E, score):
    """NaN logits, in a whole row or at one place of it, make their sequence's loss and P and their rows' gradient NaN in
    every form of the pass, and touch nothing else."""
    N, K = 512, 4
    z, ids, seq, up = _inputs(N, E, K, [0, N, N], 8)
    clean = B.kolibri_balance_loss(z, ids, 1e-3, seq_offsets=seq[:2].contiguous(), score=score, want_gz=True)[3]
    for cols in (slice(None), slice(5, 6)):
        broken = z.clone()
        broken[77, cols] = float("nan")
        for s in (seq[:2].contiguous(), seq):              # one sequence: the small form; two: the passes
            loss, counts, prob, gz = B.kolibri_balance_loss(broken, ids, 1e-3, seq_offsets=s, score=score, want_gz=True)
            alone = B.kolibri_balance_loss(broken, ids, 1e-3, seq_offsets=s, score=score)
            apart = B.kolibri_balance_loss_grad(broken, counts, K, 1e-3, seq_offsets=s, score=score)
            assert loss[0].isnan() and prob[0].isnan().all() and alone[0][0].isnan() and alone[2][0].isnan().all()
            assert not loss[1:].any() and not prob[1:].any()
            for t in (gz, apart):
                assert t[77].isnan().all()
                keep = torch.arange(N, device="cuda") != 77
                assert torch.equal(t[keep], clean[keep])
    check_status()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("N", [64, 1100])
def test_rows_far_from_zero_keep_their_bar(score, N):
    """Rows far below and above zero are held to the gradient's bar itself: the row's maximum (zero, for sigmoid scores of
    positive logits) is taken off before the exponential, so only z - c counts there.

    |z - c| is below 32 and exact but for one rounding; its product with log2 e (whose constant is half a step off too) has
    2^-23 of at most 47, the exponential 2^-22: together under 2^-17 relative.  p carries that twice, with its additions and
    the reciprocal under 2^-16, and the bracket with it stays inside the 2^-15 of the head of this file.  With sigmoid scores
    the row at +80 has scores of 1, so p has its additions' 2^-19 only, and a slope from exp(-z) with 2^-23 * 130 * ln 2,
    under 2^-16; one below the normal numbers is flushed, which is less than the bar's 1e-37."""
    E, K = 128, 4
    z, ids, seq, up = _inputs(N, E, K, [0, N], 5)
    z[7] -= 300.0
    z[9] -= 3000.0
    z[11] += 80.0
    want = _plain(z, ids, 1.0, [0, N], score, up)
    gz = B.kolibri_balance_loss(z, ids, 1.0, seq_offsets=seq, score=score, grad_loss=up, want_gz=True)[3]
    err = (gz.double() - want["gz"]).abs()
    assert (err <= want["gbar"]).all(), float((err / want["gbar"]).max())


@pytest.mark.parametrize("N", [512, 4096])
def test_even_loads_have_the_formulas_loss(N):
    """Every expert equally loaded: f = 1, so L = lambda and the gradient vanishes, exactly."""
    E, K = 64, 2
    z = torch.randn(N, E, device="cuda")
    ids = (torch.arange(N * K, device="cuda") % E).view(N, K).to(torch.int32)
    loss, counts, prob, gz = B.kolibri_balance_loss(z, ids, 0.25, want_gz=True)
    assert (counts == N * K // E).all() and float(loss) == 0.25 and not gz.any()


@pytest.mark.parametrize("score", SCORES)
def test_gradient_against_differences(score):
    """Central differences of the formula's loss in 64 bits along a direction, per sequence weighted by up."""
    N, E, K, cut = 48, 20, 3, [0, 11, 48]
    z, ids, seq, up = _inputs(N, E, K, cut, 12, spread=1.0)
    gz = B.kolibri_balance_loss(z, ids, 0.7, seq_offsets=seq, score=score, grad_loss=up, want_gz=True)[3]
    v = torch.randn(N, E, device="cuda").double()

    def total(zz):
        return float((_plain(zz, ids, 0.7, cut, score, up)["loss"] * up.double()).sum())

    e = 1e-5
    diff = (total(z.double() + e * v) - total(z.double() - e * v)) / (2 * e)
    terms = gz.double() * v
    assert abs(float(terms.sum()) - diff) <= 2.0 ** -14 * float(terms.abs().sum()) + 1e-8


def test_refusals():
    z, ids, seq, up = _inputs(16, 64, 4, [0, 4, 16], 2)
    for kw in (dict(z=z.double()), dict(z=z.t()), dict(ids=ids.long()), dict(ids=ids[:3]), dict(seq_offsets=seq.int()),
               dict(grad_loss=up[:1]), dict(gz=z[:4]), dict(loss=up[:1]), dict(counts=ids), dict(prob=z),
               dict(accumulate=True, want_gz=True), dict(ids=ids.cpu())):
        a = dict(z=z, ids=ids, seq_offsets=seq) | kw
        zz, ii = a.pop("z"), a.pop("ids")
        with pytest.raises(ValueError):
            B.kolibri_balance_loss(zz, ii, 1e-3, **a)
    with pytest.raises(B.KolibriError):
        B.kolibri_balance_loss(z, ids, 1e-3, score=5)
    with pytest.raises(B.KolibriError):
        B.kolibri_balance_loss(z, ids, float("nan"))
    with pytest.raises(B.KolibriError):
        B.kolibri_balance_loss(z, ids, 1e-3, seq_offsets=seq, ws=torch.empty(64, device="cuda", dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.kolibri_balance_loss_grad(z, ids, 4, 1e-3)


@pytest.mark.parametrize("N,cut", [(3001, [0, 1000, 3001]), (500, [3, 500])])
def test_other_stream_and_graph(N, cut):
    E, K = 384, 6
    z, ids, seq, up = _inputs(N, E, K, cut, 9)
    want = B.kolibri_balance_loss(z, ids, 1e-3, seq_offsets=seq, grad_loss=up, want_gz=True)
    out = [torch.empty_like(t) for t in want]
    ws = torch.empty(B.load().kolibri_balance_loss_workspace_size(N, E, len(cut) - 1), device="cuda", dtype=torch.uint8)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()

    def run(stream=None):
        B.kolibri_balance_loss(z, ids, 1e-3, seq_offsets=seq, grad_loss=up, loss=out[0], counts=out[1], prob=out[2],
                               gz=out[3], ws=ws, stream=stream)

    run(stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for t in out:
        t.fill_(0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    check_status()


def test_rows_behind_32_bit_offsets():
    """2.2e9 logits: the last rows come out as those rows do in a sequence of their own."""
    N, E, K, tail = 4_300_000, 512, 2, 1000
    z = torch.empty(N, E, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    ids = torch.randint(0, E, (N, K), device="cuda", dtype=torch.int32)
    seq = torch.tensor([0, N - tail, N], device="cuda")
    loss, counts, prob, gz = B.kolibri_balance_loss(z, ids, 1e-2, seq_offsets=seq, want_gz=True)
    zt, it = z[-tail:].contiguous(), ids[-tail:].contiguous()
    l2, c2, p2, g2 = B.kolibri_balance_loss(zt, it, 1e-2, want_gz=True)
    assert torch.equal(counts[1], c2[0]) and torch.equal(gz[-tail:], g2)
    assert ((prob[1] - p2[0]).abs() <= 2.0 ** -16 * p2[0]).all() and abs(float(loss[1] - l2[0])) <= 2.0 ** -15 * float(l2[0])
    assert int(counts[0].sum()) == (N - tail) * K
    check_status()
