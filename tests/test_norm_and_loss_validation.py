"""Host-side argument checks of the norm, its gradient and the balance loss
(no device needed: each case fails before anything is enqueued), and of the
Python calls' own checks."""
import math

import pytest
import torch

from expert_load_balancing_b200 import binding as B

INVALID, SHAPE, SMALL = 1, 2, 3
F = 0x10000        # a 16-byte aligned address that is never dereferenced
ODD = 0x10004      # a misaligned one
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def lib(kolibri_lib):
    return kolibri_lib


def test_rms_norm_checks(lib):
    f = lib.kolibri_rms_norm
    #        x  xt    res rt    w  wt    eps   N   d     res_out y  y8 scales stream
    assert f(None, BF16, F, BF16, F, BF16, 1e-6, 16, 2560, F, F, None, None, None) == INVALID
    assert f(ODD, BF16, F, BF16, F, BF16, 1e-6, 16, 2560, F, F, None, None, None) == INVALID
    assert f(F, 2, F, BF16, F, BF16, 1e-6, 16, 2560, F, F, None, None, None) == INVALID          # type codes
    assert f(F, BF16, F, -1, F, BF16, 1e-6, 16, 2560, F, F, None, None, None) == INVALID
    assert f(F, BF16, F, BF16, F, 7, 1e-6, 16, 2560, F, F, None, None, None) == INVALID
    assert f(F, BF16, None, BF16, F, BF16, 1e-6, 16, 2560, F, F, None, None, None) == INVALID    # res_out needs res
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, 16, 2560, F, None, None, None, None) == INVALID    # no output
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, 16, 2560, F, F, F, None, None) == INVALID          # y8 without scales
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, 16, 2560, F, F, None, F, None) == INVALID
    assert f(F, BF16, F, BF16, F, BF16, -1.0, 16, 2560, F, F, None, None, None) == INVALID
    assert f(F, BF16, F, BF16, F, BF16, math.nan, 16, 2560, F, F, None, None, None) == INVALID
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, 0, 2560, F, F, None, None, None) == INVALID
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, 16, 2564, F, F, None, None, None) == SHAPE         # d % 8
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, 16, 16392, F, F, None, None, None) == SHAPE        # d > 16384
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, 1 << 31, 2560, F, F, None, None, None) == SHAPE


def test_rms_norm_grad_checks(lib):
    need = lib.kolibri_rms_norm_grad_workspace_size(4096, 2560)
    assert need >= 4 * 2560 and need % 4 == 0
    assert lib.kolibri_rms_norm_grad_workspace_size(0, 2560) == 0
    assert lib.kolibri_rms_norm_grad_workspace_size(16, 2561) == 0
    f = lib.kolibri_rms_norm_grad
    #        gy gyt   h  ht    w  wt    eps   gres N     d     gx gw ws ws_bytes stream
    assert f(None, BF16, F, BF16, F, BF16, 1e-6, None, 4096, 2560, F, F, F, need, None) == INVALID
    assert f(F, BF16, ODD, BF16, F, BF16, 1e-6, None, 4096, 2560, F, F, F, need, None) == INVALID
    assert f(F, 3, F, BF16, F, BF16, 1e-6, None, 4096, 2560, F, F, F, need, None) == INVALID
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, ODD, 4096, 2560, F, F, F, need, None) == INVALID
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, None, 4096, 2560, None, F, F, need, None) == INVALID
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, None, 4096, 2560, F, F, None, need, None) == INVALID   # gweight needs ws
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, None, 4096, 2560, F, F, F, need - 1, None) == SMALL
    assert f(F, BF16, F, BF16, F, BF16, 1e-6, None, 4096, 4, F, F, F, need, None) == SHAPE


def test_balance_loss_checks(lib):
    size = lib.kolibri_balance_loss_workspace_size
    n, E, K, S = 4096, 384, 6, 5
    need = size(n, E, S)
    assert need >= 4 * E * (S + 1)
    assert size(682, E, 1) == 0 and size(683, E, 1) > 0 and size(682, E, 2) > 0      # a small batch needs none
    assert size(1024, 64, 1) == 0 and size(1025, 64, 1) > 0
    assert size(0, E, S) == 0 and size(n, 0, S) == 0 and size(n, 513, S) == 0 and size(n, E, 0) == 0
    f = lib.kolibri_balance_loss
    #        z  ids seq N  E  K  S  score lambda gl acc loss counts prob gz ws ws_bytes stream
    assert f(None, F, F, n, E, K, S, 0, 1e-3, F, 0, F, F, F, F, F, need, None) == INVALID
    assert f(F, ODD, F, n, E, K, S, 0, 1e-3, F, 0, F, F, F, F, F, need, None) == INVALID
    assert f(F, F, None, n, E, K, S, 0, 1e-3, F, 0, F, F, F, F, F, need, None) == INVALID       # no offsets: one sequence
    assert f(F, F, F, n, E, K, 0, 0, 1e-3, F, 0, F, F, F, F, F, need, None) == INVALID
    assert f(F, F, F, n, E, K, S, 2, 1e-3, F, 0, F, F, F, F, F, need, None) == INVALID          # score
    assert f(F, F, F, n, E, K, S, 0, math.inf, F, 0, F, F, F, F, F, need, None) == INVALID
    assert f(F, F, F, n, E, K, S, 0, 1e-3, F, 2, F, F, F, F, F, need, None) == INVALID          # accumulate
    assert f(F, F, F, n, E, K, S, 0, 1e-3, F, 0, F, F, None, F, F, need, None) == INVALID
    assert f(F, F, F, n, E, K, S, 0, 1e-3, F, 0, F, F, F, F, None, need, None) == INVALID
    assert f(F, F, F, n, E, K, S, 0, 1e-3, F, 0, F, F, F, F, F, need - 1, None) == SMALL
    assert f(F, F, F, n, E, E, S, 0, 1e-3, F, 0, F, F, F, F, F, need, None) == INVALID          # K >= E
    assert f(F, F, F, n, 386, K, S, 0, 1e-3, F, 0, F, F, F, F, F, need, None) == SHAPE          # E % 4
    assert f(F, F, F, n, E, K, 1 << 24, 0, 1e-3, F, 0, F, F, F, F, F, need, None) == SHAPE      # S E
    g = lib.kolibri_balance_loss_grad
    #        z  counts seq N  E  K  S  score lambda gl acc gz stream
    assert g(F, None, F, n, E, K, S, 0, 1e-3, F, 0, F, None) == INVALID
    assert g(F, F, F, n, E, K, S, 0, 1e-3, F, 0, None, None) == INVALID
    assert g(F, F, F, n, E, K, S, 0, 1e-3, ODD, 0, F, None) == INVALID
    assert g(F, F, None, n, E, K, 2, 0, 1e-3, F, 0, F, None) == INVALID
    assert g(F, F, F, 0, E, K, S, 0, 1e-3, F, 0, F, None) == INVALID


def test_python_calls_refuse_cpu_tensors_and_wrong_types():
    from expert_load_balancing_b200 import binding as B
    x = torch.zeros(4, 64)
    with pytest.raises((ValueError, RuntimeError)):
        B.kolibri_rms_norm(x, torch.ones(64), 1e-6)
    with pytest.raises((ValueError, RuntimeError)):
        B.kolibri_rms_norm_grad(x, x, torch.ones(64), 1e-6)
    with pytest.raises((ValueError, RuntimeError)):
        B.kolibri_balance_loss(x, torch.zeros(4, 2, dtype=torch.int32), 1e-3)
    with pytest.raises((ValueError, RuntimeError)):
        B.kolibri_balance_loss_grad(x, torch.zeros(1, 64, dtype=torch.int32), 2, 1e-3)


@pytest.mark.parametrize("bounds", [[], [0]])
def test_python_calls_refuse_boundaries_of_no_sequence(bounds):
    seq = torch.tensor(bounds, dtype=torch.int64)
    z, ids, counts = torch.zeros(8, 16), torch.zeros(8, 2, dtype=torch.int32), torch.zeros(1, 16, dtype=torch.int32)
    with pytest.raises(ValueError, match="seq_offsets"):
        B.kolibri_balance_loss(z, ids, 1e-3, seq_offsets=seq)
    with pytest.raises(ValueError, match="seq_offsets"):
        B.kolibri_balance_loss_grad(z, counts, 2, 1e-3, seq_offsets=seq)


def test_expert_fp8_checks(lib):
    size = lib.kolibri_expert_ffn_fp8_workspace_size
    n, d, Fh, E, K = 4096, 2560, 512, 384, 6
    need = size(n, d, Fh, K, 1)
    assert need >= n * (K + 1) * (Fh + 4 * Fh // 128 + 2 * d) and size(n, d, Fh, K, 0) < need
    assert size(0, d, Fh, K, 1) == 0 and size(n, 384, Fh, K, 1) == 0 and size(n, d, 64, K, 1) == 0
    assert size(n, d, Fh, 17, 1) == 0
    f = lib.kolibri_expert_ffn_fp8

    def call(skip=(), odd=(), n=n, d=d, Fh=Fh, E=E, K=K, ws_bytes=need):
        # x8 xs perm offs inv gates wgu sgu wd sd wgu_s sgu_s wd_s sd_s y ... ws
        ptr = [None if i in skip else ODD if i in odd else F for i in range(16)]
        return f(*ptr[:15], n, d, Fh, E, K, ptr[15], ws_bytes, None)

    for i in range(16):
        assert call(skip=(i,)) == INVALID, i            # one of the shared four alone missing is refused too
        assert call(odd=(i,)) == INVALID, i
    assert call(ws_bytes=need - 1) == SMALL
    assert call(n=0) == INVALID and call(K=0) == INVALID and call(K=17) == INVALID and call(E=0) == INVALID
    assert call(d=2432) == SHAPE and call(Fh=192) == SHAPE and call(E=513) == SHAPE and call(d=8448) == SHAPE
    assert call(n=1 << 29) == SHAPE


def test_row_counts_whose_products_leave_64_bits_are_refused(lib):
    """N K and N (K + 1) of such an N wrap round to a few rows: the call has to look at N first."""
    d, Fh, E = 2560, 512, 384
    for n, K in (((1 << 60) + 1, 15), ((1 << 59) + 1, 16), ((1 << 62) + 1, 3), ((1 << 62) + 1, 4), ((1 << 61) + 3, 8)):
        assert lib.kolibri_expert_ffn_fp8_workspace_size(n, d, Fh, K, 1) == 0, (n, K)
        assert lib.kolibri_expert_ffn_fp8(*[F] * 15, n, d, Fh, E, K, F, 1 << 62, None) == SHAPE, (n, K)
        assert lib.kolibri_balance_loss(F, F, None, n, E, K, 1, 0, 1e-3, None, 0, F, F, F, None, F, 1 << 62, None) == SHAPE, (n, K)
        assert lib.kolibri_balance_loss_grad(F, F, None, n, E, K, 1, 0, 1e-3, None, 0, F, None) == SHAPE, (n, K)
        assert lib.kolibri_workspace_bytes(1, n, E, K) == 0, (n, K)
        assert lib.kolibri_router_topk(F, F, n, E, K, F, F, F, None) == SHAPE, (n, K)
        assert lib.kolibri_expert_ffn(*[F] * 10, n, d, Fh, E, K, F, 1 << 62, None) == SHAPE, (n, K)
        assert lib.kolibri_expert_dispatch(F, F, n, d, K, F, None) == SHAPE, (n, K)
        assert lib.kolibri_expert_combine(F, F, F, F, n, d, K, F, None) == SHAPE, (n, K)
    for n in (1 << 31, 1 << 62, (1 << 63) - 1):
        assert lib.kolibri_balance_loss_workspace_size(n, E, 1) == 0 and lib.kolibri_balance_loss_workspace_size(n, E, 2) == 0
