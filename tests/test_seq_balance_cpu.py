"""The balance loss over packed sequences without a GPU: the oracle against the per-image loss, torch
autograd and differences, and the calls that the library refuses before it launches anything."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_moe_layer_03_b200 import binding as B

FAKE = 1 << 40          # never dereferenced: validation fails first


def _case(T=60, D=12, E=5, K=2, seed=0):
    rng = np.random.default_rng(seed)
    x, wg, b = rng.standard_normal((T, D)), rng.standard_normal((E, D)), rng.standard_normal(E)
    P = O.softmax_scores(O.gate_logits(x, wg, b))
    idx, _ = O.topk_route(P, K)
    return x, wg, b, P, idx


def test_equal_lengths_are_the_per_image_loss():
    x, wg, b, P, idx = _case()
    loss, per, counts, _ = O.balance_packed(idx, P, 2, 0.01, np.arange(0, 61, 15))
    assert abs(loss - O.balance_loss_per_sequence(idx, P, 2, 0.01, 15)) < 1e-15
    assert np.array_equal(counts.sum(0), O.expert_counts(idx, 5)) and len(per) == 4
    whole = O.balance_packed(idx, P, 2, 0.01, [0, 60])
    assert abs(whole[0] - O.balance_loss(O.expert_counts(idx, 5), P, 2, 0.01)) < 1e-15
    np.testing.assert_allclose(O.softmax_backward(P, whole[3]),
                               O.balance_loss_grad_logits(P, O.expert_counts(idx, 5), 2, 0.01), rtol=1e-12)


@pytest.mark.parametrize("offsets", [[0, 7, 7, 30, 60], [5, 20, 21, 55], [0, 60], [3, 3, 3]])
def test_gradient_matches_autograd_and_differences(offsets):
    x, wg, b, P, idx = _case(seed=len(offsets))
    K, alpha = 2, 0.3
    _, _, counts, dP = O.balance_packed(idx, P, K, alpha, offsets)
    dl = O.softmax_backward(P, dP)
    dwg, db, dx = O.router_backward(x, wg, dl)

    def loss(x, wg, b):                               # the counts held constant
        p = torch.softmax(x @ wg.t() + b, 1)
        full = [i for i in range(len(offsets) - 1) if offsets[i + 1] > offsets[i]]
        total = 0.0 * p.sum()
        for i in full:
            lo, hi = offsets[i], offsets[i + 1]
            total = total + alpha * (5 / (K * (hi - lo)) * torch.tensor(counts[i]).double() * p[lo:hi].mean(0)).sum()
        return total / max(len(full), 1)
    args = [torch.tensor(v, requires_grad=True) for v in (x, wg, b)]
    loss(*args).backward()
    for got, want in zip((dx, dwg, db), args):
        np.testing.assert_allclose(got, want.grad.numpy(), rtol=1e-9, atol=1e-14)
    # central differences: the third derivative's h^2 and the fp64 loss's 1e-16 / h, h = 1e-5
    rng = np.random.default_rng(1)
    for got, k in ((dx, 0), (dwg, 1), (db, 2)):
        step = rng.standard_normal(got.shape)
        with torch.no_grad():
            v = [torch.tensor(a) for a in (x, wg, b)]
            ends = [loss(*[u + s * 1e-5 * torch.tensor(step) if i == k else u for i, u in enumerate(v)]) for s in (1, -1)]
        assert abs(float(ends[0] - ends[1]) / 2e-5 - float((got * step).sum())) < 1e-8


def _call(cfg, n=2, off=FAKE, x=FAKE, wg=FAKE, bias=None, idx=FAKE, n_sel=None, dgate=None, aux=1.0, counts=FAKE,
          seq_loss=FAKE, loss=FAKE, dwg=FAKE, dbias=None, dx=None, acc=0, bws=FAKE, nb=None, ws=FAKE):
    nb = B.lib.moe_seq_balance_workspace_size(ctypes.byref(cfg), max(n, 0)) if nb is None else nb
    return B.lib.moe_seq_balance(ctypes.byref(cfg), x, wg, bias, off, n, idx, n_sel, dgate, aux, counts, seq_loss, loss,
                                 dwg, dbias, dx, acc, bws, nb, ws, None)


def test_arguments_are_refused_before_a_launch():
    cfg = B.make_config(1024, 384, 64, 8, 2, 0)
    per = B.make_config(1024, 384, 64, 8, 2, 0, seq_len=256)
    race = B.make_config(1024, 384, 64, 8, 2, 0, routing="race")
    need = B.moe_seq_balance_workspace_size(cfg, 2)
    cases = [(cfg, dict(n=-1), b"n_seqs"), (cfg, dict(off=None), b"n_seqs"), (per, dict(off=None, n=3), b"n_seqs"),
             (cfg, dict(dwg=None, dx=FAKE), b"dwg"), (cfg, dict(dwg=None, dbias=FAKE), b"dwg"),
             (cfg, dict(dwg=None, dgate=FAKE), b"dwg"), (cfg, dict(acc=1), b"dx_accumulate"),
             (cfg, dict(aux=float("nan")), b"aux_scale"), (race, {}, b"n_sel"), (cfg, dict(counts=None), b"seq_counts"),
             (cfg, dict(seq_loss=None), b"seq_loss"), (cfg, dict(loss=None), b"loss"), (cfg, dict(dwg=FAKE + 4), b"dwg"),
             (cfg, dict(dbias=FAKE + 8), b"dbias"), (cfg, dict(bws=None), b"bws"), (cfg, dict(bws=FAKE + 16), b"bws"),
             (cfg, dict(ws=None), b"ws"), (cfg, dict(x=None), b"x"), (cfg, dict(x=FAKE + 2), b"x"), (cfg, dict(wg=None), b"wg"),
             (cfg, dict(idx=None), b"topk_idx"), (cfg, dict(bias=FAKE + 4), b"router_bias"),
             (cfg, dict(off=FAKE + 4), b"seq_offsets"), (cfg, dict(dgate=FAKE + 4), b"dgate"),
             (cfg, dict(n_sel=FAKE + 4), b"n_sel"), (cfg, dict(dx=FAKE + 8), b"dx"), (cfg, dict(dx=FAKE), b"one buffer")]
    for c, kw, word in cases:
        assert _call(c, **kw) == B.MOE_ERR_INVALID_ARG, kw
        assert word in B.lib.moe_last_error(), (kw, B.lib.moe_last_error())
    assert _call(cfg, nb=need - 1) == B.MOE_ERR_WORKSPACE
    assert _call(cfg, n=300000) == B.MOE_ERR_UNSUPPORTED
    with pytest.raises(B.MoeError):
        B.moe_seq_balance_workspace_size(cfg, -1)
    with pytest.raises(B.MoeError):
        B.moe_seq_balance_workspace_size(B.make_config(1024, 100, 64, 8, 2, 0), 1)


def test_workspace_covers_every_shape():
    for dt in ("f32", "bf16", "f16"):
        for T in (0, 1, 17, 32768, 262144):
            n = B.moe_seq_balance_workspace_size(B.make_config(T, 1152, 64, 16, 2, 0, dt), 1)
            assert n % 256 == 0 and n >= T * 12
