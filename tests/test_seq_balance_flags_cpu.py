"""The flags of moe_seq_balance, refused before a launch, and the gradient that they are for."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_moe_layer_03_b200 import binding as B
from tests.test_seq_balance_cpu import FAKE, _call


def test_flags_are_refused_before_a_launch():
    cfg = B.make_config(1024, 384, 64, 8, 2, 0)
    for kw, word in [(dict(acc=4, dx=FAKE + 16), b"flags"), (dict(acc=-1, dx=FAKE + 16), b"flags"),
                     (dict(acc=B.MOE_SEQ_ALL_GATES), b"dgate"), (dict(acc=3, dgate=FAKE), b"dx_accumulate"),
                     (dict(acc=B.MOE_SEQ_ALL_GATES, dwg=None), b"dgate")]:
        assert _call(cfg, **kw) == B.MOE_ERR_INVALID_ARG, kw
        assert word in B.lib.moe_last_error(), (kw, B.lib.moe_last_error())


@pytest.mark.parametrize("offsets", [[5, 20, 41], [0, 30], [60, 60]])
def test_every_rows_gates_and_some_rows_balance(offsets):
    # J = sum of gate c_tk over every row + L over some: autograd against the formula
    rng = np.random.default_rng(3)
    T, D, E, K, alpha = 60, 12, 5, 2, 0.3
    x, wg, b = rng.standard_normal((T, D)), rng.standard_normal((E, D)), rng.standard_normal(E)
    P = O.softmax_scores(O.gate_logits(x, wg, b))
    idx, _ = O.topk_route(P, K)
    c = rng.standard_normal((T, K))
    dP = O.balance_packed(idx, P, K, alpha, offsets)[3]
    np.add.at(dP, (np.arange(T)[:, None], idx), c)
    dwg, db, dx = O.router_backward(x, wg, O.softmax_backward(P, dP))
    args = [torch.tensor(v, requires_grad=True) for v in (x, wg, b)]
    p = torch.softmax(args[0] @ args[1].t() + args[2], 1)
    J = (torch.tensor(c) * p.gather(1, torch.tensor(np.asarray(idx)).long())).sum()
    spans = [(lo, hi) for lo, hi in zip(offsets, offsets[1:]) if hi > lo]
    for lo, hi in spans:
        f = torch.tensor(O.expert_counts(idx[lo:hi], E)).double() * E / (K * (hi - lo))
        J = J + alpha * (f * p[lo:hi].mean(0)).sum() / len(spans)
    J.backward()
    for got, want in zip((dx, dwg, db), args):
        np.testing.assert_allclose(got, want.grad.numpy(), rtol=1e-9, atol=1e-13)


def test_the_workspace_holds_each_forms_parts():
    # by part, each rounded up to 256 bytes: tokens' sequences and losses, blocks' losses, and of the form that
    # the shape takes the sums of dl for dbias (3 router warps in each of up to 148 blocks, or one of each 16
    # tokens), dl's fragments and the partial sums of dWg
    up = lambda n: -(-max(n, 1) // 256) * 256  # noqa: E731
    for T in (1, 100, 3000, 32768):
        nblk = -(-T // 16)
        groups = min(nblk, 148)
        got = B.moe_seq_balance_workspace_size(B.make_config(T, 1152, 64, 8, 2, 0, "bf16"), 4)
        want = 256 + up(8 * T) + up(4 * T) + up(4 * nblk) + up(nblk * 3 * 512) + up(0) + up(0) \
            + up(groups * 3 * 8 * 4) + up(groups * 8 * 1152 * 4)
        assert got == want, (T, got, want)
