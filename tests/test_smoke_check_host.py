"""The smoke check of the norm + rotation gradient has to tell a right gradient from a wrong one: right
ones as a kernel rounds them pass, each planted mistake is refused, for few rows and for a single wrong
element."""

import numpy as np
import pytest
import torch

import __graft_entry__ as entry

ROT, EPS, D = 64, 1e-6, 128


def table(rot=ROT):
    ang = np.arange(400)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32).astype(np.float64)


def inputs(seed, H):
    """bf16 values in 64 bits, as the smoke run has them."""
    rng = np.random.default_rng(seed)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s)).bfloat16().double().numpy()  # noqa: E731
    w = torch.linspace(0.5, 1.5, D).bfloat16().double().numpy()
    return bf(1, H, 260, D), w, bf(1, H, 260, D), np.arange(260) + 7


def gradient(x, w, dz, pos, mistake=None):
    """By automatic differentiation, in 64 bits, with one mistake planted."""
    tx, tw = torch.from_numpy(x).requires_grad_(), torch.from_numpy(w).requires_grad_()
    t = torch.from_numpy(table())[torch.from_numpy(pos)]
    c, s = t[:, :ROT // 2], t[:, ROT // 2:]
    if mistake == "rotation turned the other way":
        s = -s
    r = 1 / (tx.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    if mistake == "norm taken as constant":
        r = r.detach()
    y = tx * r * (tw * 0 + 1 if mistake == "weight left out" else tw)
    lo, hi = y[..., :ROT // 2], y[..., ROT // 2:ROT]
    z = torch.cat([lo * c - hi * s, hi * c + lo * s, y[..., ROT:]], -1)
    z.backward(torch.from_numpy(dz))
    dw = tw.grad
    if mistake == "weight gradient not rotated back":
        dw = (torch.from_numpy(dz) * tx * r).sum((0, 1, 2)).detach()
    if mistake == "a row missing in the weight gradient":
        dw = dw - gradient(x[:, :1, :1], w, dz[:, :1, :1], pos[:1])[1].double()
    return tx.grad.bfloat16(), dw.detach().float()


@pytest.mark.parametrize("seed,H", [(s, h) for s in range(5) for h in (1, 2)])
def test_right_gradients_pass(seed, H):
    x, w, dz, pos = inputs(seed, H)
    entry.check_norm_rope_gradient(*gradient(x, w, dz, pos), x, w, dz, table(), pos, EPS, "right")


@pytest.mark.parametrize("mistake", ["norm taken as constant", "weight left out", "rotation turned the other way",
                                     "weight gradient not rotated back", "a row missing in the weight gradient"])
@pytest.mark.parametrize("seed,H", [(s, h) for s in range(5) for h in (1, 2)])
def test_wrong_gradients_are_refused(mistake, seed, H):
    x, w, dz, pos = inputs(seed, H)
    with pytest.raises(AssertionError, match="gradient of norm"):
        entry.check_norm_rope_gradient(*gradient(x, w, dz, pos, mistake), x, w, dz, table(), pos, EPS, mistake)


def test_one_wrong_element_is_refused():
    x, w, dz, pos = inputs(9, 2)
    dx, dw = gradient(x, w, dz, pos)
    for bad in (float("nan"), dx[0, 1, 200, 3].item() * 1.02):
        wrong = dx.clone()
        wrong[0, 1, 200, 3] = bad
        with pytest.raises(AssertionError):
            entry.check_norm_rope_gradient(wrong, dw, x, w, dz, table(), pos, EPS, "one element")
    with pytest.raises(AssertionError):
        entry.check_norm_rope_gradient(dx, dw * torch.linspace(1, 1.01, D), x, w, dz, table(), pos, EPS, "weights")
