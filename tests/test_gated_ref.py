"""The 64-bit form of the gated recurrence that the GPU tests compare with, against automatic
differentiation of its definition and against differences."""
import pytest
import torch

import gated_ref as R


def inputs(L, B, D, seed, z=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(x=n(L, B, D), ag=n(L, B, D), xg=n(L, B, D), param=n(D) - 3, ab=n(D), xb=n(D), z=n(L, B, D) if z else None,
                h0=n(B, D)), n(L, B, D), n(B, D)


def loss(x, ag, xg, param, ab, xb, z, h0, dy, dlast, scale):
    h, total = h0, 0.0
    for t in range(x.shape[0]):
        a = torch.exp(-scale * torch.nn.functional.softplus(param) * torch.sigmoid(ag[t] + ab))
        h = a * h + torch.sqrt(1 - a * a) * torch.sigmoid(xg[t] + xb) * x[t]
        total = total + ((h if z is None else h * torch.nn.functional.silu(z[t])) * dy[t]).sum()
    return total + (h * dlast).sum()


@pytest.mark.parametrize("z", [True, False])
def test_gradients_against_automatic_differentiation(z):
    t, dy, dlast = inputs(7, 3, 5, 1, z)
    ask = {k: v.clone().requires_grad_(True) for k, v in t.items() if v is not None}
    full = dict(ask, z=ask.get("z"))
    grads = dict(zip(ask, torch.autograd.grad(loss(**full, dy=dy, dlast=dlast, scale=2.5), list(ask.values()))))
    got = R.backward(**t, dy=dy, dlast=dlast, scale=2.5)
    names = dict(x="dx", ag="da_gate", xg="dx_gate", param="da_param", ab="da_bias", xb="dx_bias", z="dz", h0="dinitial_state")
    for k, v in grads.items():
        torch.testing.assert_close(got[names[k]][0], v, rtol=1e-9, atol=1e-11)


def test_gradients_against_differences():
    """Central differences with step s are off by s^2 / 6 of the third derivative and 2^-53 / s of the value."""
    t, dy, dlast = inputs(4, 1, 2, 2)
    got = R.backward(**t, dy=dy, dlast=dlast, scale=8.0)
    names = dict(x="dx", ag="da_gate", xg="dx_gate", param="da_param", ab="da_bias", xb="dx_bias", z="dz", h0="dinitial_state")
    s = 1e-5
    for k, name in names.items():
        flat = got[name][0].reshape(-1)
        for j in range(t[k].numel()):
            vals = []
            for sign in (1, -1):
                moved = t[k].clone()
                moved.view(-1)[j] += sign * s
                vals.append(loss(**dict(t, **{k: moved}), dy=dy, dlast=dlast, scale=8.0).item())
            assert abs((vals[0] - vals[1]) / (2 * s) - flat[j].item()) < 1e-7


def test_a_decay_of_one_has_the_gradient_of_the_limit():
    """As the recurrence gate closes, the gradients through it go to 0 and those of the state stay."""
    t, dy, dlast = inputs(5, 2, 3, 3)
    t["ag"][2] = -torch.inf
    at = R.backward(**t, dy=dy, dlast=dlast)
    t["ag"][2] = -60.0
    near = R.backward(**t, dy=dy, dlast=dlast)
    for k in at:
        assert torch.isfinite(at[k][0]).all()
        torch.testing.assert_close(at[k][0], near[k][0], rtol=1e-8, atol=1e-8)


def test_the_forward_is_the_definition():
    t, dy, _ = inputs(6, 2, 4, 4)
    y, ey, h, eh = R.forward(**t, scale=8.0)
    assert (ey > 0).all() and (ey < 1e-4).all() and (eh < 1e-4).all()
    zero = torch.zeros_like(t["h0"])
    torch.testing.assert_close((y * dy).sum(), loss(**t, dy=dy, dlast=zero, scale=8.0), rtol=1e-12, atol=1e-12)
