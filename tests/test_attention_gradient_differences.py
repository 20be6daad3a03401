"""attn_backward against differences of attn_prefill, in fp32, tightly enough that a gradient
scaled by 1.01 (or 0.99, 2, 0, -1), or one without the D term, is refused.

Along a direction e the fifth-order quotient

    (8 (f(h) - f(-h)) - (f(2h) - f(-2h))) / 12h

is off by h^4 / 30 times the fifth derivative: with h = 2^-5, the same quotient of the fp64 oracle
is off by at most 7e-6 of the slope at these sizes.  An output is off by about 2^-21 of a value of
order 1 (an exponent and a sum in fp32), the loss, a sum over n < 2^18 of them with random signs,
by 2^-21 sqrt(n), and the quotient by 1.5 / h times that, 0.012 at most.  The direction e has the
gradient's own signs, so that the slope is a sum of magnitudes, hundreds or more, no chance value
near 0.  Together below 1e-4 of the slope; ten times that is allowed.
"""

import pytest
import torch

from _mixers import randn

pytestmark = pytest.mark.gpu

TOL = 1e-3


def _slopes(x, do, **kw):
    """(quotient along the signs of each gradient, the gradient's own slope along them)."""
    import gated_delta_rule_79_b200 as g

    def loss(y):
        return (g.attn_prefill(*y, **kw)[0].double() * do.double()).sum().item()
    o, lse = g.attn_prefill(*x, **kw)
    out = []
    for i, grad in enumerate(g.attn_backward(*x, o, lse, do, **kw)):
        # every element moves by 2^-5 of its size, at least 2^-5 / 10
        h, e = 2.0 ** -5, grad.sign() * x[i].abs().clamp(min=0.1)

        def at(t):
            return loss([y + t * h * e if j == i else y for j, y in enumerate(x)])
        quotient = (8 * (at(1) - at(-1)) - (at(2) - at(-2))) / (12 * h)
        out.append((quotient, (grad.double() * e.double()).sum().item()))
    return out


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Tq,Tk,window,sinks", [(90, 90, 30, 2), (150, 150, 0, 0), (40, 130, 0, 0)])
def test_gradients_by_differences(d, Tq, Tk, window, sinks):
    x = [randn((2, t, n, d), s).cuda() for t, n, s in ((Tq, 4, 1), (Tk, 2, 2), (Tk, 2, 3))]
    do = randn((2, Tq, 4, d), 4).cuda()
    kw = dict(window=window, sinks=sinks)
    if Tq == Tk:
        kw["lengths"] = torch.tensor([Tk, Tk - 31], dtype=torch.int32, device="cuda")
    for name, (got, want) in zip(("dq", "dk", "dv"), _slopes(x, do, **kw)):
        assert want > 100 and abs(got - want) <= TOL * want, (name, got, want)
        for scale in (0.99, 1.01, 2.0, 0.0, -1.0):      # what the bound would refuse
            assert not abs(got - scale * want) <= TOL * abs(scale * want), (name, scale)
