"""dx and dweight against central differences of the 64-bit forward pass, each
by itself: along the gradient's own direction, where no cancellation hides a
mistake, over one expert's rows or one half of its weight at a time.

The inputs make every pre-activation exact in bf16 (an odd number of at most
161 over 32, never 0): x is -1, 0 or 1, the weights multiples of 1/16 up to
1/8, the bias 1/32, over 40 inputs.  So the backward call reads what the forward pass
has, no relu is at its corner, and a gradient is off by what its own call
rounds: the bounds of product_reference.backward, summed with the magnitudes of
the direction."""
import pytest
import torch

import product_reference as ref

C, N, E = 40, 24, 2
BIAS = 1 / 32


def inputs(rows, act):
    """x, w, dout for `rows` rows of the receive buffer."""
    g = torch.Generator().manual_seed(11)
    M = N * (2 if ref.gated(act) else 1)
    x = torch.randint(-1, 2, (rows, C), generator=g).bfloat16()
    w = (torch.randint(-2, 3, (E, M, C), generator=g) / 16).bfloat16()
    return x, w, torch.randn(rows, N, generator=g).bfloat16()


def pre_activations(x, w, of):
    pre = torch.zeros(x.shape[0], w.shape[1], dtype=ref.F64)
    for e, rows in of.items():
        pre[rows] = x[rows].double() @ w[e].double().t() + BIAS
    assert torch.equal(pre, pre.bfloat16().double()) and (pre[sorted(sum(of.values(), []))].abs() >= BIAS).all()
    return pre.bfloat16()


def check(act, x, w, dout, of, dx, dw):
    """dx and dw (tensors of the library's or a stand-in's results) hold against differences; returns the largest
    tolerance relative to its derivative."""
    def loss(x, w):
        total = 0.0
        for e, rows in of.items():
            v = x[rows] @ w[e].t() + BIAS
            total += (ref.activate(act, v, torch.zeros_like(v))[0] * dout[rows].double()).sum()
        return total

    x64, w64 = x.double(), w.double()
    pre = pre_activations(x, w, of)
    worst = 0.0
    for e, rows in of.items():
        want = ref.backward(act, dout[rows], pre[rows], x[rows], w[e])
        directions = [("dx", slice(None))]
        directions += [("dweight", slice(h * N, (h + 1) * N)) for h in range(w.shape[1] // N)]
        for name, part in directions:
            g, bound = (t[part] for t in want[name])
            v = g / g.norm()
            vx, vw = torch.zeros_like(x64), torch.zeros_like(w64)
            if name == "dx":
                vx[rows] = v
                got = dx[rows].double()
            else:
                vw[e, part] = v
                got = dw[e, part].double()
            num = [(loss(x64 + h * vx, w64 + h * vw) - loss(x64 - h * vx, w64 - h * vw)) / (2 * h) for h in (1e-4, 2e-4)]
            # a central difference's error grows fourfold with a doubled step
            tolerance = (bound * v.abs()).sum() + (num[1] - num[0]).abs() + 1e-6 * num[0].abs()
            value = (got * v).sum()
            assert (value - num[0]).abs() <= tolerance, (name, e, float(value), float(num[0]), float(tolerance))
            worst = max(worst, float(tolerance / num[0].abs()))
    return worst


def stand_in(act, x, w, dout, of, drop=None):
    """What the backward call computes, in 64 bits with its roundings; without the half `drop` of dpre."""
    pre = pre_activations(x, w, of)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for e, rows in of.items():
        d = ref.act_grad(act, pre[rows], dout[rows]).bfloat16().double()
        if drop is not None:
            d[:, drop * N:(drop + 1) * N] = 0
        dx[rows] = (d @ w[e].double()).bfloat16()
        dw[e] = (d.t() @ x[rows].double()).bfloat16()
    return dx, dw


@pytest.mark.parametrize("act", ref.ACTS)
def test_the_check_sees_mistakes(act):
    of = {0: list(range(0, 15)), 1: list(range(18, 27))}
    x, w, dout = inputs(30, act)
    dx, dw = stand_in(act, x, w, dout, of)
    assert check(act, x, w, dout, of, dx, dw) < 0.15
    wrong = [(dx * 0, dw), (dx, dw * 0), (dx * 1.25, dw), (dx, dw * 1.25), (dx * 0.75, dw), (dx, dw * 0.75),
             (dx.roll(1, 0), dw), (dx, dw.roll(1, 1))]
    if ref.gated(act):
        for half in range(2):
            bad = stand_in(act, x, w, dout, of, drop=half)
            wrong += [(bad[0], dw), (dx, bad[1])]
        wrong.append((dx, dw.roll(N, 1)))
    for bad in wrong:
        with pytest.raises(AssertionError):
            check(act, x, w, dout, of, *bad)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ref.ACTS)
def test_gradients_against_differences_of_one_input(act):
    import combine_ep_get_amd as ep
    from test_product import Routed, marked

    r = Routed(ep, 24, E, 1, seed=4)
    q = ep.Product.make(C, N, ref.ACTS.index(act))
    M = q.weight_rows
    x, w, dout = inputs(r.rows, act)
    bias = torch.full((E, M), BIAS, device="cuda")
    pre, out = marked(r.rows, M), marked(r.rows, N)
    ep.ep_expert_product(r.p, q, x.cuda(), *r.arrays, w.cuda(), bias, None, pre, out)
    assert torch.equal(pre[r.used].cpu(), pre_activations(x, w, r.of)[r.used])
    dx, dw = marked(r.rows, C), marked(E, M, C)
    none = act == "none"
    ep.ep_expert_product_backward(r.p, q, dout.cuda(), None if none else pre, x.cuda(), *r.arrays, w.cuda(),
                                  None if none else marked(r.rows, M), dx, dw)
    check(act, x, w, dout, r.of, dx.cpu(), dw.cpu())
