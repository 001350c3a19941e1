"""Gradients of the experts' products on the GPU against their 64-bit forms and against differences."""
import pytest
import torch

import product_reference as ref
from test_product import Routed, ep, marked, normal, untouched  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [
    # T, C, N, E, K, R, A, act
    (1, 8, 8, 1, 1, 1, 1, "silu"),
    (3, 200, 24, 8, 2, 2, 1, "swiglu"),
    (40, 72, 136, 4, 2, 1, 4, "geglu"),
    (130, 328, 264, 3, 2, 1, 16, "gelu"),
    (257, 136, 72, 5, 3, 5, 1, "relu"),
    (300, 264, 200, 4, 2, 2, 1, "none"),
    (1300, 264, 328, 2, 2, 1, 1, "swiglu"),
    (300, 2056, 136, 8, 1, 1, 1, "geglu"),    # 128 x 128 tiles
    (2400, 2056, 136, 24, 1, 2, 1, "silu"),   # 256 x 256 tiles
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_backward(ep, case):  # noqa: F811
    T, C, N, E, K, R, A, act = case
    r = Routed(ep, T, E, K, R, A, empty=0.1 if T > 4 else 0.0, hot=True, seed=T)
    q = ep.Product.make(C, N, ref.ACTS.index(act))
    M = q.weight_rows
    g = torch.Generator().manual_seed(T + 1)
    x, w, dout = normal(g, r.rows, C), normal(g, E, M, C, scale=C ** -0.5), normal(g, r.rows, N)
    pre = normal(g, r.rows, M) if act != "none" else None
    dpre = marked(r.rows, M) if act != "none" else None
    dx, dw = marked(r.rows, C), marked(E, M, C)
    before = torch.randn(E, M, C, generator=g)
    acc, db = before.cuda(), torch.full((E, M), 7.0, device="cuda")
    ws = torch.empty(ep.ep_product_workspace_bytes(r.p, q), dtype=torch.uint8, device="cuda")
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    d = [cuda(t) for t in (dout, pre, x, w)]
    ep.ep_expert_product_backward(r.p, q, d[0], d[1], d[2], *r.arrays, d[3], dpre, dx, dw, acc, db, ws)
    for e, rows in r.of.items():
        want = ref.backward(act, dout[rows], dout[rows] if pre is None else pre[rows], x[rows], w[e])
        if pre is not None:
            ref.assert_within(dpre[rows], *want["dpre"], f"dpre of expert {e}")
        ref.assert_within(dx[rows], *want["dx"], f"dx of expert {e}")
        ref.assert_within(dw[e], *want["dweight"], f"dweight of expert {e}")
        v, b = want["dweight_acc"]
        v = v + before[e].double()
        ref.assert_within(acc[e], v, b + ref.ULP32 * v.abs(), f"dweight_acc of expert {e}")
        ref.assert_within(db[e], *want["dbias"], f"dbias of expert {e}")
    assert untouched(dx, r.used)
    # each output alone gives the same bits, and dpre may take pre's place
    dx2, dw2, db2 = marked(r.rows, C), marked(E, M, C), torch.empty_like(db)
    scratch = d[1].clone() if pre is not None else None
    ep.ep_expert_product_backward(r.p, q, d[0], scratch, None, *r.arrays, d[3], scratch, dx2)
    scratch = d[1].clone() if pre is not None else None
    ep.ep_expert_product_backward(r.p, q, d[0], scratch, d[2], *r.arrays, None, scratch, None, dw2)
    scratch = d[1].clone() if pre is not None else None
    ep.ep_expert_product_backward(r.p, q, d[0], scratch, None, *r.arrays, None, scratch, None, None, None, db2, ws)
    assert torch.equal(dx2.view(torch.int16), dx.view(torch.int16))
    assert torch.equal(dw2.view(torch.int16), dw.view(torch.int16)) and torch.equal(db2, db)


def test_no_tokens_zero_the_weight_gradients(ep):  # noqa: F811
    q = ep.Product.make(72, 40, ep.EP_ACT_SILU)
    r = Routed(ep, 0, 4, 2)
    dw, db = marked(4, 40, 72), torch.full((4, 40), 7.0, device="cuda")
    ws = torch.empty(ep.ep_product_workspace_bytes(r.p, q), dtype=torch.uint8, device="cuda")
    ep.ep_expert_product_backward(r.p, q, None, None, None, *r.arrays, None, None, None, dw, None, db, ws)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("act", ref.ACTS)
def test_gradients_against_differences(ep, act):  # noqa: F811
    """dx and dweight from the library against central differences of the
    64-bit forward pass, along random directions."""
    T, C, N, E = 24, 40, 24, 2
    r = Routed(ep, T, E, 1, seed=4)
    q = ep.Product.make(C, N, ref.ACTS.index(act))
    M = q.weight_rows
    g = torch.Generator().manual_seed(8)
    x, w, dout = normal(g, r.rows, C), normal(g, E, M, C, scale=C ** -0.5), normal(g, r.rows, N)
    d = [t.cuda() for t in (x, w, dout)]
    pre, out = marked(r.rows, M), marked(r.rows, N)
    ep.ep_expert_product(r.p, q, d[0], *r.arrays, d[1], None, None, pre, out)
    dx, dw = marked(r.rows, C), marked(E, M, C)
    none = act == "none"
    dpre = None if none else marked(r.rows, M)
    ep.ep_expert_product_backward(r.p, q, d[2], None if none else pre, d[0], *r.arrays, d[1], dpre, dx, dw)

    def loss(x, w):
        return sum((ref.activate(act, x[rows] @ w[e].t(), torch.zeros(len(rows), M, dtype=ref.F64))[0] * dout[rows].double()).sum()
                   for e, rows in r.of.items())

    used = torch.tensor(r.used)
    for _ in range(3):
        vx, vw = torch.randn(x.shape, generator=g).double(), torch.randn(w.shape, generator=g).double()
        h = 1e-6
        num = (loss(x.double() + h * vx, w.double() + h * vw) - loss(x.double() - h * vx, w.double() - h * vw)) / (2 * h)
        gx, gw = dx.cpu().double()[used], dw.cpu().double()
        got = (gx * vx[used]).sum() + (gw * vw).sum()
        # pre, dpre and the two gradients are each rounded to bf16; a relu's
        # pre-activation may cross zero by its rounding only where it is tiny.
        # Each rounding is off by 2^-8 of its value at most: bound the sum of
        # the errors of the terms by 4 roundings of the terms' magnitudes,
        # through magnitudes of dx and dw that no cancellation shrinks.
        big = dout.double().abs().mean() * N
        scale = (gx.abs() * vx[used].abs()).sum() + (gw.abs() * vw.abs()).sum() + big
        assert abs(got - num) <= 4 * ref.HALF_BF16 * scale, (float(got), float(num), float(scale))
