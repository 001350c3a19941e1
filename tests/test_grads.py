"""The global norm and clipping of gradients on the GPU against 64-bit sums.

Bounds.  The norm is a 64-bit sum rounded once to fp32: half a step, 2^-24, and
as much again for the 64-bit roundings.  A clipped value is grad times an fp32
factor: the factor's half step and the product's, 2^-23 in all, and for bf16 the
last rounding's 2^-8; below the normal numbers half a subnormal step."""
import math

import pytest
import torch

from test_product import ep  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def clip(ep, grads, outs, max_norm, split=1):  # noqa: F811
    """The library's clipping; with `split`, of as many lists whose sums are added up."""
    total = torch.zeros(1, dtype=torch.float64, device="cuda")
    lists = []
    for i in range(split):
        lists.append(ep.Grads.make(grads[i::split], outs[i::split]))
        ws = torch.full((ep.ep_grad_workspace_bytes(lists[-1]),), 255, dtype=torch.uint8, device="cuda")
        part = torch.full((1,), 7.0, dtype=torch.float64, device="cuda")
        ep.ep_grad_square_sum(lists[-1], part, ws)
        total += part
    norm = torch.full((2,), 7.0, device="cuda")
    for one in lists:
        ep.ep_grad_clip(one, total, max_norm, norm)
    assert norm[1] == 7
    return float(norm[0]), float(total)


def check(grads, outs, before, norm, square, max_norm):
    exact = sum(float((b.double() ** 2).sum()) for b in before)
    assert abs(square - exact) <= 2.0 ** -40 * exact
    assert abs(norm - math.sqrt(exact)) <= 2.0 ** -23 * math.sqrt(exact)
    root = math.sqrt(square)
    factor = max_norm / root if root > max_norm else 1.0
    for o, b in zip(outs, before):
        if factor == 1.0:
            assert torch.equal(o, b)
            continue
        want = b.double() * factor
        tol = want.abs() * (2.0 ** -23 + (2.0 ** -8 if o.dtype == BF else 0)) + (2.0 ** -133 if o.dtype == BF else 2.0 ** -149)
        assert ((o.double() - want).abs() <= tol).all()


def flat_views(sizes, dtype, offset, seed):
    """Consecutive pieces of one buffer, from an odd place on, with a value between them that nobody owns."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn(sum(sizes) + len(sizes) + offset + 8, device="cuda", generator=g).to(dtype)
    views, at = [], offset
    for n in sizes:
        views.append(buf[at:at + n])
        at += n + 1
    return buf, views


SIZES = [0, 1, 2, 3, 7, 8, 9, 15, 16, 17, 4095, 16383, 16384, 16385, 16391, 16392, 32768 + 5, 100003]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_sizes_and_addresses(ep, dtype, offset, shift):  # noqa: F811
    """shift: how far the outputs' addresses are from the gradients', in values."""
    for max_norm in (0.5, 1e9):
        buf, grads = flat_views(SIZES, dtype, offset, offset)
        before = [g.clone() for g in grads]
        held = buf.clone()
        target = torch.full((buf.numel() + 16,), 77.0, device="cuda", dtype=dtype)
        outs, at = [], offset + shift
        for n in SIZES:
            outs.append(target[at:at + n])
            at += n + 1
        norm, square = clip(ep, grads, outs, max_norm)
        check(grads, outs, before, norm, square, max_norm)
        assert torch.equal(buf, held)
        owned = torch.zeros(target.numel(), dtype=torch.bool, device="cuda")
        at = offset + shift
        for n in SIZES:
            owned[at:at + n] = True
            at += n + 1
        assert (target[~owned] == 77).all()
        # in place: the same, and what lies between stays
        norm2, square2 = clip(ep, grads, grads, max_norm)
        assert (norm2, square2) == (norm, square)
        assert all(torch.equal(g, o) for g, o in zip(grads, outs))
        if max_norm > 1e6:
            assert torch.equal(buf, held)


@pytest.mark.parametrize("split", [1, 3])
def test_many_gradients_of_both_types(ep, split):  # noqa: F811
    """More than a launch holds, of either type, empty ones among them, and lists that several ranks would hold."""
    g = torch.Generator().manual_seed(1)
    sizes = torch.randint(0, 3000, (200,), generator=g).tolist()
    grads = [(torch.randn(n, generator=g) * 10 ** (i % 5 - 2)).to(BF if i % 3 else FP).cuda() for i, n in enumerate(sizes)]
    before = [t.clone() for t in grads]
    outs = [torch.empty_like(t) for t in grads]
    norm, square = clip(ep, grads, outs, 2.0, split)
    check(grads, outs, before, norm, square, 2.0)
    assert (norm, square) == clip(ep, grads, outs, 2.0, split)


def test_magnitudes_that_fp32_squares_lose(ep):  # noqa: F811
    for size in (1e25, 3e38, 1e-25, 1e-38):
        grads = [torch.full((1000,), size, device="cuda"), torch.full((999,), -size, device="cuda", dtype=BF)]
        before = [t.clone() for t in grads]
        outs = [torch.empty_like(t) for t in grads]
        for max_norm in (0.0, 1e-30, 1.0, 1e38, math.inf):
            norm, square = clip(ep, grads, outs, max_norm)
            exact = sum(float((b.double() ** 2).sum()) for b in before)
            assert abs(square - exact) <= 2.0 ** -40 * exact
            root = math.sqrt(square)
            factor = max_norm / root if root > max_norm else 1.0
            for o, b in zip(outs, before):
                want = b.double() * factor
                # the factor itself may be a subnormal number
                tol = want.abs() * (2.0 ** -23 + 2.0 ** -8) + b.double().abs() * 2.0 ** -149 + 2.0 ** -133
                assert ((o.double() - want).abs() <= tol).all()


def test_norms_that_are_not_finite_scale_nothing(ep):  # noqa: F811
    for bad in (math.inf, -math.inf, math.nan):
        grads = [torch.randn(5000, device="cuda"), torch.randn(70, device="cuda").to(BF)]
        grads[0][4321] = bad
        before = [t.clone() for t in grads]
        outs = [torch.zeros_like(t) for t in grads]
        norm, _ = clip(ep, grads, outs, 0.1)
        assert math.isinf(norm) if math.isinf(bad) else math.isnan(norm)
        for o, b in zip(outs, before):
            assert torch.equal(o.nan_to_num(1e9, 2e9, 3e9), b.nan_to_num(1e9, 2e9, 3e9))


@pytest.mark.parametrize("shift", [0, 1])
def test_unscaled_gradients_keep_their_bits(ep, shift):  # noqa: F811
    """Signalling NaNs too, in whole vectors and in what lies before and after them."""
    for dtype, bits, pattern in ((FP, torch.int32, 0x7F800001), (BF, torch.int16, 0x7F81)):
        buf = torch.randn(5010, device="cuda").to(dtype)
        for at in (0, 1, 6, 7, 100, 4997, 4998, 4999):
            buf.view(bits)[1 + at] = pattern
        grad = buf[1:5001]
        out = torch.zeros(5010, device="cuda", dtype=dtype)[1 + shift:5001 + shift]
        norm, _ = clip(ep, [grad], [out], 0.1)
        assert math.isnan(norm) and torch.equal(out.view(bits), grad.view(bits))


def test_no_gradients(ep):  # noqa: F811
    assert clip(ep, [], [], 1.0) == (0.0, 0.0)
    empty = torch.empty(0, device="cuda")
    assert clip(ep, [empty], [empty], 1.0) == (0.0, 0.0)
    one = ep.Grads.make([torch.ones(3, device="cuda")])
    ep.ep_grad_clip(one, torch.full((1,), 3.0, dtype=torch.float64, device="cuda"), 1.0)  # without the norm
    assert torch.allclose(one.tensors[0][0], torch.full((3,), 3 ** -0.5, device="cuda"))


def test_more_than_2_31_values(ep):  # noqa: F811
    n = (1 << 31) + 12345
    g = torch.zeros(n, device="cuda", dtype=BF)
    out = torch.ones(n, device="cuda", dtype=BF)
    at = torch.tensor([0, 1, (1 << 30) + 3, (1 << 31) - 1, 1 << 31, n - 1], device="cuda")
    g[at] = 2.0
    norm, square = clip(ep, [g], [out], 1.0)
    assert square == 24.0
    want = torch.full((6,), 2.0 / math.sqrt(24.0), device="cuda", dtype=BF)
    assert torch.equal(out[at], want)
    out[at] = 0
    assert not out.view(torch.int16).view(-1).any()


def test_graph_and_stream(ep):  # noqa: F811
    """Replays follow the gradients in the captured buffers, for two graphs with workspaces of their own."""
    grads = [torch.randn(n, device="cuda").to(t) for n, t in ((5000, BF), (33, FP), (70000, FP))]
    outs = [[torch.empty_like(t) for t in grads] for _ in range(2)]
    lists = [ep.Grads.make(grads, o) for o in outs]
    ws = [torch.empty(ep.ep_grad_workspace_bytes(lists[0]), dtype=torch.uint8, device="cuda") for _ in range(2)]
    square = [torch.empty(1, dtype=torch.float64, device="cuda") for _ in range(2)]
    norm = [torch.empty(1, device="cuda") for _ in range(2)]
    batches = [[torch.randn_like(t) * s for t in grads] for s in (1, 3)]

    def step(i):
        ep.ep_grad_square_sum(lists[i], square[i], ws[i])
        ep.ep_grad_clip(lists[i], square[i], 10.0, norm[i])

    want = []
    for b in batches:
        for t, v in zip(grads, b):
            t.copy_(v)
        step(0)
        want.append([norm[0].clone()] + [t.clone() for t in outs[0]])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(1)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([norm[1], *outs[1]], want[1]))
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(i)
    for n in range(4):
        for t, v in zip(grads, batches[n % 2]):
            t.copy_(v)
        for i in range(2):
            norm[i].zero_()
            for t in outs[i]:
                t.zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip([norm[i], *outs[i]], want[n % 2]))


def test_bound_calls(ep):  # noqa: F811
    grads = [torch.randn(1000, device="cuda")]
    one = ep.Grads.make(grads, [torch.empty_like(grads[0])])
    ws = torch.empty(ep.ep_grad_workspace_bytes(one), dtype=torch.uint8, device="cuda")
    square, norm = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda")
    calls = [ep.ep_grad_square_sum(one, square, ws, bind=True), ep.ep_grad_clip(one, square, 1.0, norm, bind=True)]
    for _ in range(2):
        grads[0].mul_(2)
        for c in calls:
            c()
        exact = math.sqrt(float((grads[0].double() ** 2).sum()))
        assert abs(float(norm) - exact) <= 2.0 ** -23 * exact
