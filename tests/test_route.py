"""The router, its balance loss and its gradient on the GPU against their 64-bit forms."""
import pytest
import torch

import route_reference as ref
from product_reference import assert_within
from test_product import ep  # noqa: F401

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def ranks(E):
    return next(r for r in range(1, E + 1) if E % r == 0 and E // r <= 256)


class Call:
    """One problem's arrays, with a marked row before and after each output."""

    def __init__(self, ep, logits, K, kind=0, normalise=True, scale=1.0, bias=None, mask=None):  # noqa: F811
        self.ep, self.logits, self.bias, self.mask, self.K = ep, logits, bias, mask, K
        self.T, self.E = logits.shape
        self.kind, self.normalise, self.scale = kind, normalise, scale
        self.p = ep.Problem.make(self.T, 64, self.E, K, ranks(self.E), 1, 1, 1)
        self.r = ep.Router.make(kind, normalise, scale, logits.dtype == torch.bfloat16)
        d = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.d_logits, self.d_bias, self.d_mask = d(logits), d(bias), d(mask)
        self.ws = torch.full((ep.ep_route_workspace_bytes(self.p, self.r),), 255, dtype=torch.uint8, device="cuda")
        self.fresh()

    def fresh(self):
        T, E, K = self.T, self.E, self.K
        self.idx = torch.full((T + 1, K), 777, dtype=torch.int32, device="cuda")
        self.w = torch.full((T + 1, K), 77.0, device="cuda")
        self.stats = [torch.full((E + 1,), 777, dtype=torch.int32, device="cuda"),
                      torch.full((2,), 777, dtype=torch.int32, device="cuda"), torch.full((E + 1,), 77.0, device="cuda"),
                      torch.full((3,), 77.0, device="cuda")]

    def route(self, stats=False):
        self.ep.ep_route(self.p, self.r, self.d_logits, self.d_bias, self.d_mask, self.idx, self.w,
                         *(self.stats + [self.ws] if stats else []))
        assert (self.idx[-1] == 777).all() and (self.w[-1] == 77).all()
        return self.idx[:-1].cpu(), self.w[:-1].cpu()

    def balance(self, idx):
        self.ep.ep_balance_loss(self.p, self.r, self.d_logits, idx.cuda(), self.d_mask, *self.stats, self.ws)

    def backward(self, idx, count, tokens, dw, dlosses):
        d = lambda t: None if t is None else t.cuda()  # noqa: E731
        out = torch.full((self.T + 1, self.E), 77.0, device="cuda", dtype=self.logits.dtype)
        self.ep.ep_route_backward(self.p, self.r, self.d_logits, d(idx), self.d_mask, d(count), d(tokens), d(dw), d(dlosses),
                                  out)
        assert (out[-1] == 77).all()
        return out[:-1].cpu()

    def check_choices(self, idx, w):
        want = ref.choose(self.kind, self.logits, self.bias, self.mask, self.K)
        assert torch.equal(idx, want), (idx != want).nonzero()[:4]
        value, bound = ref.weights(self.kind, self.normalise, self.scale, self.logits, want)
        assert_within(w, value, bound, "weights")
        return want

    def check_stats(self, idx):
        want = ref.statistics(self.kind, self.logits, idx, self.mask, self.K)
        for t, name in zip(self.stats, ("expert_count", "token_count", "prob_sum", "losses")):
            value, bound = want[name]
            assert t[-1].item() in (77, 777), name
            if name.endswith("count"):
                assert torch.equal(t[:-1].cpu().long(), torch.as_tensor(value).view(-1)), name
            else:
                assert_within(t[:-1], value, bound, name)
        return want


def inputs(T, E, bf16, seed, masked=0.0, size=1.5):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * size + torch.randn(E, generator=g) * 0.5
    mask = None
    if masked:
        mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8)
        logits[mask == 0] = NAN
    return (logits.bfloat16() if bf16 else logits), mask, g


CASES = [
    # T, E, K, kind, normalise, scale, bf16, bias, masked
    (1, 1, 1, 0, True, 1.0, False, False, 0.0),
    (1, 2, 4, 1, True, 1.0, True, False, 0.0),          # more choices than experts
    (3, 7, 3, 0, False, 2.5, False, True, 0.0),
    (5, 64, 8, 1, False, 1.0, True, True, 0.4),
    (33, 65, 6, 1, True, 2.5, False, True, 0.2),
    (100, 127, 4, 0, True, 1.0, True, False, 0.1),
    (17, 128, 32, 0, False, 1.0, False, False, 0.0),    # more choices than lanes of a token
    (128, 256, 8, 0, True, 1.0, True, False, 0.0),
    (1000, 256, 8, 1, True, 2.5, False, True, 0.05),
    (31, 255, 20, 1, False, 1.0, False, True, 0.0),
    (9, 257, 17, 1, True, 1.0, True, True, 0.3),
    (64, 512, 8, 0, False, -1.5, False, True, 0.0),
    (13, 513, 8, 0, True, 1.0, False, True, 0.2),
    (70, 1024, 32, 1, False, 1.0, True, False, 0.0),
    (6, 2047, 9, 1, True, 1.0, False, True, 0.0),
    (40, 2048, 32, 0, True, 1.0, True, False, 0.1),
    (6, 2048, 32, 0, False, 1.0, False, True, 0.0),
    (5000, 60, 4, 0, True, 1.0, False, False, 0.0),
]
ids = lambda c: "-".join(map(str, c))  # noqa: E731


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_route(ep, case):  # noqa: F811
    T, E, K, kind, normalise, scale, bf16, biased, masked = case
    logits, mask, g = inputs(T, E, bf16, T + E, masked)
    c = Call(ep, logits, K, kind, normalise, scale, torch.randn(E, generator=g) * 0.2 if biased else None, mask)
    idx, w = c.route()
    want = c.check_choices(idx, w)
    c.fresh()
    again, w2 = c.route(stats=True)
    assert torch.equal(again, idx) and torch.equal(w2, w)
    c.check_stats(want)
    first = [t.clone() for t in c.stats]
    c.fresh()
    c.balance(want)
    c.check_stats(want)
    assert all(torch.equal(a[:-1], b[:-1]) for a, b in zip(first, c.stats))


@pytest.mark.parametrize("case", CASES, ids=ids)
@pytest.mark.parametrize("terms", ["weights", "losses", "both"])
def test_route_backward(ep, case, terms):  # noqa: F811
    T, E, K, kind, normalise, scale, bf16, biased, masked = case
    logits, mask, g = inputs(T, E, bf16, T * 3 + E, masked)
    c = Call(ep, logits, K, kind, normalise, scale, None, mask)
    idx = ref.choose(kind, logits, None, mask, K)
    want = ref.statistics(kind, logits, idx, mask, K)
    count, tokens = want["expert_count"][0].int(), torch.tensor([want["token_count"][0]], dtype=torch.int32)
    dw = torch.randn(T, K, generator=g) if terms != "losses" else None
    dl = torch.tensor([3.0, 0.7]) if terms != "weights" else None
    if terms == "weights":
        got = c.backward(idx, None, None, dw, None)
    else:
        got = c.backward(idx if dw is not None else None, count, tokens, dw, dl)
    value, bound = ref.gradient(kind, normalise, scale, logits, idx, mask, count, tokens, dw, dl, K, bf16)
    assert_within(got, value, bound, "dlogits")
    if mask is not None:
        assert not got[mask == 0].any()


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("normalise", [True, False])
def test_gradient_against_differences(ep, kind, normalise):  # noqa: F811
    """Along a random direction, against differences of the objective: central ones of step h are off by h^2 of its
    third derivative, here far below the gradient's own bound."""
    T, E, K = 40, 96, 6
    logits, _, g = inputs(T, E, False, 5)
    c = Call(ep, logits, K, kind, normalise, 1.5)
    idx = ref.choose(kind, logits, None, None, K)
    st = ref.statistics(kind, logits, idx, None, K)
    count, tokens = st["expert_count"][0].int(), torch.tensor([T], dtype=torch.int32)
    dw, dl = torch.randn(T, K, generator=g), torch.tensor([2.0, 0.5])
    got = c.backward(idx, count, tokens, dw, dl).double()
    _, bound = ref.gradient(kind, normalise, 1.5, logits, idx, None, count, tokens, dw, dl, K, False)
    way = torch.randn(T, E, generator=g, dtype=torch.float64)
    live = torch.ones(T, dtype=torch.bool)
    f = lambda h: ref.objective(kind, normalise, 1.5, logits.double() + h * way, idx, live, count, T, dw, dl, K)  # noqa: E731
    h = 1e-5
    slope = (f(h) - f(-h)) / (2 * h)
    assert abs((got * way).sum() - slope) <= (bound * way.abs()).sum() + 1e-7 * (got * way).abs().sum()


def test_equal_logits_go_to_the_lowest_expert(ep):  # noqa: F811
    for E, K, bf16 in ((256, 8, False), (256, 8, True), (65, 32, False), (600, 17, True), (2048, 32, False)):
        g = torch.Generator().manual_seed(E)
        for logits in (torch.zeros(6, E), torch.randint(-2, 3, (50, E), generator=g).float(), -torch.zeros(6, E)):
            logits = logits.bfloat16() if bf16 else logits
            for bias in (None, torch.zeros(E), torch.randint(-1, 2, (E,), generator=g) * 0.25):
                for kind in (0, 1):
                    c = Call(ep, logits, K, kind, bias=bias)
                    c.check_choices(*c.route())


@pytest.mark.parametrize("E", [128, 129])
@pytest.mark.parametrize("T", [16, 32, 33, 64, 1024, 1025, 4096, 4097])
def test_where_forms_change(ep, T, E):  # noqa: F811
    """Both sides of the numbers of tokens at which another number of workgroups or of lanes works."""
    logits, _, g = inputs(T, E, T % 2 == 1, T, 0.0)
    c = Call(ep, logits, 6, 1, True, 1.0, torch.randn(E, generator=g) * 0.2)
    want = c.check_choices(*c.route(stats=True))
    c.check_stats(want)
    first = [t.clone() for t in c.stats]
    c.fresh()
    c.balance(want)
    assert all(torch.equal(a[:-1], b[:-1]) for a, b in zip(first, c.stats))


def test_signed_zeros_are_equal(ep):  # noqa: F811
    logits = torch.tensor([[0.0, -0.0, 0.0, -0.0, -1.0], [-0.0, 0.0, -0.0, 0.0, 1.0]])
    idx, _ = Call(ep, logits, 4).route()
    assert idx.tolist() == [[0, 1, 2, 3], [4, 0, 1, 2]]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("E", [40, 256, 700])
def test_sums_that_differ_below_fp32(ep, kind, E):  # noqa: F811
    """The bias makes every expert's sum with its score equal but for fp32's rounding of the bias: the order is that
    of the sums in 64 bits."""
    g = torch.Generator().manual_seed(E)
    row = torch.randn(1, E, generator=g)
    s = ref.scores(kind, row.double())[0][0]
    bias = (0.75 - s).float()
    for logits in (row, torch.cat([row, row.flip(1), row * 0.5], 0)):
        c = Call(ep, logits, 16, kind, bias=bias)
        idx = c.route()[0]
        assert torch.equal(idx, ref.choose(kind, logits, bias, None, 16))


def test_neighbouring_logits(ep):  # noqa: F811
    """Logits one step of fp32 apart, far from and near to zero, in every order."""
    for base in (1.0, -1.0, 3.0e-39, 1.0e30, -250.0):
        steps = torch.arange(200, dtype=torch.int32)[torch.randperm(200, generator=torch.Generator().manual_seed(1))]
        v = (torch.tensor([base]).view(torch.int32) + steps).view(torch.float32).view(1, 200)
        c = Call(ep, v, 32, 0)
        c.check_choices(*c.route())


def test_values_that_are_not_finite(ep):  # noqa: F811
    E, K = 32, 4
    g = torch.Generator().manual_seed(3)
    clean = torch.randn(8, E, generator=g)
    logits = clean.clone()
    logits[0] = -INF                      # no expert at all
    logits[1, 3:] = -INF                  # fewer than K
    logits[2, 5] = NAN
    logits[3, 6] = INF
    logits[4] = NAN
    logits[5, ::2] = torch.finfo(torch.float32).min
    for kind in (0, 1):
        for bias in (None, torch.randn(E, generator=g) * 0.1):
            for normalise in (True, False):
                c = Call(ep, logits, K, kind, normalise, 1.0, bias)
                idx, w = c.route()
                assert (idx[0] == -1).all() and (w[0] == 0).all()
                assert set(idx[1].tolist()) == {0, 1, 2, -1} and w[1, 3] == 0 and (w[1, :3] > 0).all()
                if kind == 1 or bias is None:
                    assert 5 not in idx[2].tolist() and (idx[2] >= 0).all()
                    assert idx[3, 0] == 6 or bias is not None
                if normalise and (kind == 1 or bias is None):
                    assert torch.isfinite(w[2]).all()     # the NaN is not among the chosen
                if not normalise and kind == 0:
                    assert torch.isnan(w[2][idx[2] >= 0]).all()
                assert (idx[4] == -1).all() and (w[4] == 0).all()
                for t in (5, 6, 7):
                    want = ref.choose(kind, logits[t:t + 1], bias, None, K)
                    assert torch.equal(idx[t:t + 1], want)
                    value, bound = ref.weights(kind, normalise, 1.0, logits[t:t + 1], want)
                    assert_within(w[t:t + 1], value, bound)
    # the statistics: a row of -inf does not count, a NaN shows
    c = Call(ep, logits[[0, 1, 5, 6, 7]].contiguous(), K)
    idx, _ = c.route(stats=True)
    c.check_stats(ref.choose(0, c.logits, None, None, K))
    assert c.stats[1][0] == 4
    c = Call(ep, logits, K)
    c.route(stats=True)
    assert torch.isnan(c.stats[3][:2]).all()
    # and a padded NaN does not, nor does it reach its neighbours' gradients
    mask = torch.ones(8, dtype=torch.uint8)
    mask[2:5] = 0
    c = Call(ep, logits, K, mask=mask)
    idx, _ = c.route(stats=True)
    assert torch.isfinite(c.stats[3][:2]).all() and c.stats[1][0] == 4
    got = c.backward(idx, c.stats[0][:-1].cpu(), c.stats[1][:-1].cpu(), torch.ones(8, K), torch.ones(2))
    assert torch.isfinite(got).all() and not got[mask == 0].any() and not got[0].any() and got[6].any()


@pytest.mark.parametrize("kind", [0, 1])
def test_extreme_logits(ep, kind):  # noqa: F811
    """Rows far from zero on either side, and rows whose scores underflow but for one."""
    g = torch.Generator().manual_seed(9)
    logits = torch.randn(12, 64, generator=g)
    logits[0:3] -= 300
    logits[3:6] += 300
    logits[6:9] *= 60
    logits[9, 1:] -= 200
    mask = None
    for normalise in (True, False):
        c = Call(ep, logits, 5, kind, normalise)
        want = c.check_choices(*c.route(stats=True))
        st = c.check_stats(want)
        dw, dl = torch.randn(12, 5, generator=g), torch.tensor([1.0, 1e-3])
        count, tokens = st["expert_count"][0].int(), torch.tensor([12], dtype=torch.int32)
        got = c.backward(want, count, tokens, dw, dl)
        value, bound = ref.gradient(kind, normalise, 1.0, logits, want, mask, count, tokens, dw, dl, 5, False)
        assert_within(got, value, bound)


def test_everything_padded_and_no_tokens(ep):  # noqa: F811
    logits = torch.full((20, 48), NAN)
    c = Call(ep, logits, 4, mask=torch.zeros(20, dtype=torch.uint8))
    idx, w = c.route(stats=True)
    assert (idx == -1).all() and not w.any()
    assert not c.stats[0][:-1].any() and c.stats[1][0] == 0 and not c.stats[2][:-1].any() and not c.stats[3][:2].any()
    got = c.backward(idx, c.stats[0][:-1].cpu(), c.stats[1][:1].cpu(), torch.ones(20, 4), torch.ones(2))
    assert not got.any()
    c = Call(ep, torch.zeros(0, 48), 4)
    c.route(stats=True)
    assert not c.stats[0][:-1].any() and c.stats[1][0] == 0 and not c.stats[2][:-1].any() and not c.stats[3][:2].any()
    c.balance(torch.zeros(0, 4, dtype=torch.int32))
    assert c.backward(None, c.stats[0][:-1], c.stats[1][:1], None, torch.ones(2)).numel() == 0


def test_given_choices(ep):  # noqa: F811
    """Twice the same expert, ids outside the range and empty entries."""
    T, E, K = 50, 20, 6
    logits, mask, g = inputs(T, E, False, 8, 0.2)
    idx = torch.randint(-2, E + 3, (T, K), generator=g, dtype=torch.int32)
    idx[0] = 7
    idx[1] = -1
    idx[2] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 0, 1, 1])
    for kind in (0, 1):
        for normalise in (True, False):
            c = Call(ep, logits, K, kind, normalise, mask=mask)
            c.balance(idx)
            st = c.check_stats(idx)
            dw, dl = torch.randn(T, K, generator=g), torch.tensor([1.0, 1.0])
            count, tokens = st["expert_count"][0].int(), torch.tensor([st["token_count"][0]], dtype=torch.int32)
            got = c.backward(idx, count, tokens, dw, dl)
            value, bound = ref.gradient(kind, normalise, 1.0, logits, idx, mask, count, tokens, dw, dl, K, False)
            # an expert named twice has both terms
            assert_within(got, value, bound * K)


def test_counts_summed_over_ranks(ep):  # noqa: F811
    """Two ranks that add up their counts get the gradient of the loss of the whole batch."""
    T, E, K = 64, 32, 4
    logits, _, _ = inputs(T, E, False, 11)
    idx = ref.choose(0, logits, None, None, K)
    whole = ref.statistics(0, logits, idx, None, K)
    count, tokens = whole["expert_count"][0].int(), torch.tensor([T], dtype=torch.int32)
    dl = torch.tensor([1.0, 0.1])
    value, bound = ref.gradient(0, True, 1.0, logits, idx, None, count, tokens, None, dl, K, False)
    got = torch.cat([Call(ep, h.contiguous(), K).backward(None, count, tokens, None, dl) for h in logits.split(24)])
    assert_within(got, value, bound)


def test_gradient_into_the_logits(ep):  # noqa: F811
    for bf16 in (False, True):
        logits, _, g = inputs(37, 100, bf16, 12)
        c = Call(ep, logits, 4)
        idx = ref.choose(0, logits, None, None, 4)
        dw = torch.randn(37, 4, generator=g)
        want = c.backward(idx, None, None, dw, None)
        x = c.d_logits.clone()
        ep.ep_route_backward(c.p, c.r, x, idx.cuda(), None, None, None, dw.cuda(), None, x)
        assert torch.equal(x.cpu(), want)


def test_other_stream_and_graph(ep):  # noqa: F811
    """The same bits on another stream and from replays of a graph, whose inputs change between them."""
    T, E, K = 300, 96, 4
    batches = [inputs(T, E, False, s)[0].cuda() for s in (1, 2)]
    c = Call(ep, batches[0].cpu(), K)
    dw, dl = torch.randn(T, K, device="cuda"), torch.ones(2, device="cuda")
    dlogits = torch.empty_like(c.d_logits)

    def step():
        ep.ep_route(c.p, c.r, c.d_logits, None, None, c.idx, c.w, *c.stats, c.ws)
        ep.ep_route_backward(c.p, c.r, c.d_logits, c.idx, None, c.stats[0], c.stats[1], dw, dl, dlogits)

    def all_outputs():
        return [t.clone() for t in (c.idx, c.w, *c.stats, dlogits)]

    want = []
    for b in batches:
        c.d_logits.copy_(b)
        step()
        want.append(all_outputs())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(all_outputs(), want[1]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(4):
        c.d_logits.copy_(batches[n % 2])
        for t in (c.idx, c.w, *c.stats):
            t[:-1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(all_outputs(), want[n % 2]))


def test_bound_call(ep):  # noqa: F811
    logits, _, _ = inputs(10, 16, False, 4)
    c = Call(ep, logits, 2)
    want = c.route()
    call = ep.ep_route(c.p, c.r, c.d_logits, None, None, c.idx, c.w, bind=True)
    c.r.score, c.p.num_tokens = 7, 3  # later changes are not seen
    c.idx[:-1].zero_()
    call()
    assert torch.equal(c.idx[:-1].cpu(), want[0]) and torch.equal(c.w[:-1].cpu(), want[1])


def test_many_tokens(ep):  # noqa: F811
    """More tokens than the workgroups take in one round, and the sums of all of them."""
    T, E, K = 70001, 16, 2
    logits, mask, _ = inputs(T, E, True, 6, 0.01)
    c = Call(ep, logits, K, mask=mask)
    idx, w = c.route(stats=True)
    want = c.check_choices(idx, w)
    st = c.check_stats(want)
    got = c.backward(want, st["expert_count"][0].int(), torch.tensor([st["token_count"][0]], dtype=torch.int32), None,
                     torch.tensor([1e4, 1.0]))
    value, bound = ref.gradient(0, True, 1.0, logits, want, mask, st["expert_count"][0], st["token_count"][0], None,
                                torch.tensor([1e4, 1.0]), K, True)
    assert_within(got, value, bound)


@pytest.mark.parametrize("E,K", [(20, 4), (100, 8), (256, 12), (256, 13)])
def test_many_tokens_whose_order_is_close(ep, E, K):  # noqa: F811
    """As the equal logits and the close sums above, with four tokens a wave: rows of equal values, of few values, and of
    sums that only 64 bits tell apart, among ordinary ones."""
    T = 1500
    g = torch.Generator().manual_seed(E + K)
    logits = torch.randn(T, E, generator=g)
    logits[100:300] = 0.25
    logits[300:500] = torch.randint(-1, 2, (200, E), generator=g).float()
    for kind in (0, 1):
        s = ref.scores(kind, logits[1000:1001].double())[0][0]
        for bias in (None, torch.zeros(E), (0.75 - s).float()):
            x = logits.clone()
            x[1000:1200:3] = logits[1000]
            c = Call(ep, x, K, kind, bias=bias)
            c.check_choices(*c.route(stats=True))
        c = Call(ep, logits.bfloat16(), K, kind)
        c.check_choices(*c.route())


def test_gradients_of_weights_that_are_not_there(ep):  # noqa: F811
    """What dweights hold for empty entries and padded tokens does not matter."""
    for T in (30, 1100):
        E, K = 24, 4
        logits, mask, g = inputs(T, E, False, 21, 0.2)
        idx = ref.choose(0, logits, None, mask, K)
        idx[3, 2] = -1
        idx[4] = -1
        dw = torch.randn(T, K, generator=g)
        for kind in (0, 1):
            for normalise in (True, False):
                c = Call(ep, logits, K, kind, normalise, mask=mask)
                want = c.backward(idx, None, None, dw, None)
                worse = dw.clone()
                worse[3, 2] = NAN
                worse[4] = INF
                worse[mask == 0] = NAN
                assert torch.equal(c.backward(idx, None, None, worse, None), want)
                assert not want[4].any() and not want[mask == 0].any()


def test_another_device_is_refused(ep, monkeypatch):  # noqa: F811
    logits, _, _ = inputs(4, 8, False, 1)
    c = Call(ep, logits, 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="device 0 with device 1 current"):
        c.route()
    with pytest.raises(ValueError, match="device 0 with device 1 current"):
        ep.ep_grad_clip(ep.Grads.make([torch.ones(3, device="cuda")]), torch.ones(1, dtype=torch.float64, device="cuda"), 1.0)
