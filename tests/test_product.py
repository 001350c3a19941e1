"""The experts' products (bf16 and FP8) on the GPU against their 64-bit forms."""
import numpy as np
import pytest
import torch

import product_reference as ref

pytestmark = pytest.mark.gpu

SENTINEL = 0x7A51  # bf16 bits that no result has


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    import combine_ep_get_amd as ep
    ep.load()
    return ep


def marked(*shape):
    return torch.full(shape, SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16)


def untouched(t, rows):
    """Whether every row of t outside `rows` still holds the sentinel."""
    keep = torch.ones(t.shape[0], dtype=torch.bool, device=t.device)
    keep[rows] = False
    return bool((t.view(torch.int16)[keep] == SENTINEL).all())


class Routed:
    """A random routing, laid out by the library, checked against the definition."""

    def __init__(self, ep, T, E, K, R=1, A=1, S=None, hidden=8, empty=0.0, hot=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        key = torch.rand(T, E, generator=g) + (torch.arange(E) < 1) * (0.8 if hot else 0.0)
        self.idx = key.topk(K, 1).indices.int() if T else torch.zeros(0, K, dtype=torch.int32)
        self.idx[torch.rand(T, K, generator=g) < empty] = -1
        self.p = ep.Problem.make(T, hidden, E, K, R, 1, A, 1)
        self.p.rank_stride_rows = S or max(1, ep.ep_rank_stride_hint(self.p))
        self.bufs = ep.alloc_layout(self.p)
        ep.ep_get_layout(self.p, self.idx.cuda(), *self.bufs.args())
        self.of, self.slot, _, _ = ref.layout(self.idx, E, R, self.p.rank_stride_rows, A)
        assert torch.equal(self.bufs.token_slot.cpu(), self.slot)
        self.rows = self.p.num_rows
        self.used = sorted(r for v in self.of.values() for r in v)
        self.arrays = (self.bufs.expert_count, self.bufs.expert_offset)


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


CASES = [
    # T, C, N, E, K, R, A, act, bias, residual, pre
    (1, 8, 8, 1, 1, 1, 1, "none", False, False, False),
    (1, 200, 24, 8, 2, 2, 1, "swiglu", True, True, True),
    (5, 72, 136, 4, 2, 1, 4, "geglu", True, False, True),
    (33, 64, 128, 2, 1, 2, 1, "gelu", False, True, True),
    (130, 1000, 264, 3, 2, 1, 16, "silu", True, True, False),
    (257, 136, 72, 5, 3, 5, 1, "relu", True, False, True),
    (300, 520, 200, 16, 4, 4, 8, "swiglu", False, True, True),
    (700, 256, 520, 4, 2, 2, 1, "geglu", True, True, True),
    (1100, 328, 392, 2, 2, 1, 1, "silu", True, True, True),
    (600, 64, 264, 1, 1, 1, 1, "swiglu", False, False, True),
    (90, 328, 1096, 2, 1, 1, 1, "geglu", True, True, True),    # small tiles, gated
    (9, 264, 1000, 3, 1, 1, 1, "gelu", True, True, False),     # few rows, several tiles of outputs
    (150, 1032, 72, 2, 1, 2, 1, "relu", False, False, True),   # an odd number of steps and a part step
    (700, 264, 4360, 8, 1, 2, 1, "silu", True, True, True),      # 128 x 128 tiles
    (300, 136, 2056, 4, 1, 1, 1, "swiglu", True, False, True),   # the same, gated
    (4000, 72, 8200, 16, 2, 4, 1, "none", False, False, False),  # more tiles than workgroups
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:8])))
def test_product(ep, case):
    T, C, N, E, K, R, A, act, bias, residual, pre = case
    r = Routed(ep, T, E, K, R, A, empty=0.1 if T > 4 else 0.0, hot=True, seed=T)
    q = ep.Product.make(C, N, ref.ACTS.index(act))
    M = q.weight_rows
    g = torch.Generator().manual_seed(T + 1)
    x, w = normal(g, r.rows, C), normal(g, E, M, C, scale=C ** -0.5)
    b = torch.randn(E, M, generator=g) if bias else None
    res = normal(g, r.rows, N) if residual else None
    out, pr = marked(r.rows, N), marked(r.rows, M) if pre else None
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    args = (r.p, q, cuda(x), *r.arrays, cuda(w), cuda(b), cuda(res), pr, out)
    ep.ep_expert_product(*args)
    for e, rows in r.of.items():
        o, ob, v, vb = ref.product(act, x[rows], w[e], None if b is None else b[e], None if res is None else res[rows])
        ref.assert_within(out[rows], o, ob, f"out of expert {e}")
        if pre:
            ref.assert_within(pr[rows], v, vb, f"pre of expert {e}")
    assert untouched(out, r.used)
    if pre:
        assert untouched(pr, r.used)
    # the same call again, with the residual in out's place: the same bits
    first = out.clone()
    if residual:
        out.copy_(res)
        ep.ep_expert_product(r.p, q, args[2], *r.arrays, args[5], args[6], out, None, out)
        assert torch.equal(out.view(torch.int16)[r.used], first.view(torch.int16)[r.used])


@pytest.mark.parametrize("T,C,N,act", [(1, 264, 40, "none"), (37, 512, 264, "none"), (100, 72, 200, "gelu"), (513, 200, 136, "swiglu")])
def test_dense(ep, T, C, N, act):
    p = ep.Problem.make(T, 8, 1, 1, 1, 1, 1, T)
    q = ep.Product.make(C, N, ref.ACTS.index(act))
    g = torch.Generator().manual_seed(T)
    x, w, b, res = normal(g, T, C), normal(g, q.weight_rows, C, scale=C ** -0.5), torch.randn(q.weight_rows, generator=g), normal(g, T, N)
    out = marked(T + 3, N)
    ep.ep_expert_product(p, q, x.cuda(), None, None, w.cuda(), b.cuda(), res.cuda(), None, out)
    o, ob, _, _ = ref.product(act, x, w, b, res)
    ref.assert_within(out[:T], o, ob)
    assert untouched(out, list(range(T)))


def test_no_tokens_and_no_valid_entry(ep):
    q = ep.Product.make(64, 64, ep.EP_ACT_SILU)
    for T in (0, 3):
        r = Routed(ep, T, 4, 2, empty=1.1)
        out = marked(max(r.rows, 1), 64)
        x, w = torch.zeros(max(r.rows, 1), 64).bfloat16().cuda(), torch.zeros(4, 64, 64).bfloat16().cuda()
        ep.ep_expert_product(r.p, q, x, *r.arrays, w, None, None, None, out)
        assert untouched(out, [])


def test_slice_overflow_keeps_the_rows_inside(ep):
    """Rows past the slice have no slot: what is inside is computed, the next slice is not touched."""
    r = Routed(ep, 90, 4, 2, R=2, S=50)
    assert ep.ep_read_status(r.bufs.workspace) == ep.EP_ERR_CAPACITY
    q = ep.Product.make(72, 40)
    g = torch.Generator().manual_seed(3)
    x, w = normal(g, r.rows, 72), normal(g, 4, 40, 72)
    out = marked(r.rows, 40)
    ep.ep_expert_product(r.p, q, x.cuda(), *r.arrays, w.cuda(), None, None, None, out)
    for e, rows in r.of.items():
        o, ob, _, _ = ref.product("none", x[rows], w[e])
        ref.assert_within(out[rows], o, ob, f"expert {e}")
    assert untouched(out, r.used)


@pytest.mark.parametrize("T", [20, 400])
def test_values_that_are_not_finite_stay_in_their_row(ep, T):
    """NaN and infinities in one row, in rows of no expert and in the weights
    of an expert without rows reach no other row."""
    C, N, E = 136, 72, 4
    r = Routed(ep, T, E, 1, R=1, S=T + 9)
    r.idx[r.idx == 2] = 1  # expert 2 has no rows
    ep.ep_get_layout(r.p, r.idx.cuda(), *r.bufs.args())
    of, _, _, _ = ref.layout(r.idx, E, 1, T + 9)
    used = sorted(v for rows in of.values() for v in rows)
    q = ep.Product.make(C, N, ep.EP_ACT_NONE)
    g = torch.Generator().manual_seed(5)
    x, w = normal(g, r.rows, C), normal(g, E, N, C)
    clean = marked(r.rows, N)
    ep.ep_expert_product(r.p, q, x.cuda(), *r.arrays, w.cuda(), None, None, None, clean)
    bad = used[len(used) // 2]
    x[bad, 7] = float("nan")
    x[used[0], C - 1] = float("inf")
    x[[i for i in range(r.rows) if i not in used]] = float("nan")
    w[2] = float("inf")
    out = marked(r.rows, N)
    ep.ep_expert_product(r.p, q, x.cuda(), *r.arrays, w.cuda(), None, None, None, out)
    assert torch.isnan(out[bad]).all()
    assert torch.isinf(out[used[0]]).all()
    rest = [i for i in used if i not in (bad, used[0])]
    assert torch.equal(out[rest], clean[rest])
    assert untouched(out, used)


def test_rows_past_32_bits(ep):
    """A slice that starts past 4 GiB of x and out."""
    C, N, S = 16384, 8192, 300_000
    r = Routed(ep, 6, 2, 1, R=2, S=S)
    assert max(r.used) >= S
    q = ep.Product.make(C, N)
    g = torch.Generator().manual_seed(0)
    x = torch.empty(r.rows, C, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor(r.used)
    xs, w = normal(g, len(r.used), C), normal(g, 2, N, C, scale=C ** -0.5)
    x[rows.cuda()] = xs.cuda()
    out = torch.empty(r.rows, N, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_product(r.p, q, x, *r.arrays, w.cuda(), None, None, None, out)
    for e, of in r.of.items():
        o, b, _, _ = ref.product("none", xs[[r.used.index(i) for i in of]], w[e])
        ref.assert_within(out[of], o, b)


FP8_CASES = [
    (1, 128, 128, 4, 2, 1, "swiglu", "token", False, False),
    (30, 256, 384, 8, 2, 2, "none", "padded", True, True),
    (200, 640, 256, 4, 2, 2, "swiglu", "column", True, False),
    (700, 384, 512, 3, 2, 1, "geglu", "token", False, True),
    (513, 256, 128, 1, 1, 1, "silu", "column", True, True),
    (260, 1152, 128, 2, 2, 1, "none", "padded", False, False),
    (90, 1664, 256, 2, 1, 1, "geglu", "column", True, False),
    (400, 640, 2048, 8, 1, 1, "swiglu", "padded", True, True),   # 128 x 128 tiles
    (11, 384, 256, 3, 2, 1, "swiglu", "padded", True, True),
    (40, 256, 128, 300, 2, 2, "silu", "token", False, True),
]


@pytest.mark.parametrize("case", FP8_CASES, ids=lambda c: "-".join(map(str, c[:8])))
def test_product_fp8(ep, case):
    """The rows and scales that ep_dispatch_fp8 leaves, in its three scale layouts."""
    T, C, N, E, K, R, act, lay, bias, residual = case
    r = Routed(ep, T, E, K, R, hidden=C, empty=0.1 if T > 4 else 0.0, seed=T)
    nsf = C // 128
    ts, hs = {"token": (nsf, 1), "padded": ((nsf + 31) // 32 * 32, 1), "column": (1, (r.rows + 15) // 16 * 16)}[lay]
    g = torch.Generator().manual_seed(T)
    xt = normal(g, T, C).cuda()
    xq, xs = torch.empty(T, C, dtype=torch.uint8, device="cuda"), torch.empty(T, nsf, device="cuda")
    ep.ep_quantize_fp8(r.p, xt, xq, xs)
    recv = torch.zeros(r.rows, C, dtype=torch.uint8, device="cuda")
    recv_sf = torch.zeros((r.rows - 1) * ts + (nsf - 1) * hs + 1, device="cuda")
    ep.ep_dispatch_fp8(r.p, xq, xs, None, r.bufs.token_slot, recv, recv_sf, ts, hs)
    q = ep.Product.make(C, N, ref.ACTS.index(act))
    M = q.weight_rows
    w = (torch.randn(E, M, C, generator=g) * 64).to(torch.float8_e4m3fn)
    ws = (torch.rand(E, M // 128, nsf, generator=g) + 0.5) * (C ** -0.5 / 64)
    b = torch.randn(E, M, generator=g) if bias else None
    res = normal(g, r.rows, N) if residual else None
    out = marked(r.rows, N)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    ep.ep_expert_product_fp8(r.p, q, recv, recv_sf, ts, hs, *r.arrays, cuda(w), cuda(ws), cuda(b), cuda(res), out)
    codes = recv.cpu().view(torch.float8_e4m3fn).to(torch.float32)
    sf = recv_sf.cpu()
    for e, rows in r.of.items():
        at = torch.tensor(rows, dtype=torch.long)[:, None] * ts + torch.arange(nsf)[None] * hs
        o, ob, _, _ = ref.product(act, codes[rows], w[e].to(torch.float32), None if b is None else b[e],
                                  None if res is None else res[rows], scales=(sf[at], ws[e]))
        ref.assert_within(out[rows], o, ob, f"expert {e}")
    assert untouched(out, r.used)


@pytest.mark.parametrize("T,E,K", [(24, 8, 2), (900, 4, 2)])
def test_graph_and_streams(ep, T, E, K):
    """A captured call replays to the eager bits between other work, and two streams do not disturb each other."""
    C, N = 264, 136
    r = Routed(ep, T, E, K, seed=9)
    q = ep.Product.make(C, N, ep.EP_ACT_SWIGLU)
    g = torch.Generator().manual_seed(1)
    x, w = normal(g, r.rows, C).cuda(), normal(g, E, 2 * N, C, scale=0.06).cuda()
    want, out = marked(r.rows, N), marked(r.rows, N)
    ep.ep_expert_product(r.p, q, x, *r.arrays, w, None, None, None, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_expert_product(r.p, q, x, *r.arrays, w, None, None, None, out)
    for _ in range(3):
        out.view(torch.int16).fill_(SENTINEL)
        graph.replay()
        other = (x.float() * 2).sum()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.isfinite(other)
    outs, streams = [marked(r.rows, N) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for o, s in zip(outs, streams):
        call = ep.ep_expert_product(r.p, q, x, *r.arrays, w, None, None, None, o, stream=s, bind=True)
        for _ in range(5):
            call()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))
