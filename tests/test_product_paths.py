"""The experts' products on the kernels that long and large calls take.

The tile follows from the sizes: 64 x 64 below 128 tiles of 128 x 128; bf16
256 x 256 from 160 rows an expert (gradients 64) and 192 such tiles; else 128 x
128.  The kernel for few rows takes experts of up to 16 rows on average and 64 tiles of
128 weight rows in all.  Experts' rows are uneven, so that a tile computes from one to
all of its fragments."""
import pytest
import torch

import product_reference as ref
from test_product import SENTINEL, Routed, ep, marked, normal, untouched  # noqa: F401

pytestmark = pytest.mark.gpu


class Counted(Routed):
    """Routed, with a given number of tokens for every expert, in shuffled order."""

    def __init__(self, ep, counts, R=1, A=1, S=None, hidden=8, seed=0):  # noqa: F811
        T, E = sum(counts) + 3, len(counts)
        super().__init__(ep, T, E, 1, R, A, S=S or T + E * A, hidden=hidden, seed=seed)
        ids = torch.cat([torch.repeat_interleave(torch.arange(E), torch.tensor(counts)), torch.full((3,), -1)])
        self.idx = ids[torch.randperm(T, generator=torch.Generator().manual_seed(seed))].int()[:, None].contiguous()
        ep.ep_get_layout(self.p, self.idx.cuda(), *self.bufs.args())
        self.of, self.slot, _, _ = ref.layout(self.idx, E, R, self.p.rank_stride_rows, A)
        self.used = sorted(r for v in self.of.values() for r in v)


def cuda(t):
    return None if t is None else t.cuda()


UNEVEN = (40, 100, 180, 256, 257, 300, 520, 0)  # 207 on average
FEW = (1, 2, 0, 16, 17, 33, 4, 5, 6, 7, 8, 9, 1, 1, 1, 1)  # 7 on average, 18 row tiles of 16

FORWARD = [
    # counts, R, A, C, N, act, bias, residual, pre
    # 256 x 256: full and part steps of k, even and odd numbers of them
    (UNEVEN, 2, 1, 328, 1704, "swiglu", True, True, True),
    (UNEVEN, 1, 16, 320, 1704, "geglu", True, False, True),
    (UNEVEN, 4, 1, 392, 3400, "silu", False, True, True),
    (UNEVEN, 1, 1, 256, 3400, "none", True, True, False),
    (UNEVEN, 1, 1, 200, 3400, "gelu", True, False, True),
    (UNEVEN, 8, 1, 512, 3400, "relu", False, True, False),
    # 128 x 128
    (UNEVEN, 2, 1, 392, 1032, "swiglu", True, True, True),
    (UNEVEN, 1, 1, 328, 1096, "gelu", True, True, True),
    # few rows
    (FEW, 2, 1, 264, 248, "swiglu", True, True, True),
    (FEW, 1, 4, 200, 256, "geglu", False, False, True),
    (FEW, 4, 1, 1032, 504, "silu", True, True, False),
    (FEW, 1, 1, 128, 504, "none", False, True, True),
    # as few, but more tiles than that
    (FEW, 2, 1, 264, 1096, "swiglu", True, True, True),
    (FEW, 4, 1, 1032, 1096, "silu", True, True, False),
]


@pytest.mark.parametrize("case", FORWARD, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-" + "-".join(map(str, c[1:6])))
def test_forward(ep, case):  # noqa: F811
    counts, R, A, C, N, act, bias, residual, pre = case
    r = Counted(ep, counts, R, A, seed=C)
    q, E = ep.Product.make(C, N, ref.ACTS.index(act)), len(counts)
    M = q.weight_rows
    g = torch.Generator().manual_seed(C + 1)
    x, w = normal(g, r.rows, C), normal(g, E, M, C, scale=C ** -0.5)
    b = torch.randn(E, M, generator=g) if bias else None
    res = normal(g, r.rows, N) if residual else None
    x[[i for i in range(r.rows) if i not in set(r.used)]] = float("nan")  # rows of no expert reach none
    out, pr = marked(r.rows, N), marked(r.rows, M) if pre else None
    d = [cuda(t) for t in (x, w, b, res)]
    ep.ep_expert_product(r.p, q, d[0], *r.arrays, *d[1:], pr, out)
    for e, rows in r.of.items():
        o, ob, v, vb = ref.product(act, x[rows], w[e], None if b is None else b[e], None if res is None else res[rows])
        ref.assert_within(out[rows], o, ob, f"out of expert {e}")
        if pre:
            ref.assert_within(pr[rows], v, vb, f"pre of expert {e}")
    assert untouched(out, r.used) and (not pre or untouched(pr, r.used))
    again = marked(r.rows, N)
    ep.ep_expert_product(r.p, q, d[0], *r.arrays, *d[1:], None, again)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


FP8 = [
    # counts, R, C, N, act, bias, residual
    (UNEVEN, 2, 1152, 1024, "swiglu", True, True),     # 128 x 128, nine blocks of scales
    (UNEVEN, 1, 1280, 2048, "silu", False, True),      # ten
    ((58, 1, 1, 1), 1, 384, 2048, "none", True, True),  # few rows
    ((103, 1, 1, 1, 1, 1, 1), 1, 256, 512, "geglu", True, False),
    ((103, 1, 1, 1, 1, 1, 1), 1, 1152, 2048, "swiglu", True, True),  # as few, but more tiles
]


@pytest.mark.parametrize("case", FP8, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-" + "-".join(map(str, c[1:5])))
@pytest.mark.parametrize("column", [False, True])
def test_forward_fp8(ep, case, column):  # noqa: F811
    counts, R, C, N, act, bias, residual = case
    r = Counted(ep, counts, R, seed=C)
    q, E, nsf = ep.Product.make(C, N, ref.ACTS.index(act)), len(counts), C // 128
    M = q.weight_rows
    g = torch.Generator().manual_seed(C)
    x = (torch.randn(r.rows, C, generator=g) * 64).to(torch.float8_e4m3fn)
    xs = torch.rand(r.rows, nsf, generator=g) / 64 + 1 / 128
    w = (torch.randn(E, M, C, generator=g) * 64).to(torch.float8_e4m3fn)
    ws = (torch.rand(E, M // 128, nsf, generator=g) + 0.5) * (C ** -0.5 / 64)
    b = torch.randn(E, M, generator=g) if bias else None
    res = normal(g, r.rows, N) if residual else None
    out = marked(r.rows, N)
    sf, ts, hs = (xs.t().contiguous(), 1, r.rows) if column else (xs, nsf, 1)
    ep.ep_expert_product_fp8(r.p, q, cuda(x), cuda(sf), ts, hs, *r.arrays, cuda(w), cuda(ws), cuda(b), cuda(res), out)
    for e, rows in r.of.items():
        o, ob, _, _ = ref.product(act, x[rows].float(), w[e].float(), None if b is None else b[e],
                                  None if res is None else res[rows], scales=(xs[rows], ws[e]))
        ref.assert_within(out[rows], o, ob, f"expert {e}")
    assert untouched(out, r.used)


BACKWARD = [
    # counts, R, C, N, act
    (UNEVEN, 2, 3400, 168, "swiglu"),  # 256 x 256, six steps of the weight's rows, up to nine of an expert's
    (UNEVEN, 1, 3400, 328, "silu"),
    (UNEVEN, 1, 1032, 264, "gelu"),    # 128 x 128
    (UNEVEN, 8, 136, 72, "geglu"),     # 64 x 64
]


@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-" + "-".join(map(str, c[1:])))
def test_backward(ep, case):  # noqa: F811
    counts, R, C, N, act = case
    r = Counted(ep, counts, R, seed=C)
    q, E = ep.Product.make(C, N, ref.ACTS.index(act)), len(counts)
    M = q.weight_rows
    g = torch.Generator().manual_seed(C)
    x, w = normal(g, r.rows, C), normal(g, E, M, C, scale=C ** -0.5)
    dout, pre = normal(g, r.rows, N), normal(g, r.rows, M)
    rest = [i for i in range(r.rows) if i not in set(r.used)]
    for t in (x, dout, pre):
        t[rest] = float("nan")
    before = torch.randn(E, M, C, generator=g)
    dpre, dx, dw, acc = marked(r.rows, M), marked(r.rows, C), marked(E, M, C), before.cuda()
    db = torch.full((E, M), 7.0, device="cuda")
    ws = torch.empty(ep.ep_product_workspace_bytes(r.p, q), dtype=torch.uint8, device="cuda")
    ep.ep_expert_product_backward(r.p, q, cuda(dout), cuda(pre), cuda(x), *r.arrays, cuda(w), dpre, dx, dw, acc, db, ws)
    for e, rows in r.of.items():
        want = ref.backward(act, dout[rows], pre[rows], x[rows], w[e])
        ref.assert_within(dpre[rows], *want["dpre"], f"dpre of expert {e}")
        ref.assert_within(dx[rows], *want["dx"], f"dx of expert {e}")
        ref.assert_within(dw[e], *want["dweight"], f"dweight of expert {e}")
        v, b = want["dweight_acc"]
        v = v + before[e].double()
        ref.assert_within(acc[e], v, b + ref.ULP32 * v.abs(), f"dweight_acc of expert {e}")
        ref.assert_within(db[e], *want["dbias"], f"dbias of expert {e}")
    assert untouched(dx, r.used) and untouched(dpre, r.used)


def test_buffers_past_32_bits(ep):  # noqa: F811
    """Forward and backward of a second slice that starts past 4 GiB of every
    row buffer, with more rows an expert than the kernel for few takes."""
    C = N = 1032
    r = Routed(ep, 400, 2, 1, R=2, S=2_200_000)
    assert all(len(v) > 16 for v in r.of.values()) and r.p.rank_stride_rows * C * 2 > 1 << 32
    q = ep.Product.make(C, N, ep.EP_ACT_SILU)
    g = torch.Generator().manual_seed(0)
    at = torch.tensor(r.used).cuda()
    local = {e: [r.used.index(i) for i in rows] for e, rows in r.of.items()}
    xs, ds, w = normal(g, len(r.used), C), normal(g, len(r.used), N), normal(g, 2, N, C, scale=C ** -0.5)
    x, dout, pre, out, dx = (marked(r.rows, C) for _ in range(5))
    x[at], dout[at] = xs.cuda(), ds.cuda()
    ep.ep_expert_product(r.p, q, x, *r.arrays, w.cuda(), None, None, pre, out)
    ps = pre[at].cpu()
    dw = marked(2, N, C)
    ep.ep_expert_product_backward(r.p, q, dout, pre, x, *r.arrays, w.cuda(), pre, dx, dw)
    for e, rows in local.items():
        o, ob, v, vb = ref.product("silu", xs[rows], w[e])
        ref.assert_within(out[at][rows], o, ob, f"out of expert {e}")
        ref.assert_within(ps[rows], v, vb, f"pre of expert {e}")
        want = ref.backward("silu", ds[rows], ps[rows], xs[rows], w[e])
        ref.assert_within(pre[at][rows], *want["dpre"], f"dpre of expert {e}")
        ref.assert_within(dx[at][rows], *want["dx"], f"dx of expert {e}")
        ref.assert_within(dw[e], *want["dweight"], f"dweight of expert {e}")
    for t in (out, pre, dx):
        assert int((t.view(torch.int16) != SENTINEL).any(1).sum()) == len(r.used)


@pytest.mark.parametrize("column", [False, True])
def test_fp8_buffers_past_32_bits(ep, column):  # noqa: F811
    C, N, nsf = 1024, 128, 8
    r = Routed(ep, 90, 2, 1, R=2, S=4_400_000)
    assert r.p.rank_stride_rows * C > 1 << 32
    q = ep.Product.make(C, N)
    g = torch.Generator().manual_seed(0)
    at = torch.tensor(r.used).cuda()
    xs = (torch.randn(len(r.used), C, generator=g) * 64).to(torch.float8_e4m3fn)
    fs = torch.rand(len(r.used), nsf, generator=g) / 64
    w = (torch.randn(2, N, C, generator=g) * 64).to(torch.float8_e4m3fn)
    ws = torch.rand(2, N // 128, nsf, generator=g) / 512
    x, sf, out = torch.zeros(r.rows, C, dtype=torch.uint8, device="cuda"), torch.zeros(r.rows, nsf, device="cuda"), marked(r.rows, N)
    x[at], sf[at] = xs.view(torch.uint8).cuda(), fs.cuda()
    ts, hs = (1, r.rows) if column else (nsf, 1)
    sf = sf.t().contiguous() if column else sf
    ep.ep_expert_product_fp8(r.p, q, x, sf, ts, hs, *r.arrays, w.cuda(), ws.cuda(), None, None, out)
    for e, of in r.of.items():
        rows = [r.used.index(i) for i in of]
        o, b, _, _ = ref.product("none", xs[rows].float(), w[e].float(), scales=(fs[rows], ws[e]))
        ref.assert_within(out[at][rows], o, b, f"expert {e}")
    assert int((out.view(torch.int16) != SENTINEL).any(1).sum()) == len(r.used)


def test_captured_training_step(ep):  # noqa: F811
    """Forward with pre, combine's gradient and backward in one graph: every
    replay, between other work and with new values in the inputs, gives the eager bits."""
    T, H, N, E, K = 300, 136, 72, 4, 2
    r = Routed(ep, T, E, K, R=2, hidden=H, seed=2)
    up, down = ep.Product.make(H, N, ep.EP_ACT_SWIGLU), ep.Product.make(N, H)
    g = torch.Generator().manual_seed(3)
    xs = [normal(g, r.rows, H).cuda() for _ in range(2)]
    w1, w2, b1 = normal(g, E, 2 * N, H, scale=0.1).cuda(), normal(g, E, H, N, scale=0.1).cuda(), torch.randn(E, 2 * N, generator=g).cuda()
    dout, tw = normal(g, T, H).cuda(), torch.rand(T, K, generator=g).cuda()
    x, wsp = xs[0].clone(), torch.empty(ep.ep_product_workspace_bytes(r.p, up), dtype=torch.uint8, device="cuda")

    def buffers():
        return dict(pre=marked(r.rows, 2 * N), h=marked(r.rows, N), y=marked(r.rows, H), dy=marked(r.rows, H),
                    dtw=torch.zeros(T, K, device="cuda"), dh=marked(r.rows, N), dw2=marked(E, H, N), dpre=marked(r.rows, 2 * N),
                    dx=marked(r.rows, H), dw1=marked(E, 2 * N, H), db1=torch.zeros(E, 2 * N, device="cuda"))

    def step(b):
        ep.ep_expert_product(r.p, up, x, *r.arrays, w1, b1, None, b["pre"], b["h"])
        ep.ep_expert_product(r.p, down, b["h"], *r.arrays, w2, None, None, None, b["y"])
        ep.ep_combine_backward(r.p, dout, b["y"], r.bufs.token_slot, tw, b["dy"], b["dtw"])
        ep.ep_expert_product_backward(r.p, down, b["dy"], None, b["h"], *r.arrays, w2, None, b["dh"], b["dw2"])
        ep.ep_expert_product_backward(r.p, up, b["dh"], b["pre"], x, *r.arrays, w1, b["dpre"], b["dx"], b["dw1"], None,
                                      b["db1"], wsp)

    bits = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32)  # noqa: E731
    want = []
    for v in xs:
        x.copy_(v)
        want.append(buffers())
        step(want[-1])
    got = buffers()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got)
    for n in range(4):
        x.copy_(xs[n % 2])
        for t in got.values():
            bits(t).fill_(SENTINEL)
        graph.replay()
        other = (dout.float() * 2).sum()
        torch.cuda.synchronize()
        assert torch.isfinite(other)
        for k, t in got.items():
            assert torch.equal(bits(t)[r.used] if t.shape[0] == r.rows else bits(t),
                               bits(want[n % 2][k])[r.used] if t.shape[0] == r.rows else bits(want[n % 2][k])), (n, k)


@pytest.mark.parametrize("T", [24, 700])
def test_captured_fp8_product(ep, T):  # noqa: F811
    C, N, E = 384, 256, 4
    r = Routed(ep, T, E, 2, hidden=C, seed=T)
    q, nsf = ep.Product.make(C, N, ep.EP_ACT_SWIGLU), C // 128
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(r.rows, C, generator=g) * 64).to(torch.float8_e4m3fn).cuda()
    w = (torch.randn(E, 2 * N, C, generator=g) * 64).to(torch.float8_e4m3fn).cuda()
    xs, ws = torch.rand(r.rows, nsf, generator=g).cuda() / 64, torch.rand(E, 2 * N // 128, nsf, generator=g).cuda() / 512
    want, out = marked(r.rows, N), marked(r.rows, N)
    ep.ep_expert_product_fp8(r.p, q, x, xs, nsf, 1, *r.arrays, w, ws, None, None, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_expert_product_fp8(r.p, q, x, xs, nsf, 1, *r.arrays, w, ws, None, None, out)
    for _ in range(3):
        out.view(torch.int16).fill_(SENTINEL)
        graph.replay()
        other = xs.sum()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.isfinite(other)
