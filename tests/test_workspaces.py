"""Workspace sizes: what the largest call needs serves the smaller ones."""
import random

import pytest
import torch

import combine_ep_get_amd as ep
import route_reference as ref
from test_product_abi import A, BAD, P, Q, tokens, tokens_fp8
from test_route_abi import R, balance, grads, route, tokens_fp4

TOKENS = [0, 1, 2, 4, 5, 31, 32, 33, 64, 65, 500, 1023, 1024, 1025, 2048, 3000, 4095, 4096, 4097, 8192, 16384, 16385, 70000, 1 << 20]


@pytest.mark.parametrize("E", [1, 8, 64, 65, 128, 129, 256, 257, 512, 1000, 2048])
def test_the_routers_workspace_never_falls(E):
    ranks = next(r for r in range(1, E + 1) if E % r == 0 and E // r <= 256)
    need = {}
    for T in TOKENS:
        for K in (1, 2, 8, 11, 12, 13, 16, 32):
            p = P(T=T, E=E, K=K, R=ranks, S=1)
            need[T, K] = ep.ep_route_workspace_bytes(p, R())
            assert need[T, K] > 0
            for fn in (route, balance):
                assert fn(p=p, n=need[T, K] - 1) == BAD
    for (T, K), n in need.items():
        assert all(n >= m for (t, k), m in need.items() if t <= T and k <= K), (T, K)
    assert max(need.values()) <= 256 + 512 * (12 + 8 * E)


@pytest.mark.gpu
@pytest.mark.parametrize("E,K", [(256, 8), (64, 4), (130, 13)])
def test_short_batches_in_the_longest_ones_workspace(E, K):
    """The statistics of every length from one workspace, whatever an earlier call left in it."""
    g = torch.Generator().manual_seed(E)
    long, r = P(T=8192, E=E, K=K, R=1, S=1), R()
    ws = torch.full((ep.ep_route_workspace_bytes(long, r),), 255, dtype=torch.uint8, device="cuda")
    for T in (8192, 4096, 3000, 1025, 1024, 33, 32, 1, 4097):
        logits = torch.randn(T, E, generator=g)
        p = P(T=T, E=E, K=K, R=1, S=1)
        idx, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
        stats = [torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda"),
                 torch.empty(E, device="cuda"), torch.empty(2, device="cuda")]
        ep.ep_route(p, r, logits.cuda(), None, None, idx, w, *stats, ws)
        choice = ref.choose(0, logits, None, None, K)
        assert torch.equal(idx.cpu(), choice)
        want = ref.statistics(0, logits, choice, None, K)
        for t, name in zip(stats, ("expert_count", "token_count", "prob_sum", "losses")):
            value, bound = want[name]
            if name.endswith("count"):
                assert torch.equal(t.cpu().long(), torch.as_tensor(value).view(-1)), (T, name)
            else:
                assert ((t.cpu().double() - value).abs() <= bound).all(), (T, name)


def grads_need(counts):
    array = grads(*[(A, A, n, i % 2, 0) for i, n in counts])
    need = ep.load().ep_grad_workspace_bytes(array, len(counts))
    assert ep.load().ep_grad_square_sum(array, len(counts), A, A, need - 1, None) == BAD
    return need


@pytest.mark.parametrize("seed", range(4))
def test_a_part_of_the_gradients_needs_no_more(seed):
    """Without some of them (experts that no token reached), and with shorter ones."""
    r = random.Random(seed)
    few = [(i, r.randint(1, 9)) for i in range(64)]
    large = [(i, 200_000_000 + i) for i in range(64, 130)]
    mixed = [(i, int(2 ** r.uniform(0, 40)) - 1) for i in range(300)]
    for counts in (few + large, large + few, mixed):
        whole = grads_need(counts)
        for _ in range(20):
            part = [c for c in counts if r.random() < 0.95]
            assert grads_need(part) <= whole
            assert grads_need([(i, n - r.randint(0, n)) for i, n in part]) <= whole
    assert grads_need(few[1:] + large) <= grads_need(few + large)


@pytest.mark.gpu
def test_parts_of_the_gradients_in_the_whole_lists_workspace():
    """What lies behind the workspace stays, and every sum is that of its list."""
    g = torch.Generator().manual_seed(1)
    tensors = [torch.randn(n, generator=g).cuda() for n in [5] * 64 + [300_000] * 70]
    need = ep.ep_grad_workspace_bytes(ep.Grads.make(tensors))
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    square = torch.empty(1, dtype=torch.float64, device="cuda")
    for left_out in (set(), {0}, set(range(0, 64, 2)), set(range(64, 134)), set(range(134))):
        part = [t for i, t in enumerate(tensors) if i not in left_out]
        ep.ep_grad_square_sum(ep.Grads.make(part), square, ws, need)
        want = sum(float((t.double() ** 2).sum()) for t in part)
        assert abs(float(square) - want) <= 2.0 ** -40 * want
    assert (ws[need:] == 255).all()


def hidden_rows(p, q):
    """The status and the hidden rows: all that the bf16 and FP8 layers use."""
    return 256 + p.num_tokens * p.num_topk * q.out_features * 2


@pytest.mark.parametrize("sizes", [dict(T=128, E=256, K=8, H=7168), dict(T=5, E=8, K=3, H=256)], ids=("many", "few"))
def test_the_few_token_layers_workspace_by_its_weights(sizes):
    p, q = P(S=1, **sizes), Q(C=sizes["H"], N=2048)
    need = [ep.ep_moe_tokens_weights_workspace_bytes(p, q, w) for w in (ep.EP_WEIGHTS_BF16, ep.EP_WEIGHTS_FP8, ep.EP_WEIGHTS_FP4)]
    assert need[0] == need[1] == hidden_rows(p, q)
    assert need[2] == ep.ep_moe_tokens_workspace_bytes(p, q) >= need[0]
    for fn, n in zip((tokens, tokens_fp8, tokens_fp4), need):
        assert fn(p=p, q=q, n=n - 1) == BAD
    for w in (-1, 3):
        assert ep.ep_moe_tokens_weights_workspace_bytes(p, q, w) == 0


def test_sizes_that_only_some_weights_take():
    """Rows of the 4-bit layer are not counted where it refuses the sizes."""
    many = dict(T=128, E=256, K=8, S=1)
    for p, q, takes in ((P(H=7168, **many), Q(C=7168, N=2056), (1, 0, 0)), (P(H=264, **many), Q(C=264, N=2048), (1, 0, 0)),
                        (P(H=224, **many), Q(C=224, N=2048), (1, 0, 1)), (P(H=260, **many), Q(C=260, N=2048), (0, 0, 0))):
        need = [ep.ep_moe_tokens_weights_workspace_bytes(p, q, w) for w in range(3)]
        assert [int(n > 0) for n in need] == list(takes)
        assert ep.ep_moe_tokens_workspace_bytes(p, q) == max(need)
        assert need[0] in (0, hidden_rows(p, q))


@pytest.mark.gpu
def test_the_bf16_layer_in_its_own_workspace():
    """Nothing behind the bytes that its size call names is written."""
    g = torch.Generator().manual_seed(3)
    T, H, I, E, K = 64, 256, 128, 64, 4
    p, q = P(T=T, H=H, E=E, K=K, R=1, S=1), ep.Product.make(H, I, ep.EP_ACT_RELU)
    x, w1, w2 = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((T, H), (E, I, H), (E, H, I)))
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32).cuda()
    small, large = ep.ep_moe_tokens_weights_workspace_bytes(p, q, ep.EP_WEIGHTS_BF16), ep.ep_moe_tokens_workspace_bytes(p, q)
    assert small == hidden_rows(p, q) < large
    outs = []
    for n in (small, large):
        ws = torch.full((large,), 255, dtype=torch.uint8, device="cuda")
        outs.append(torch.empty_like(x))
        ep.ep_moe_tokens(p, q, x, idx, None, w1, None, w2, None, None, outs[-1], ws, n)
        assert ep.ep_read_status(ws) == ep.EP_OK and (ws[small:] == 255).all()
    assert torch.equal(*outs)
