"""GPU parity of tv_token_sample against the float64 oracle: tokens equal,
probabilities to float32."""

import numpy as np
import pytest
import torch

from gpu_helpers import to_np
from oracle import accept as OA
from oracle import sampling as OS
from speculative_decoding_tree_attn_gb300 import capi

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _logits(R, V, dtype, seed, spread=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(R, V, generator=g, device="cuda") * spread).to(DT[dtype])


def _check(x, u, **kw):
    """probs: the weight is good to 2^-39, its float32, the reciprocal's and the product are a half step each."""
    dev = {k: torch.as_tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda() for k, v in kw.items()}
    ut = torch.as_tensor(u, dtype=torch.float32).cuda()
    probs = torch.full(x.shape, 5.0, device="cuda")
    tokens = capi.tv_token_sample(x, ut, probs=probs, **dev)
    alone = capi.tv_token_sample(x, ut, **dev)
    torch.cuda.synchronize()
    want, p = OS.token_sample(to_np(x), ut.cpu().numpy(), **{k: v.cpu().numpy() for k, v in dev.items()})
    np.testing.assert_array_equal(tokens.cpu().numpy(), want)
    assert torch.equal(tokens, alone)
    got = probs.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(p))
    live = ~np.isnan(p)
    assert ((got == 0) == (p < 2.0 ** -125))[live & ((p == 0) | (p > 2.0 ** -120))].all()
    assert (np.abs(got - p)[live] <= 3.01 * 2.0 ** -24 * p[live] + 2.0 ** -120).all()
    return tokens, probs


@pytest.mark.parametrize("V", [1, 2, 7, 255, 257, 4096, 16384, 16385, 33001, 128000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_limit_alone_and_together(V, dtype):
    rng = np.random.default_rng(V)
    x = _logits(6, V, dtype, V)
    u = rng.uniform(size=6)
    k, p, least, t = rng.integers(1, V + 1, size=6), rng.uniform(0.1, 1.0, size=6), 10 ** rng.uniform(-4, -0.5, size=6), \
        rng.uniform(0.3, 2.0, size=6)
    for kw in (dict(), dict(temperature=t), dict(top_k=k), dict(top_p=p), dict(min_p=least), dict(top_k=k, top_p=p),
               dict(temperature=t, top_k=k, min_p=least, top_p=p)):
        _check(x, u, **kw)


def test_the_longest_rows_and_many_short_ones():
    x = _logits(2, 1 << 20, "f32", 21)
    _check(x, [0.3, 0.999], top_p=[0.9, 0.5])
    _check(x, [0.3, 0.999], top_k=[100000, 40], top_p=[0.7, 1.0])
    x = _logits(3000, 700, "bf16", 22)
    u = np.linspace(0.0, 0.999, 3000)
    _check(x, u, top_k=[9] * 3000, top_p=[0.8] * 3000)
    _check(x, u, min_p=[0.05] * 3000)


def test_limits_that_are_off_and_at_their_ends():
    x = _logits(12, 1000, "f32", 5)
    u = np.linspace(0.0, 0.99, 12)
    inf = float("inf")
    _check(x, u, top_k=[0, -3, 1, 2, 999, 1000, 1001, 2 ** 31 - 1, 5, 5, 5, 5],
           top_p=[1.0, 2.0, 0.0, -1.0, 1e-30, 0.999999, 1.0, inf, 0.5, -inf, 1.0, 0.2],
           min_p=[0.0, -1.0, 0.0, 1.0, 2.0, 1e-30, 0.0, 0.5, inf, 0.1, 0.0, 0.0])
    nan = float("nan")
    a = capi.tv_token_sample(x[:2], torch.tensor([0.3, 0.6]).cuda(), top_p=torch.tensor([nan, nan]).cuda(),
                             min_p=torch.tensor([nan, nan]).cuda())
    assert torch.equal(a, capi.tv_token_sample(x[:2], torch.tensor([0.3, 0.6]).cuda()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("least", [1e-40, 1e-30, 1e-20, 1e-13, 1e-12, 1e-11, 1e-9])
def test_limits_below_a_unit_of_the_sums(least, dtype):
    """min_p below 2^-43 and just above it, on logits down to -100: sorted (top_k 9), by bins, without other limits."""
    rng = np.random.default_rng(3)
    x = torch.from_numpy(np.stack([rng.permutation(np.linspace(0.0, -100.0, 1000)) for _ in range(4)])).to(DT[dtype]).cuda()
    u = rng.uniform(size=4)
    for kw in (dict(), dict(top_k=[9, 99, 300, 999]), dict(top_p=[0.3, 0.9999, 1.0, 1.0 - 2.0 ** -24]),
               dict(top_k=[300, 999, 9, 40], top_p=[1.0 - 2.0 ** -24] * 4), dict(temperature=[0.7, 3.0, 1.5, 1e-3])):
        _check(x, u, min_p=[least] * 4, **kw)
    two = torch.tensor([[0.0, -32.0]], device="cuda", dtype=DT[dtype])
    _, probs = _check(two, [0.5], min_p=[least])
    assert bool(probs[0, 1] > 0) == (np.exp(-32.0) >= least)


@pytest.mark.parametrize("u", [1.0 - 2.0 ** -24, 1.0 - 2.0 ** -23, 1.0])
def test_a_draw_among_weights_of_a_few_units(u):
    """200,000 tokens of 5.3 2^-43 behind one of 1, min_p between 5 and 5.3 of these units, a draw among them: a kept token
    (which one is beyond the sums' resolution)."""
    x = torch.full((3, 200000), -28.14, device="cuda")
    x[:, 0] = 0.0
    tokens, probs = torch.full((3,), -7, dtype=torch.int32, device="cuda"), torch.zeros_like(x)
    col = lambda *v: torch.tensor(v, device="cuda")
    capi.tv_token_sample(x, col(u, u, u), top_p=col(1.0 - 2.0 ** -24, 1.0, 1.0 - 2.0 ** -24),
                         min_p=col(5.2 * 2.0 ** -43, 5.2 * 2.0 ** -43, 0.0), tokens=tokens, probs=probs)
    assert ((tokens >= 0) & (tokens < 200000)).all()
    assert (probs.gather(1, tokens.long()[:, None]) > 0).all()


def test_uniforms_at_the_ends():
    x = _logits(6, 5000, "f32", 6)
    u = [0.0, 1.0 - 2.0 ** -24, 1.0, 1.5, -0.5, 2.0 ** -149]
    _check(x, u, top_p=[0.7] * 6)
    _check(x, u)
    a = capi.tv_token_sample(x[:1], torch.tensor([float("nan")]).cuda())
    assert torch.equal(a, capi.tv_token_sample(x[:1], torch.zeros(1).cuda()))


@pytest.mark.parametrize("V,C", [(3000, 3000), (20000, 20000), (100000, 100000), (100000, 700), (40000, 5)])
def test_equal_logits_go_by_their_index(V, C):
    """C equal largest logits in a row of V (all of them, many, a few), cut by each limit."""
    rng = np.random.default_rng(C)
    x = torch.full((5, V), -2.0, device="cuda")
    for r in range(5):
        x[r, torch.from_numpy(rng.permutation(V)[:C]).cuda()] = 1.0
    u = rng.uniform(size=5)
    _check(x, u, top_k=[1, 2, C // 2 + 1, C, V])
    _check(x, u, top_p=[0.01, 0.25, 0.5, 0.9, 0.99])
    _check(x, u, top_k=[C, C, C, C - 1, 3], top_p=[0.01, 0.25, 0.5, 0.9, 0.99], min_p=[0.5] * 5)


def test_nearly_equal_logits():
    """A row within a few float32 steps: one bin of weights holds all of it."""
    rng = np.random.default_rng(8)
    x = torch.from_numpy((1.0 + rng.integers(0, 50, size=(4, 60000)) * 2.0 ** -23).astype(np.float32)).cuda()
    _check(x, rng.uniform(size=4), top_k=[100, 0, 59999, 30000], top_p=[1.0, 0.5, 0.3, 0.999])


@pytest.mark.parametrize("t", [2.0 ** -61, 1e-12, 1e-3, 50.0, 1e9, 3e38])
def test_hot_and_cold(t):
    x = _logits(3, 9000, "f32", 9)
    _check(x, [0.1, 0.5, 0.9], temperature=[t] * 3, top_p=[1.0, 0.9, 0.3], top_k=[0, 0, 77])


def test_greedy_rows_take_the_first_largest():
    x = _logits(4, 30000, "bf16", 10)
    x[1, 100] = x[1, 20000] = x[1].max()
    x[2] = -0.0
    x[2, 5:] = 0.0
    tokens, probs = _check(x, [0.5] * 4, temperature=[0.0, 0.0, 0.0, 1.0], top_p=[0.5] * 4)
    assert int(tokens[2]) == 0 and (probs[0].count_nonzero() == 1)


def test_excluded_tokens_and_rows_without_a_distribution():
    inf, nan = float("inf"), float("nan")
    x = _logits(9, 20000, "f32", 11)
    x[0, ::2] = -inf
    x[1] = -inf
    x[2, 19999] = inf
    x[3, 7] = nan
    x[4] = -inf
    x[4, 777] = -3e38
    x[5, 1:] = -inf
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = [1.0] * 6 + [-1.0, inf, nan]
    tokens, _ = _check(x, [0.5] * 9, temperature=t, top_k=[50] * 9, top_p=[0.9] * 9)
    assert tokens.tolist()[1:6] == [-1, -1, -1, 777, 0] and tokens.tolist()[6:] == [-1] * 3
    capi.tv_token_sample(x, torch.full((9,), 0.5).cuda(), temperature=torch.tensor(t).cuda(), status=status)
    assert int(status) == capi.TV_DEV_BAD_PARAM


def test_values_at_the_end_of_float32():
    x = torch.tensor([[3.4e38, -3.4e38, 3.39e38, 0.0], [-3.4e38, -3.4e38, -3.4e38, -3.4e38], [1e-45, 0.0, -1e-45, 1e-40]])
    _check(x.cuda(), [0.4, 0.6, 0.99], temperature=[1.0, 1.0, 2.0 ** -59])


def test_draws_follow_the_distribution():
    """100,000 draws of one row against its probabilities: chi-square with 9 degrees, 99.99 % at 33.7."""
    x = torch.log(torch.tensor([5.0, 1.0, 0.0, 3.0, 2.0, 4.0, 0.5, 0.25, 0.0, 1.5, 2.5, 6.0])).cuda().expand(100000, 12)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    tok = capi.tv_token_sample(x.contiguous(), torch.rand(100000, generator=g, device="cuda"))
    n = torch.bincount(tok, minlength=12).cpu().numpy()
    p = torch.softmax(x[0], 0).double().cpu().numpy()
    assert n[p == 0].sum() == 0
    assert ((n - 1e5 * p)[p > 0] ** 2 / (1e5 * p[p > 0])).sum() < 33.7


def test_odd_widths_leave_their_neighbours_alone():
    """Rows that start off a 16-byte boundary, and outputs between guards."""
    x = _logits(7, 1003, "bf16", 13)
    buf = torch.full((9, 1003), 5.0, device="cuda")
    probs = buf.view(-1)[1004:1004 + 7 * 1003].view(7, 1003)
    tokens = torch.full((9,), -7, dtype=torch.int32, device="cuda")
    u = torch.rand(7, device="cuda")
    capi.tv_token_sample(x, u, top_p=torch.full((7,), 0.8).cuda(), tokens=tokens[1:8], probs=probs)
    assert int(tokens[0]) == -7 and int(tokens[8]) == -7
    flat = buf.view(-1)
    assert (flat[:1004] == 5.0).all() and (flat[1004 + 7 * 1003:] == 5.0).all()
    want, _ = OS.token_sample(to_np(x), u.cpu().numpy(), top_p=np.full(7, 0.8, dtype=np.float32))
    np.testing.assert_array_equal(tokens[1:8].cpu().numpy(), want)


def test_leading_shape_stream_and_graph():
    x = _logits(12, 5003, "f32", 14).view(3, 4, 5003)
    u, p = torch.rand(3, 4, device="cuda"), torch.full((3, 4), 0.9, device="cuda")
    want = capi.tv_token_sample(x, u, top_p=p)
    assert want.shape == (3, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = capi.tv_token_sample(x, u, top_p=p, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    tokens = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.tv_token_sample(x, u, top_p=p, tokens=tokens)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(tokens, want)


def test_drafted_rows_feed_acceptance():
    """A drafter's tokens and distributions, and the target's, straight into the chain walk: the oracle's emissions."""
    B, K, V = 6, 4, 3000
    target, draft = _logits(B * (K + 1), V, "f32", 15).view(B, K + 1, V), _logits(B * K, V, "f32", 16).view(B, K, V)
    draft = draft * 0.3 + target[:, :K]
    p, q = torch.empty(B, K + 1, V, device="cuda"), torch.empty(B, K, V, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(17)
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")
    full = lambda *s: torch.full(s, 0.9, device="cuda")
    tokens = capi.tv_token_sample(draft, rand(B, K), temperature=full(B, K), top_p=full(B, K), probs=q)
    capi.tv_token_sample(target, rand(B, K + 1), top_p=full(B, K + 1), probs=p)
    u, u_final = rand(B, K), rand(B)
    out, n = capi.tv_chain_accept_sample(p, q, tokens, u, u_final)
    want, wn = OA.verify_chain(tokens.cpu().numpy(), q.cpu().numpy(), p.cpu().numpy(), np.full(B, K), u.cpu().numpy(),
                               u_final.cpu().numpy())[:2]
    np.testing.assert_array_equal(out.cpu().numpy(), want)
    np.testing.assert_array_equal(n.cpu().numpy(), wn)
    assert (q.gather(2, tokens.long()[..., None]) > 0).all()
