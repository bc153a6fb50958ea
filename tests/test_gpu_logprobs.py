"""GPU parity of tv_token_logprobs against the float64 oracle: values within
their float32 error, alternatives equal index by index."""

import numpy as np
import pytest
import torch

from gpu_helpers import to_np
from oracle import attention as OA
from oracle import kvcache as OK
from oracle import logprobs as OL
from oracle import tree as OT
from speculative_decoding_tree_attn_gb300 import capi
from speculative_decoding_tree_attn_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _check(logits, tokens, node=None, top_k=0, want_status=0):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = capi.tv_token_logprobs(logits, tokens, node=node, top_k=top_k, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == want_status
    x = to_np(logits)
    ref = OL.token_logprobs(x, tokens.cpu().numpy(), None if node is None else node.cpu().numpy(), top_k)
    lp, ent, ids, top = (to_np(g).astype(np.float64) if g.dtype != torch.int32 else to_np(g) for g in got)
    np.testing.assert_array_equal(ids, ref[2])
    # S and sum e (x - m) are float32 sums of V / 256 terms one after another at most, joined in 16 steps; an
    # exponential is off by 2^-21 and by its argument's rounding, 2 * 2^-24 of |x - m|, which is under 104 where e > 0
    V = x.shape[-1]
    spread = 104.0
    rel = (V / 256 + 16) * 2.0 ** -24 + 2.0 ** -21 + 2 * 2.0 ** -24 * spread
    rows = np.arange(tokens.shape[1])[None].repeat(x.shape[0], 0) if node is None else to_np(node).clip(0, x.shape[1] - 1)
    best = np.abs(np.take_along_axis(np.nan_to_num(x.astype(np.float64)).max(-1), rows, 1))  # |m| [B, C]
    with np.errstate(invalid="ignore"):
        for g, r, m in ((lp, ref[0], best), (top, ref[3], np.broadcast_to(best[..., None], ref[3].shape))):
            fin = np.isfinite(r)
            assert np.array_equal(np.isnan(g), np.isnan(r)) and np.array_equal(g[~fin & ~np.isnan(r)], r[~fin & ~np.isnan(r)])
            # ln S moves by rel; the subtractions round at |x| <= |result| + |m| + ln V, at |m| and at ln V
            assert (np.abs(g - r)[fin] <= rel + 4 * 2.0 ** -24 * (2 * (m[fin] + np.log(V)) + np.abs(r[fin]))).all()
        fin = np.isfinite(ref[1])
        assert np.array_equal(np.isnan(ent), ~fin)
        # H = ln S + T, T = (1/S) sum e (m - x) <= H: each off by rel of itself
        assert (np.abs(ent - ref[1])[fin] <= rel + (2 * rel + 4 * 2.0 ** -24) * (np.log(V) + ref[1][fin])).all()
    return got


def _rows(B, N, V, dtype, seed, std=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(B, N, V, generator=g, device="cuda") * std).to(DT[dtype])
    t = torch.randint(0, V, (B, N), generator=g, device="cuda", dtype=torch.int32)
    return x, t


@pytest.mark.parametrize("V", [1, 2, 7, 31, 32, 33, 255, 257, 1000, 4099, 32000, 128000, 151936, 262147])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_vocabulary(V, dtype):
    """Odd vocabularies leave rows off 16-byte boundaries."""
    x, t = _rows(2, 3, V, dtype, V)
    _check(x, t, top_k=min(V, 20))


@pytest.mark.parametrize("K", [0, 1, 2, 5, 31, 32])
def test_every_k(K):
    x, t = _rows(3, 5, 5000, "bf16", 7 + K)
    _check(x, t, top_k=K)


@pytest.mark.parametrize("rows", [1, 2, 8, 20, 40, 76, 152, 153, 305, 700])
@pytest.mark.parametrize("dtype,V", [("f32", 9001), ("bf16", 33000)])
def test_every_number_of_rows(rows, dtype, V):
    x, t = _rows(1, rows, V, dtype, rows)
    _check(x, t, top_k=8)


def test_paths_padding_and_repeated_rows():
    x, _ = _rows(4, 10, 3001, "f32", 3)
    node = torch.tensor([[0, 3, 9, -1], [0, -1, -1, -1], [5, 5, 5, 5], [-1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    tok = torch.tensor([[4, 3000, 0, -1], [17, -1, -1, -1], [1, 2, 2, 3], [-1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    _check(x, tok, node, 4)
    _check(x, tok, node, 0)


def test_bad_tokens_and_nodes_are_flagged_and_skipped():
    x, _ = _rows(1, 3, 100, "f32", 4)
    tok = torch.tensor([[5, 100, -2, 7]], dtype=torch.int32, device="cuda")
    ok = torch.tensor([[0, 1, 2, 2]], dtype=torch.int32, device="cuda")
    _check(x, tok, ok, 3, want_status=capi.TV_DEV_BAD_TOKEN)
    node = torch.tensor([[0, 3, -5, 2]], dtype=torch.int32, device="cuda")
    _check(x, torch.full_like(tok, 9), node, 3, want_status=capi.TV_DEV_BAD_TOPOLOGY)


def _special():
    inf = float("inf")
    V = 40000
    ramp = torch.arange(V).float() / 64
    one = torch.full((V,), -inf)
    one[31234] = 2.5
    few = torch.full((V,), -inf)
    few[[5, 17777, 39999]] = torch.tensor([1.0, 3.0, 1.0])
    low = torch.full((V,), torch.finfo(torch.bfloat16).min)
    low[123] = 4.0
    nan, pinf = torch.randn(V), torch.randn(V)
    nan[777], pinf[888] = float("nan"), inf
    zero = torch.zeros(V)
    zero[::2] = -0.0
    return {"rising": ramp, "falling": ramp.flip(0), "all alike": torch.full((V,), -3.25), "one left": one,
            "few left": few, "lowest value masks": low, "none left": torch.full((V,), -inf), "a nan": nan,
            "an inf": pinf, "zeros of both signs": zero, "two levels": (torch.arange(V) % 2).float(),
            "peaked": torch.cat((torch.full((V - 1,), -60.0), torch.tensor([40.0]))),
            "large": torch.randn(V) * 1e4, "huge": torch.randn(V) * 1e37,
            "sawtooth": (torch.arange(V) % 997).float(), "late peak": torch.cat((torch.zeros(V - 40), torch.arange(40.0)))}


@pytest.mark.parametrize("name", sorted(_special()))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("copies", [1, 400])
def test_special_rows(name, dtype, copies):
    """Ties, orders, excluded tokens and rows without a distribution; alone (a row over several SMs) and in numbers."""
    x = _special()[name].to(DT[dtype]).cuda().view(1, 1, -1)
    tok = torch.tensor([[31234]], dtype=torch.int32, device="cuda")
    first = _check(x, tok, top_k=32)
    if copies > 1:
        many = capi.tv_token_logprobs(x.expand(1, 1, -1).contiguous(), tok.expand(1, copies).contiguous(),
                                      node=torch.zeros(1, copies, dtype=torch.int32, device="cuda"), top_k=32)
        ref = OL.token_logprobs(to_np(x), tok.cpu().numpy(), None, 32)
        for m, f in zip(many, first):
            assert torch.equal(torch.nan_to_num(m[:, :1].float()), torch.nan_to_num(m[:, -1:].float()))
        np.testing.assert_array_equal(to_np(many[2][0, 0]), ref[2][0, 0])
        np.testing.assert_allclose(to_np(many[0][0, 0]), ref[0][0, 0], rtol=2e-5, atol=2e-5)


@pytest.mark.parametrize("name", sorted(_special()))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_special_rows_over_a_cluster(name, dtype):
    """Three times each row behind one another: ties and peaks in several of its CTAs."""
    x = _special()[name].to(DT[dtype]).cuda().repeat(3).view(1, 1, -1)
    tok = torch.tensor([[71234]], dtype=torch.int32, device="cuda")
    _check(x, tok, top_k=32)


@pytest.mark.parametrize("rows", [1, 5, 19, 20, 38, 39, 76, 77, 152, 153])
@pytest.mark.parametrize("dtype,V", [("f32", 70003), ("bf16", 50001), ("bf16", 140007)])
def test_every_split_of_a_row(rows, dtype, V):
    x, t = _rows(1, rows, V, dtype, rows)
    _check(x, t, top_k=8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_at_the_ends_of_the_type(dtype):
    """A row masked to the lowest value throughout is uniform; one logit near the largest value takes everything."""
    V, lo = 30011, torch.finfo(DT[dtype]).min
    x = torch.full((1, 4, V), lo, dtype=DT[dtype], device="cuda")
    x[0, 1, 77] = -lo
    x[0, 2, :] = -lo
    x[0, 3, 5] = lo / 2
    t = torch.tensor([[9, 77, 8, 9]], dtype=torch.int32, device="cuda")
    lp, ent, ids, top = (g[0].tolist() for g in capi.tv_token_logprobs(x, t, top_k=2))
    # one float32 sum of V equal terms, rel of the bound above: under 2e-5
    for r in (0, 2):
        assert abs(lp[r] + np.log(V)) <= 2e-5 and abs(ent[r] - np.log(V)) <= 2e-4 and ids[r] == [0, 1]
    assert lp[1] == 0 and ent[1] == 0 and ids[1] == [77, 0] and top[1][0] == 0 and top[1][1] < -1e38
    assert lp[3] < -1e38 and ent[3] == 0 and ids[3] == [5, 0] and top[3][0] == 0


@pytest.mark.parametrize("at", [2.0 ** 20, -2.0 ** 20])
@pytest.mark.parametrize("V", [40, 5000, 100000])
def test_logits_about_a_million(at, V):
    """Rows whose threads' maxima lie on both sides of 2^20, where the sums' reference changes."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = at + torch.randn(1, 3, V, generator=g, device="cuda") * 3
    x[0, 1, ::2], x[0, 1, 1::2] = at + 1, at - 1
    x[0, 2] = at + torch.linspace(-9, 9, V, device="cuda")
    t = x.argmax(-1).to(torch.int32)
    lp, ent, ids, top = (to_np(y) for y in capi.tv_token_logprobs(x, t, top_k=5))
    ref = OL.token_logprobs(to_np(x), t.cpu().numpy(), None, 5)
    np.testing.assert_array_equal(ids, ref[2])
    # logits are within 2^5 of each other, so their differences are exact: what is left are rel, as in _check with a
    # spread of 2^5, and the roundings of results under 2^6
    rel = (V / 256 + 16) * 2.0 ** -24 + 2.0 ** -21 + 2 * 2.0 ** -24 * 32
    bound = rel + 4 * 2.0 ** -24 * 64
    assert np.abs(lp - ref[0]).max() <= bound and np.abs(top - ref[3]).max() <= bound
    assert np.abs(ent - ref[1]).max() <= rel + (2 * rel + 4 * 2.0 ** -24) * 32


def test_what_greedy_acceptance_returns():
    """out and path of the greedy walk go straight in; each emitted token is its row's first alternative."""
    w = W.WORKLOADS["gqa_b8_l512_2048_n26"]
    parent, *_ = OT.build_tree(w.paths())
    g = W.greedy_inputs(w, parent, device="cuda")
    out, n_out, path = capi.tv_tree_accept_greedy(g["tokens"], torch.from_numpy(parent.astype(np.int32)).cuda(),
                                                  logits=g["logits"], out_cols=7)
    lp, ent, ids, top = _check(g["logits"], out, path, 3)
    assert torch.equal(ids[..., 0], out) and torch.equal(torch.where(out >= 0, top[..., 0], 0.0), lp)


def test_outputs_given_and_captured():
    x, t = _rows(2, 4, 20000, "f32", 11)
    outs = dict(logprob=torch.empty(2, 4, device="cuda"), entropy=torch.empty(2, 4, device="cuda"),
                top_ids=torch.empty(2, 4, 6, dtype=torch.int32, device="cuda"),
                top_logprobs=torch.empty(2, 4, 6, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        capi.tv_token_logprobs(x, t, top_k=6, **outs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.tv_token_logprobs(x, t, top_k=6, **outs)
    for seed in (12, 13):
        x2, t2 = _rows(2, 4, 20000, "f32", seed)
        x.copy_(x2)
        t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs.values(), capi.tv_token_logprobs(x2, t2, top_k=6)):
            assert torch.equal(got, want)


def test_a_call_on_another_stream_allocates_there():
    x, t = _rows(2, 4, 20000, "f32", 14)
    want = capi.tv_token_logprobs(x, t, top_k=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        outs.append(capi.tv_token_logprobs(x, t, top_k=6, stream=s))
        torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_row_offsets_past_32_bits():
    V = 128000
    N = (1 << 32) // V + 3
    x = torch.zeros(1, N, V, dtype=torch.bfloat16, device="cuda")
    x[0, N - 1].normal_()
    node = torch.tensor([[N - 1, 0]], dtype=torch.int32, device="cuda")
    tok = torch.tensor([[5, 6]], dtype=torch.int32, device="cuda")
    got = capi.tv_token_logprobs(x, tok, node=node, top_k=5)
    small = torch.stack((x[0, N - 1], x[0, 0]))[None].contiguous()
    want = _check(small, tok, None, 5)
    for g, w_ in zip(got, want):
        assert torch.equal(g, w_)


def test_nothing_to_do():
    x, t = _rows(2, 3, 50, "f32", 1)
    for tok, lg in ((t[:, :0].contiguous(), x), (t[:0], x[:0])):
        lp, ent, ids, top = capi.tv_token_logprobs(lg, tok, top_k=2)
        assert lp.numel() == 0 and ids.shape[-1] == 2


@pytest.mark.parametrize("captured", [False, True])
def test_a_plain_step_then_a_tree_step(captured):
    """Prompts appended, two plain steps (append, attend, report), a tree step over the same cache: every stage
    against the oracle's own chain of stages."""
    B, Hq, Hkv, D, bs, V = 3, 8, 2, 128, 16, 1500
    g = torch.Generator(device="cuda")
    g.manual_seed(17)
    dt = torch.bfloat16

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda").to(dt)

    lens0 = np.array([30, 1, 77])
    table_np, nblk = W.block_table_for(lens0 + 20, bs, 17)
    table = torch.from_numpy(table_np).cuda()
    kc, vc = torch.zeros(nblk, Hkv, bs, D, dtype=dt, device="cuda"), torch.zeros(nblk, Hkv, bs, D, dtype=dt, device="cuda")
    cs = capi.tv_rope_table(128, D)
    cu = torch.from_numpy(np.concatenate(([0], np.cumsum(lens0))).astype(np.int32)).cuda()
    kp, vp = randn(int(cu[-1]), Hkv, D), randn(int(cu[-1]), Hkv, D)
    lens = [torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(4)]
    steps = [(randn(B, Hq + 2 * Hkv, D), randn(B, 1, V), torch.randint(0, V, (B, 1), generator=g, device="cuda",
                                                                       dtype=torch.int32)) for _ in range(2)]
    ws = capi.alloc_workspace(capi.tv_decode_attn_workspace_size(Hq, Hkv, D, dt))
    q_out = [torch.empty(B, Hq, D, dtype=dt, device="cuda") for _ in steps]
    attn = [torch.empty(B, Hq, D, dtype=dt, device="cuda") for _ in steps]
    res = [[torch.empty(B, 1, device="cuda"), torch.empty(B, 1, device="cuda"),
            torch.empty(B, 1, 4, dtype=torch.int32, device="cuda"), torch.empty(B, 1, 4, device="cuda")] for _ in steps]

    def serve():
        capi.tv_kv_append(kp, vp, kc, vc, table, lens[0], cos_sin=cs, cu_new=cu, new_seq_lens=lens[1])
        for i, (qkv, logits, tok) in enumerate(steps):
            capi.tv_kv_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kc, vc, table, lens[1 + i], cos_sin=cs,
                              q=qkv[:, :Hq], q_out=q_out[i], new_seq_lens=lens[2 + i])
            capi.tv_decode_attn(q_out[i], kc, vc, table, lens[2 + i], out=attn[i], workspace=ws,
                                flags=capi.TV_ATTN_WORKSPACE_ZEROED)
            capi.tv_token_logprobs(logits, tok, top_k=4, logprob=res[i][0], entropy=res[i][1], top_ids=res[i][2],
                                   top_logprobs=res[i][3])

    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            serve()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            serve()
        for x in (kc, vc):
            x.zero_()
        graph.replay()
    else:
        serve()
    torch.cuda.synchronize()

    okc, ovc, olen, _ = OK.append_tokens(to_np(kc) * 0, to_np(vc) * 0, table_np, np.zeros(B, int), to_np(kp), to_np(vp),
                                         lens0, rope_base=10000.0)
    for i, (qkv, logits, tok) in enumerate(steps):
        x = to_np(qkv)
        okc, ovc, olen, oq = OK.append_tokens(okc, ovc, table_np, olen, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:],
                                              np.ones(B, int), q=x[:, :Hq], rope_base=10000.0)
        ref, _ = OA.decode_attention(oq, okc, ovc, table_np, olen)
        assert np.abs(to_np(attn[i]) - ref).max() <= 2e-2  # the library's tolerance for rows rotated and rounded to bf16
        np.testing.assert_array_equal(to_np(lens[2 + i]), olen)
        r = OL.token_logprobs(to_np(logits), to_np(tok), None, 4)
        np.testing.assert_array_equal(to_np(res[i][2]), r[2])
        np.testing.assert_allclose(to_np(res[i][0]), r[0], atol=2e-5)
    # the tree step reads what the plain steps left
    parent, _, _, _, n = capi.tv_tree_build(W.PAGE_TREE_PATHS)
    par = torch.from_numpy(parent).cuda()
    q, kt, vt = randn(B, n, Hq, D), randn(B, n, Hkv, D), randn(B, n, Hkv, D)
    kt_rot, q_rot = kt.clone(), q.clone()
    mask, _, _ = capi.tv_tree_prepare(par, lens[3], kt_rot, cs, q=q_rot)
    out = capi.tv_tree_attn_verify(q_rot, kc, vc, table, lens[3], kt_rot, vt, mask)
    ref, _ = OA.tree_attention(to_np(q), okc, ovc, table_np, olen, to_np(kt), to_np(vt), parent)
    assert np.abs(to_np(out) - ref).max() <= 2e-2


def _signs(got):
    lp, ent, ids, top = got
    assert not (lp > 0).any() and not (ent < 0).any() and not (top > 0).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(2000, 64), (500, 9000), (4, 100000)])
def test_confident_rows_keep_their_signs(dtype, rows, V):
    """A log probability is never above 0 and an entropy never below: rows that one token has to itself, nearly to
    itself, and shares, at many sizes of its logit; a row over one CTA and over several."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    t = torch.randint(0, V, (1, rows), generator=g, device="cuda", dtype=torch.int32)
    best = torch.rand(1, rows, 1, generator=g, device="cuda") * 80 - 40
    for rest in (-float("inf"), -60.0, -30.0, -17.0, -12.0):
        x = (best + rest).expand(1, rows, V).clone()
        x.scatter_(2, t[..., None].long(), best)
        x = x.to(DT[dtype])
        got = _check(x, t, top_k=3)
        _signs(got)
        if rest == -float("inf"):  # the rounding of a sum of one term, taken away again
            assert (got[0].abs() <= 2.0 ** -20).all() and (got[1] <= 2.0 ** -20).all()
    x = (torch.randn(1, rows, V, generator=g, device="cuda") * 6 + best).to(DT[dtype])
    _signs(_check(x, t, top_k=3))


@pytest.mark.parametrize("name", sorted(_special()))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_copy_of_a_special_row(name, dtype):
    """400 entries of one row: all four outputs the same in each, the first within the bounds of the oracle."""
    x = _special()[name].to(DT[dtype]).cuda().view(1, 1, -1)
    many = capi.tv_token_logprobs(x, torch.full((1, 400), 31234, dtype=torch.int32, device="cuda"),
                                  node=torch.zeros(1, 400, dtype=torch.int32, device="cuda"), top_k=32)
    for m in many:
        bits = m.view(torch.int32)
        assert torch.equal(bits, bits[:, :1].expand_as(bits))
    # entries of their own are one CTA each too: the same bits, within the bounds of _check
    rows = x.expand(1, 160, -1).contiguous()
    first = _check(rows, torch.full((1, 160), 31234, dtype=torch.int32, device="cuda"), top_k=32)
    for m, f in zip(many, first):
        assert torch.equal(m[:, 0].view(torch.int32), f[:, 0].view(torch.int32))
