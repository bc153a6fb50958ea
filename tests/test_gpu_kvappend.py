"""GPU parity of tv_kv_append (new tokens' K/V into the paged cache, keys and
queries rotated on the way) against the float64 oracle and, bit for bit,
against tv_rope_apply."""

import numpy as np
import pytest
import torch

from gpu_helpers import to_np
from oracle import kvcache as OK
from speculative_decoding_tree_attn_gb300 import capi
from speculative_decoding_tree_attn_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _case(lens, counts, Hq, Hkv, D, dtype, bs, seed, pad=0, fused=True, max_pos=None):
    """Cache, table and packed q/k/v rows (slices of one projection when fused)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[dtype]
    lens, counts = np.asarray(lens, dtype=np.int32), np.asarray(counts, dtype=np.int32)
    table, nblk = W.block_table_for(lens + counts, bs, seed, spare_blocks=2)
    T = int(counts.sum()) + pad
    c = {"k_cache": torch.randn(nblk, Hkv, bs, D, generator=g, device="cuda").to(dt),
         "v_cache": torch.randn(nblk, Hkv, bs, D, generator=g, device="cuda").to(dt),
         "table": torch.from_numpy(table).cuda(), "lens": torch.from_numpy(lens).cuda(), "counts": counts,
         "cu": torch.from_numpy(np.concatenate(([0], np.cumsum(counts))).astype(np.int32)).cuda()}
    rows = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").to(dt)
    c["q"], c["k"], c["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    if not fused:
        c["q"], c["k"], c["v"] = (c[n].contiguous() for n in "qkv")
    c["cs"] = capi.tv_rope_table(int((lens + counts).max()) + 1 if max_pos is None else max_pos, D)
    return c


def _append(c, rope=True, cu=True, status=None, q_out=None):
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    q, lens = capi.tv_kv_append(c["k"], c["v"], kc, vc, c["table"], c["lens"], cos_sin=c["cs"] if rope else None,
                                q=c["q"] if rope else None, q_out=q_out, cu_new=c["cu"] if cu else None, status=status)
    torch.cuda.synchronize()
    return kc, vc, lens, q


def _oracle(c, rope=True, max_pos=None):
    return OK.append_tokens(to_np(c["k_cache"]), to_np(c["v_cache"]), c["table"].cpu().numpy(),
                            c["lens"].cpu().numpy(), to_np(c["k"]), to_np(c["v"]), c["counts"],
                            q=to_np(c["q"]) if rope else None, rope_base=10000.0 if rope else None, max_pos=max_pos)


def _held(got, want, pair_norm, dt):
    """One rounding to the type (half a step of the value, and of the type's smallest spacing), plus the float32
    rotation: the table entry is off by half a step of float32, the product and the sum by another each, so by
    3 * 2^-24 of |x1| + |x2| <= 2 * pair_norm together, with room for the rounding after it."""
    got = to_np(got).astype(np.float64)
    u = torch.finfo(dt).eps / 2
    assert (np.abs(got - want) <= u * np.abs(want) * (1 + u) + 2 * 3 * 2.0 ** -24 * pair_norm * (1 + u)).all()


def _check(c, kc, vc, lens, q, rope=True):
    okc, ovc, olens, oq = _oracle(c, rope)
    dt = c["k_cache"].dtype
    np.testing.assert_array_equal(lens.cpu().numpy(), olens)
    np.testing.assert_array_equal(to_np(vc), ovc)
    if not rope:
        np.testing.assert_array_equal(to_np(kc), okc)
        return
    half = okc.shape[-1] // 2
    norm = np.sqrt(okc[..., :half] ** 2 + okc[..., half:] ** 2)
    _held(kc, okc, np.concatenate((norm, norm), -1), dt)
    n = int(c["counts"].sum())
    norm = np.sqrt(oq[:n, :, :half] ** 2 + oq[:n, :, half:] ** 2)
    _held(q[:n], oq[:n], np.concatenate((norm, norm), -1), dt)


@pytest.mark.parametrize("lens,counts,Hq,Hkv,D,dtype,bs", [
    ([0], [1], 1, 1, 64, "f32", 16),
    ([37], [1], 32, 8, 128, "bf16", 16),
    ([0, 15, 16, 17, 100], [1, 1, 1, 1, 1], 8, 2, 128, "bf16", 16),
    ([0, 3, 0, 40, 7], [17, 0, 64, 1, 0], 4, 4, 256, "bf16", 24),
    ([5, 0, 31], [300, 129, 2], 5, 1, 16, "f32", 1),
    ([1, 2], [33, 1000], 3, 3, 32, "bf16", 7),
    ([0] * 70, list(range(70)), 6, 2, 64, "f32", 64),
    ([2048], [2049], 64, 8, 128, "bf16", 64),
])
def test_append_matches_the_oracle(lens, counts, Hq, Hkv, D, dtype, bs):
    c = _case(lens, counts, Hq, Hkv, D, dtype, bs, 1000 + D + bs, pad=3)
    q_out = torch.full((c["q"].shape[0], Hq, D), 7.0, device="cuda", dtype=DT[dtype])
    kc, vc, got, q = _append(c, q_out=q_out)
    _check(c, kc, vc, got, q)
    assert (q[int(np.sum(counts)):] == 7.0).all()  # rows behind the last request


def test_append_without_rotation_copies_bits():
    c = _case([3, 0, 20], [5, 1, 40], 2, 2, 64, "bf16", 16, 5)
    c["k"].view(torch.int16)[0, 0, :4] = torch.tensor([0x7F81, -1, 0x7F80, -32768], device="cuda", dtype=torch.int16)
    kc, vc, got, q = _append(c, rope=False)
    assert q is None
    okc, ovc, olens, _ = _oracle(c, rope=False)
    np.testing.assert_array_equal(got.cpu().numpy(), olens)
    np.testing.assert_array_equal(to_np(vc), ovc)
    np.testing.assert_array_equal(to_np(kc), okc)  # NaN equals NaN here
    blk, slot = int(c["table"][0, 0]), 3
    assert torch.equal(kc[blk, 0, slot, :4].view(torch.int16), c["k"][0, 0, :4].view(torch.int16))


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128)])
def test_rotation_has_the_bits_of_rope_apply(dtype, D):
    c = _case([7, 100, 0], [4, 4, 4], 8, 2, D, dtype, 16, 9, fused=False)
    kc, vc, lens, q = _append(c, cu=False)  # no offsets: T / B tokens each
    pos = c["lens"][:, None] + torch.arange(4, device="cuda", dtype=torch.int32)[None]
    q2, k2 = c["q"].clone().view(3, 4, 8, D), c["k"].clone().view(3, 4, 2, D)
    capi.tv_rope_apply(q2, k2, pos.contiguous(), c["cs"])
    assert torch.equal(q.view(3, 4, 8, D), q2)
    bs = 16
    for b in range(3):
        for j in range(4):
            p = int(pos[b, j])
            assert torch.equal(kc[int(c["table"][b, p // bs]), :, p % bs], k2[b, j])
    assert torch.equal(lens, c["lens"] + 4)


def test_in_place_queries_and_offsets_agree():
    c = _case([9, 50], [6, 6], 4, 1, 64, "bf16", 16, 11)
    kc, vc, lens, q = _append(c)
    q_in = c["q"].clone()
    c2 = dict(c, q=q_in)
    kc2, vc2, lens2, q2 = _append(c2, cu=False, q_out=q_in)
    assert q2.data_ptr() == q_in.data_ptr()
    assert torch.equal(q, q2) and torch.equal(kc, kc2) and torch.equal(vc, vc2) and torch.equal(lens, lens2)


def _one_by_one(c, cs, q_out, status, skip=()):
    """The same appends a request at a time, from contiguous rows."""
    kc, vc, lens = c["k_cache"].clone(), c["v_cache"].clone(), c["lens"].clone()
    at = 0
    for b, n in enumerate(c["counts"]):
        rows = slice(at, at + int(n))
        at += int(n)
        if n == 0 or b in skip:
            continue
        lens[b] = capi.tv_kv_append(c["k"][rows], c["v"][rows], kc, vc, c["table"][b:b + 1].contiguous(),
                                    c["lens"][b:b + 1].contiguous(), cos_sin=cs, q=None if q_out is None else c["q"][rows],
                                    q_out=None if q_out is None else q_out[rows], status=status)[1][0]
    return kc, vc, lens


@pytest.mark.parametrize("Hq,Hkv,D,dtype,bs", [(4, 1, 64, "bf16", 24), (4, 1, 128, "bf16", 16), (2, 1, 256, "bf16", 64),
                                               (2, 1, 64, "f32", 16), (8, 2, 64, "f32", 1), (16, 8, 16, "bf16", 16),
                                               (1, 1, 32, "f32", 7), (1, 1, 256, "f32", 16)])
@pytest.mark.parametrize("rope", ["q and k", "k", "none"])
def test_long_prompts_of_few_heads(Hq, Hkv, D, dtype, bs, rope):
    """Tens of thousands of tokens in one call have the bits of a call per request."""
    rng = np.random.default_rng(D + Hq)
    counts = rng.integers(0, 1500, 40)
    counts[[3, 17]] = 0, 1
    c = _case(rng.integers(0, 300, 40), counts, Hq, Hkv, D, dtype, bs, 31, pad=5)
    cs = None if rope == "none" else c["cs"]
    outs = [torch.full((c["q"].shape[0], Hq, D), 7.0, device="cuda", dtype=DT[dtype]) for _ in range(2)]
    if rope != "q and k":
        outs = [None, None]
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, lens = capi.tv_kv_append(c["k"], c["v"], kc, vc, c["table"], c["lens"], cos_sin=cs, cu_new=c["cu"],
                                q=None if outs[0] is None else c["q"], q_out=outs[0], status=status)
    kc1, vc1, lens1 = _one_by_one(c, cs, outs[1], status)
    assert torch.equal(kc, kc1) and torch.equal(vc, vc1) and torch.equal(lens, lens1) and int(status.item()) == 0
    assert outs[0] is None or torch.equal(*outs)
    if rope == "q and k":
        _check(c, kc, vc, lens, outs[0])


def test_long_prompts_with_faults_and_without_offsets():
    c = _case([9, 0, 1000, 30, 3], [4000] * 5, 4, 1, 64, "bf16", 16, 37, max_pos=4600)
    c["table"][0, 100] = -1
    c["table"][3, 7] = c["k_cache"].shape[0]
    c["lens"][4] = -2
    outs = [torch.full((c["q"].shape[0], 4, 64), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    seen = torch.zeros(3, dtype=torch.int32, device="cuda")
    want = _one_by_one(c, c["cs"], outs[1], seen[2:])
    for i, cu in enumerate((c["cu"], None)):
        kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
        outs[0].fill_(7.0)
        _, lens = capi.tv_kv_append(c["k"], c["v"], kc, vc, c["table"], c["lens"], cos_sin=c["cs"], cu_new=cu, q=c["q"],
                                    q_out=outs[0], status=seen[i:i + 1])
        assert torch.equal(kc, want[0]) and torch.equal(vc, want[1]) and torch.equal(lens, want[2]) and torch.equal(*outs)
    assert seen.tolist() == [capi.TV_DEV_BAD_POSITION | capi.TV_DEV_OUT_OVERFLOW] * 3
    c["cu"][5] += 1  # past the rows: the last request gets nothing, the others as before
    c["lens"][4] = 3
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    _, lens = capi.tv_kv_append(c["k"], c["v"], kc, vc, c["table"], c["lens"], cos_sin=c["cs"], cu_new=c["cu"], q=c["q"],
                                status=seen[:1])
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1]) and torch.equal(lens[:4], want[2][:4]) and int(lens[4]) == 3
    assert int(seen[0]) & capi.TV_DEV_BAD_OFFSETS


def test_tokens_that_cannot_be_placed_end_the_length():
    """A short table row, a bad entry, a position past the rotary table, a negative length, bad offsets."""
    bs = 16
    c = _case([14, 3, 30, 5, 0], [4, 30, 6, 3, 2], 2, 1, 64, "f32", bs, 13, max_pos=33)
    table = c["table"].clone()
    table[1, 1] = c["k_cache"].shape[0] + 4  # positions 16..31 of request 1
    c["table"] = table
    lens = c["lens"].clone()
    lens[3] = -2
    c["lens"] = lens
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc, got, q = _append(c, status=status)
    okc, ovc, olens, oq = _oracle(c, max_pos=33)
    assert int(status.item()) == capi.TV_DEV_OUT_OVERFLOW | capi.TV_DEV_BAD_POSITION
    np.testing.assert_array_equal(olens, [18, 16, 33, -2, 2])
    np.testing.assert_array_equal(got.cpu().numpy(), olens)
    np.testing.assert_array_equal(to_np(vc), ovc)
    np.testing.assert_allclose(to_np(kc), okc, atol=1e-5)
    # offsets that decrease or leave [0, T]: those requests get nothing, the others all of theirs
    cu = torch.tensor([0, 4, 34, 30, 43, 99], dtype=torch.int32, device="cuda")
    status.zero_()
    kc2, vc2, got, q = _append(dict(c, cu=cu, lens=torch.tensor([14, 0, 0, 5, 0], dtype=torch.int32, device="cuda"),
                                    table=c["table"].clamp(max=c["k_cache"].shape[0] - 1)), status=status)
    assert int(status.item()) & capi.TV_DEV_BAD_OFFSETS
    assert got.tolist()[0] == 18 and got.tolist()[2] == 0 and got.tolist()[4] == 0


def test_a_zero_batch_and_zero_tokens():
    c = _case([4, 5], [0, 0], 2, 1, 64, "f32", 16, 17)
    for cu in (True, False):
        kc, vc, lens, q = _append(c, cu=cu)
        assert torch.equal(lens, c["lens"]) and torch.equal(kc, c["k_cache"]) and torch.equal(vc, c["v_cache"])
    e = dict(c, lens=c["lens"][:0], table=c["table"][:0], cu=c["cu"][:1])
    kc, vc, lens, q = _append(e)
    assert lens.numel() == 0 and torch.equal(kc, c["k_cache"])


def test_cache_offsets_past_32_bits():
    """A cache of more than 2^32 bytes (and elements past 2^31): the last blocks are written where they belong."""
    Hkv, bs, D = 8, 64, 128
    nblk = (1 << 31) // (Hkv * bs * D) + 8
    kc = torch.zeros(nblk, Hkv, bs, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.tensor([[nblk - 1], [nblk - 2], [0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([63, 0, 5], dtype=torch.int32, device="cuda")
    k = torch.randn(3, Hkv, D, device="cuda").to(torch.bfloat16)
    v = torch.randn(3, Hkv, D, device="cuda").to(torch.bfloat16)
    _, new = capi.tv_kv_append(k, v, kc, vc, table, lens)
    assert new.tolist() == [64, 1, 6]
    for b, (blk, slot) in enumerate([(nblk - 1, 63), (nblk - 2, 0), (0, 5)]):
        assert torch.equal(kc[blk, :, slot], k[b]) and torch.equal(vc[blk, :, slot], v[b])
    assert int((kc != 0).any(-1).sum()) == int((k != 0).any(-1).sum())


def test_append_then_tree_attention_reads_the_prompt():
    """A prompt put in by tv_kv_append serves tree attention as the same prefix written by hand."""
    w = W.Workload("case", 3, 8, 2, 128, "bf16", ("fixed", 0), 16, (0.7, 0.15), 10, 4, 23)
    parent, _, _, _, n = capi.tv_tree_build(W.PAGE_TREE_PATHS)
    lens = np.array([50, 1, 130], dtype=np.int32)
    inp = W.attention_inputs(w, device="cuda", seq_lens=lens)
    mask, _, _ = capi.tv_tree_mask(torch.from_numpy(parent).cuda(), inp["seq_lens"])
    want = capi.tv_tree_attn_verify(inp["q"], inp["k_cache"], inp["v_cache"], inp["block_table"], inp["seq_lens"],
                                    inp["k_tree"], inp["v_tree"], mask)
    rows = []
    for cache in (inp["k_cache"], inp["v_cache"]):
        rows.append(torch.cat([cache[inp["block_table"][b].long()].transpose(1, 2).reshape(-1, 2, 128)[:int(lens[b])]
                               for b in range(3)]))
    kc, vc = torch.zeros_like(inp["k_cache"]), torch.zeros_like(inp["v_cache"])
    cu = torch.from_numpy(np.concatenate(([0], np.cumsum(lens))).astype(np.int32)).cuda()
    _, new = capi.tv_kv_append(rows[0], rows[1], kc, vc, inp["block_table"], torch.zeros_like(inp["seq_lens"]),
                               cu_new=cu)
    assert torch.equal(new, inp["seq_lens"])
    got = capi.tv_tree_attn_verify(inp["q"], kc, vc, inp["block_table"], new, inp["k_tree"], inp["v_tree"], mask)
    assert torch.equal(got, want)


def test_one_token_with_any_stride():
    c = _case([7], [1], 4, 2, 64, "bf16", 16, 31, fused=False)
    want = _append(c, cu=False)
    odd = {}
    for n in "qkv":
        odd[n] = torch.empty(c[n].shape[1], 64, 1, device="cuda", dtype=torch.bfloat16).permute(2, 0, 1)
        odd[n].copy_(c[n])
        assert odd[n].stride(0) == 1
    for a, b in zip(_append(dict(c, **odd), cu=False), want):
        assert torch.equal(a, b)


def test_a_step_captured_and_replayed():
    """Replays append at the lengths that are in the buffer then; the offsets may change too."""
    c = _case([5, 30], [1, 1], 4, 2, 64, "bf16", 16, 33, fused=False)
    kc, vc = torch.zeros_like(c["k_cache"]), torch.zeros_like(c["v_cache"])
    new, q_out = torch.empty_like(c["lens"]), torch.empty_like(c["q"])
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lens = c["lens"].clone()

    def call():
        capi.tv_kv_append(c["k"], c["v"], kc, vc, c["table"], lens, cos_sin=c["cs"], q=c["q"], q_out=q_out, cu_new=cu,
                          new_seq_lens=new)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for at, offsets in (([5, 30], [0, 1, 2]), ([0, 14], [0, 0, 2]), ([4, 2], [0, 2, 2])):
        lens.copy_(torch.tensor(at, dtype=torch.int32))
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        kc.zero_()
        vc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
        q2, l2 = capi.tv_kv_append(c["k"], c["v"], k2, v2, c["table"], lens, cos_sin=c["cs"], q=c["q"], cu_new=cu)
        assert torch.equal(kc, k2) and torch.equal(vc, v2) and torch.equal(new, l2) and torch.equal(q_out, q2)
        assert l2.tolist() == [at[b] + offsets[b + 1] - offsets[b] for b in range(2)]


def test_binding_checks_every_argument():
    c = _case([7, 3], [2, 2], 4, 2, 64, "bf16", 16, 35, fused=False)
    good = dict(k_new=c["k"], v_new=c["v"], k_cache=c["k_cache"], v_cache=c["v_cache"], block_table=c["table"],
                seq_lens=c["lens"], cos_sin=c["cs"], q=c["q"], cu_new=c["cu"])
    bad = dict(k_new=c["k"].float(), v_new=c["v"][:3], k_cache=c["k_cache"][0], v_cache=c["v_cache"].float(),
               block_table=c["table"].long(), seq_lens=c["lens"].cpu(), cos_sin=c["cs"][:, 0], q=c["q"][0],
               cu_new=c["cu"][:2], q_out=c["q"].float(), new_seq_lens=c["lens"].long(), status=c["lens"].float())
    for name, x in bad.items():
        with pytest.raises(ValueError, match=name):
            capi.tv_kv_append(**{**good, name: x})
    with pytest.raises(capi.TVError, match="cos_sin"):
        capi.tv_kv_append(**{**good, "cos_sin": None})
    with pytest.raises(capi.TVError, match="alias"):
        capi.tv_kv_append(**good, new_seq_lens=c["lens"])


def test_a_bad_block_before_the_end_of_the_table():
    """One request with a missing block and, behind it, positions past the rotary table: both are reported, and the
    queries past the table are left as they were."""
    c = _case([10], [60], 2, 1, 64, "f32", 16, 41, max_pos=50)
    c["table"][0, 1] = -1
    q_out = torch.full((60, 2, 64), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc, lens, q = _append(c, status=status, q_out=q_out)
    assert int(status.item()) == capi.TV_DEV_OUT_OVERFLOW | capi.TV_DEV_BAD_POSITION
    assert lens.tolist() == [16]
    assert (q[40:] == 7.0).all() and (q[:40] != 7.0).any(-1).all()
    okc, ovc, olens, _ = _oracle(c, max_pos=50)
    np.testing.assert_array_equal(to_np(vc), ovc)
    np.testing.assert_array_equal(olens, [16])


def _random_offsets(rng, B, T):
    """Offsets in order, then some of them moved anywhere, a little past [0, T] too."""
    cu = np.sort(rng.integers(0, T + 1, B + 1))
    cu[0], cu[-1] = 0, T
    for i in rng.choice(B + 1, size=int(rng.integers(1, 4)), replace=False):
        cu[i] = rng.integers(-2, T + 3)
    return cu.astype(np.int32)


@pytest.mark.parametrize("B,T", [(3, 10), (5, 45), (33, 200), (100, 900), (1500, 3000), (40, 9000)])
def test_offsets_out_of_order_count_no_token_that_is_not_stored(B, T):
    """Whatever the offsets, a length that is returned covers rows of its request that are in the cache; a batch in
    order has all of them.  9000 tokens of one head go eight to a warp."""
    rng = np.random.default_rng(B)
    bs, Hkv, D = 16, 1, 64
    lens0 = rng.integers(0, 40, B).astype(np.int32)
    width = (40 + T) // bs + 2 if B <= 100 else 8
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    k = torch.randn(T, Hkv, D, generator=g, device="cuda")
    v = torch.randn(T, Hkv, D, generator=g, device="cuda")
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    lens = torch.from_numpy(lens0).cuda()
    cases = [np.array([0, 10, 5, 8], dtype=np.int32)] if B == 3 else []
    cases += [_random_offsets(rng, B, T) for _ in range(12)]
    for cu in cases:
        kc = torch.full((B * width, Hkv, bs, D), 7.0, device="cuda")
        vc = kc.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        _, new = capi.tv_kv_append(k, v, kc, vc, table, lens, cu_new=torch.from_numpy(cu).cuda(), status=status)
        n = (new - lens).cpu().numpy()
        ordered = (np.diff(cu) >= 0).all() and cu[0] >= 0 and cu[-1] <= T
        assert (n >= 0).all()
        if ordered:
            assert int(status) & capi.TV_DEV_BAD_OFFSETS == 0
        else:
            assert int(status) & capi.TV_DEV_BAD_OFFSETS
        for b in range(B):
            s0, s1 = int(cu[b]), int(cu[b + 1])
            room = max(0, min(s1 - s0, width * bs - int(lens0[b])))
            assert n[b] in ((room,) if ordered else (0, room))
            if n[b]:
                at = torch.arange(int(lens0[b]), int(lens0[b]) + int(n[b]), device="cuda")
                blk = table[b, at // bs].long()
                assert torch.equal(kc[blk, :, at % bs], k[s0:s0 + n[b]]) and torch.equal(vc[blk, :, at % bs], v[s0:s0 + n[b]])
