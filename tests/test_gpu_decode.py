"""GPU parity of tv_decode_attn (one new token per request over the paged
cache) against the float64 oracle, with score caps, windows, kept first keys
and distance biases, on split and whole rows."""

import numpy as np
import pytest
import torch

from gpu_helpers import to_np
from oracle import attention as OA
from speculative_decoding_tree_attn_gb300 import capi
from speculative_decoding_tree_attn_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _case(lens, Hq, Hkv, D, dtype, bs, seed, spare=2, poison=True, qscale=1.0):
    """q, caches, table; with ``poison`` every cache slot that holds no key is NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[dtype]
    lens = np.asarray(lens, dtype=np.int32)
    table, nblk = W.block_table_for(lens, bs, seed, spare_blocks=spare)
    c = {"q": (torch.randn(lens.size, Hq, D, generator=g, device="cuda") * qscale).to(dt),
         "k": torch.randn(nblk, Hkv, bs, D, generator=g, device="cuda").to(dt),
         "v": torch.randn(nblk, Hkv, bs, D, generator=g, device="cuda").to(dt),
         "table": torch.from_numpy(table).cuda(), "lens": torch.from_numpy(lens).cuda()}
    if poison:
        _poison(c, [np.arange(n) for n in lens])
    return c


def _poison(c, keys):
    """NaN in every cache slot that is not one of the requests' given positions."""
    bs = c["k"].shape[2]
    keep = np.zeros((c["k"].shape[0], bs), dtype=bool)
    table = c["table"].cpu().numpy()
    for b, t in enumerate(keys):
        keep[table[b, t // bs], t % bs] = True
    gone = torch.from_numpy(~keep).cuda()[:, None, :, None]
    for n in "kv":
        c[n].masked_fill_(gone, float("nan"))


def _run(c, **opt):
    B, Hq, D = c["q"].shape
    lse = torch.full((B, Hq), 123.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = capi.tv_decode_attn(c["q"], c["k"], c["v"], c["table"], c["lens"], lse=lse, status=status, **opt)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out, lse


def _check(c, out, lse, lens=None, **opt):
    """The kernel's own errors, all relative to sum p|v| (A) or absolute in a score: a score's float32 sum of D
    products (D 2^-24 |q||k| scale), its roundings through scale, cap, bias and log2 e (16 of them at the largest score)
    and the cap's tanh (2^-20 of cap); a weight 2^-21 for the exponential and, for bf16, 2^-16 for being held in two
    bf16 parts; float32 sums of up to L/8 + 16 terms one after another; the output rounded once."""
    q, k, v = (np.nan_to_num(to_np(c[n]).astype(np.float64)) for n in ("q", "k", "v"))
    table = c["table"].cpu().numpy()
    lens = c["lens"].cpu().numpy() if lens is None else np.asarray(lens)
    oopt = {n: (to_np(x) if isinstance(x, torch.Tensor) else x) for n, x in opt.items()}
    ref, rlse = OA.decode_attention(q, k, v, table, lens, **oopt)
    mean, _ = OA.decode_attention(q, k, np.abs(v), table, lens, **oopt)
    D, dt = q.shape[-1], c["q"].dtype
    scale = opt.get("scale") or 1.0 / np.sqrt(D)
    top = np.linalg.norm(q, axis=-1) * np.linalg.norm(k, axis=-1).max() * abs(scale)  # [B, Hq], Cauchy-Schwarz
    big = top.copy()
    cap = opt.get("softcap", 0.0)
    if cap:
        big = np.minimum(big, cap)
    if opt.get("slopes") is not None:
        big = big + np.abs(oopt["slopes"])[None] * np.maximum(lens, 1)[:, None]
    ds = D * 2.0 ** -24 * top + 16 * 2.0 ** -24 * np.maximum(top, big) + 2.0 ** -20 * cap
    sums = (lens[:, None] / 8 + 16) * 2.0 ** -24 + 2.0 ** -21
    w = 2 * ds + 2 * sums + (2.0 ** -16 if dt == torch.bfloat16 else 0.0)
    got, glse = to_np(out).astype(np.float64), to_np(lse).astype(np.float64)
    u = torch.finfo(dt).eps / 2
    bound = u * np.abs(ref) + (1 + u) * w[..., None] * mean
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= bound).all(), float((np.abs(got - ref) - bound).max())
    fin = np.isfinite(rlse)
    assert np.array_equal(np.isfinite(glse), fin) and (glse[~fin] == -np.inf).all()
    err = np.abs(np.where(fin, glse, 0) - np.where(fin, rlse, 0))
    lb = ds + sums + 4 * 2.0 ** -24 * np.abs(np.where(fin, rlse, 0))
    assert (err <= lb).all(), float((err - lb).max())
    assert (got[~fin] == 0).all()


LENS = [0, 1, 15, 16, 17, 127, 128, 129, 255, 300, 1000]


@pytest.mark.parametrize("Hq,Hkv,D,dtype,bs", [
    (4, 4, 64, "f32", 16), (32, 8, 128, "bf16", 16), (8, 1, 128, "bf16", 64), (8, 1, 256, "bf16", 16),
    (10, 2, 64, "bf16", 24), (12, 1, 128, "bf16", 1), (16, 1, 64, "bf16", 7), (40, 1, 128, "bf16", 16),
    (6, 2, 256, "f32", 13), (18, 1, 128, "f32", 32), (17, 1, 256, "bf16", 48), (3, 3, 128, "bf16", 128),
    (128, 1, 64, "bf16", 16), (5, 1, 64, "f32", 256),
])
@pytest.mark.parametrize("num_ctas", [0, 5])
def test_every_length_and_layout(Hq, Hkv, D, dtype, bs, num_ctas):
    c = _case(LENS, Hq, Hkv, D, dtype, bs, 2000 + Hq + D + bs)
    out, lse = _run(c, num_ctas=num_ctas)
    _check(c, out, lse)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128)])
@pytest.mark.parametrize("num_ctas", [1, 2, 3, 37, 151, 1000, 4096])
def test_splits(dtype, D, num_ctas):
    c = _case([3000, 0, 77, 4097, 1], 8, 2, D, dtype, 16, 31 + D)
    out, lse = _run(c, num_ctas=num_ctas)
    _check(c, out, lse)


@pytest.mark.parametrize("G,D,dtype", [(1, 64, "bf16"), (4, 128, "bf16"), (8, 128, "bf16"), (16, 64, "bf16"),
                                       (12, 128, "bf16"), (3, 256, "bf16"), (1, 64, "f32"), (2, 128, "f32"),
                                       (8, 256, "f32"), (5, 128, "f32")])
@pytest.mark.parametrize("num_ctas", [4, 10, 16])
def test_heads_read_together(G, D, dtype, num_ctas):
    """Enough work a CTA that its warps take several KV heads at a time; requests cut between CTAs, unused slots."""
    c = _case([1000, 990, 0, 1003, 997, 1, 960, 1000, 985], 8 * G, 8, D, dtype, 16, 2500 + G + D)
    out, lse = _run(c, num_ctas=num_ctas)
    _check(c, out, lse)


@pytest.mark.parametrize("G,Hkv", [(16, 1), (9, 2), (16, 3), (12, 8), (40, 4)])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("num_ctas", [0, 1, 6, 33])
def test_many_heads_on_one(G, Hkv, D, num_ctas):
    """KV heads with more than 8 query heads, requests whole, cut and shared by warps, one after another in a CTA."""
    c = _case([700, 0, 3000, 33, 1, 16, 500], G * Hkv, Hkv, D, "bf16", 16, 2600 + G + D)
    out, lse = _run(c, num_ctas=num_ctas)
    _check(c, out, lse)


OPTIONS = [
    dict(softcap=5.0), dict(softcap=30.0, scale=0.7), dict(window=1), dict(window=100), dict(window=128, n_sink=4),
    dict(window=33, n_sink=17), dict(window=1000, n_sink=50), dict(window=5, n_sink=100000), dict(n_sink=4),
    dict(slopes=True), dict(slopes=True, softcap=10.0, window=200, n_sink=3), dict(scale=0.0),
    dict(scale=-0.3), dict(window=2 ** 31 - 1, n_sink=2 ** 31 - 1),
]


@pytest.mark.parametrize("opt", OPTIONS, ids=[str(i) for i in range(len(OPTIONS))])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,bs", [(8, 2, 128, "bf16", 16), (12, 1, 64, "bf16", 10), (5, 1, 64, "f32", 16)])
def test_masks_caps_and_biases(opt, Hq, Hkv, D, dtype, bs):
    """Invisible keys are poisoned too: a window or kept first keys read nothing else."""
    opt = dict(opt)
    lens = [0, 1, 4, 33, 128, 500, 1025]
    c = _case(lens, Hq, Hkv, D, dtype, bs, 50 + Hq + bs, poison=False, qscale=3.0)
    if opt.pop("slopes", None):
        opt["slopes"] = torch.pow(2.0, -8.0 * torch.arange(1, Hq + 1, device="cuda").float() / Hq)
    w, s = opt.get("window", 0), opt.get("n_sink", 0)
    keys = [np.arange(n) for n in lens]
    if w:
        keys = [t[(t >= t.size - w) | (t < s)] for t in keys]
    _poison(c, keys)
    for num_ctas in (0, 9):
        out, lse = _run(c, num_ctas=num_ctas, **opt)
        _check(c, out, lse, **opt)


@pytest.mark.parametrize("cap,scale", [(50.0, None), (50.0, 3.0), (8.0, 0.5), (1.0, 0.3)])
def test_a_cap_keeps_float32(cap, scale):
    """The cap's tanh is good to a few float32 roundings of itself, small scores and large: the output's error against
    the oracle, over its norm, stays by the float32 sums' own (D / 2 roundings of a score, at most 2^-24 of it each)."""
    c = _case([900, 2000, 64], 4, 2, 128, "f32", 16, 63)
    opt = dict(softcap=cap, **({"scale": scale} if scale else {}))
    out, lse = _run(c, **opt)
    ref, rlse = OA.decode_attention(to_np(c["q"]), np.nan_to_num(to_np(c["k"])), np.nan_to_num(to_np(c["v"])),
                                    c["table"].cpu().numpy(), c["lens"].cpu().numpy(), **opt)
    # a score's error: 6 roundings for the tanh and at most 62 in the sum of its 128 products, of the largest score's size
    top = min(cap, float(np.abs(rlse).max()))
    assert np.linalg.norm(to_np(out) - ref) <= 2 * 68 * 2.0 ** -24 * max(top, 1.0) * np.linalg.norm(ref)
    assert np.abs(to_np(lse) - rlse).max() <= 68 * 2.0 ** -24 * max(top, 1.0)


def test_a_cap_near_zero():
    """Every score is held at the cap: all keys alike, zeros among them."""
    c = _case([300, 17], 4, 2, 64, "bf16", 16, 61)
    c["q"][0, 0] = 0
    for cap in (1e-3, 1e-30, 1e-38):
        out, lse = _run(c, softcap=cap)
        _check(c, out, lse, softcap=cap)


def test_one_request_with_any_stride():
    c = _case([100], 4, 2, 64, "bf16", 16, 62)
    want, _ = _run(c)
    odd = torch.empty(4, 64, 1, device="cuda", dtype=torch.bfloat16).permute(2, 0, 1)
    odd.copy_(c["q"])
    assert odd.stride(0) == 1
    got, _ = _run(dict(c, q=odd))
    assert torch.equal(got, want)


def test_extreme_scores():
    """Scores far apart and all alike: one key takes everything, or all share it."""
    c = _case([700, 64], 4, 1, 128, "bf16", 16, 71, qscale=60.0)
    out, lse = _run(c)
    _check(c, out, lse)
    c["q"].zero_()
    out, lse = _run(c)
    _check(c, out, lse)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128)])
@pytest.mark.parametrize("num_ctas", [0, 3])
def test_scores_of_minus_infinity(dtype, D, num_ctas):
    """A bias that takes all but a request's last two keys below float32: the last key has all the weight."""
    lens = [1000, 17, 1, 300, 2, 0]
    c = _case(lens, 8, 2, D, dtype, 16, 73)
    slopes = torch.full((8,), 2e38, device="cuda")
    out, lse = _run(c, slopes=slopes, num_ctas=num_ctas)
    q, k = (to_np(c[n]).astype(np.float64) for n in "qk")
    for b, L in enumerate(lens):
        if L == 0:
            assert (out[b] == 0).all() and (lse[b] == -np.inf).all()
            continue
        blk, slot = int(c["table"][b, (L - 1) // 16]), (L - 1) % 16
        assert torch.equal(out[b], c["v"][blk, :, slot].repeat_interleave(4, 0))
        key = k[blk, :, slot].repeat(4, 0)
        s = (q[b] * key).sum(-1) / np.sqrt(D)
        # the float32 sum of D products and the roundings through scale and log2 e
        size = np.linalg.norm(q[b], axis=-1) * np.linalg.norm(key, axis=-1) / np.sqrt(D)
        assert (np.abs(to_np(lse)[b] - s) <= (D + 16) * 2.0 ** -24 * size).all()


def test_strided_queries_and_a_given_output():
    c = _case([40, 9, 200], 8, 2, 128, "bf16", 16, 81)
    want, _ = _run(c)
    wide = torch.full((3, 12, 128), 5.0, device="cuda", dtype=torch.bfloat16)
    wide[:, 2:10] = c["q"]
    out = torch.full_like(want, 9.0)
    got, _ = _run(dict(c, q=wide[:, 2:10]), out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)


def test_lengths_outside_the_table_are_clamped():
    c = _case([48, 32, 5], 4, 1, 64, "bf16", 16, 91)
    c["lens"] = torch.tensor([1 << 30, 32, -7], dtype=torch.int32, device="cuda")
    c["table"] = c["table"].contiguous()
    out, lse = _run(c)
    _check(c, out, lse, lens=[48, 32, 0])


def test_blocks_outside_the_cache_count_as_zeros():
    """Entries outside [0, num_blocks) read as zero keys and values and are flagged; hidden ones are not looked at."""
    c = _case([100, 64, 40], 4, 2, 64, "bf16", 16, 101, poison=False)
    table = c["table"].clone()
    nblk = c["k"].shape[0]
    table[0, 2], table[1, 0], table[2, 0] = nblk, -1, 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = capi.tv_decode_attn(c["q"], c["k"], c["v"], table, c["lens"], status=status)
    assert int(status.item()) == capi.TV_DEV_BAD_BLOCK
    z = dict(c, k=torch.cat((c["k"], torch.zeros_like(c["k"][:1]))), v=torch.cat((c["v"], torch.zeros_like(c["v"][:1]))))
    z["table"] = torch.where((table < 0) | (table >= nblk), nblk, table)
    want, _ = _run(z)
    assert torch.equal(out, want)
    status.zero_()
    capi.tv_decode_attn(c["q"][2:], c["k"], c["v"], table[2:], c["lens"][2:], window=8, status=status)
    assert int(status.item()) == 0


def test_workspace_serves_calls_of_every_size():
    """A zeroed workspace stays good from call to call; unflagged calls take any contents; results never change."""
    shapes = [([5000, 3], 8, 2, 128, "bf16", 16, 0), ([100] * 40, 16, 16, 64, "f32", 24, 7),
              ([2000], 40, 1, 64, "bf16", 16, 500), ([0, 0, 0], 8, 1, 256, "bf16", 16, 0)]
    ws = capi.alloc_workspace(16 << 20)
    cases = [(_case(*s[:6], 111), s[6]) for s in shapes]
    want = [_run(c, num_ctas=n) for c, n in cases]
    for _ in range(3):
        for (c, n), (o, l) in zip(cases, want):
            got, lse = _run(c, num_ctas=n, workspace=ws, flags=capi.TV_ATTN_WORKSPACE_ZEROED)
            assert torch.equal(got, o) and torch.equal(lse, l)
            assert int(ws[:16384].max()) == 0
    ws.random_(0, 256)
    for (c, n), (o, l) in zip(cases, want):
        got, lse = _run(c, num_ctas=n, workspace=ws)
        assert torch.equal(got, o) and torch.equal(lse, l)
        ws.random_(0, 256)


@pytest.mark.parametrize("Hq,Hkv,D,dtype,num_ctas", [(8, 1, 256, "bf16", 0), (16, 1, 128, "bf16", 0), (2, 2, 64, "f32", 0),
                                                      (4, 1, 128, "f32", 700), (12, 1, 64, "bf16", 25), (1, 1, 64, "f32", 65)])
def test_requests_in_many_pieces(Hq, Hkv, D, dtype, num_ctas):
    """Long requests cut into up to hundreds of pieces: the same bits each time, and the counters zero after each call."""
    c = _case([9000, 5, 20000], Hq, Hkv, D, dtype, 16, 2700 + D)
    nbytes = capi.tv_decode_attn_workspace_size(Hq, Hkv, D, DT[dtype], num_ctas)
    ws = capi.alloc_workspace(nbytes)
    runs = []
    for _ in range(3):
        runs.append(_run(c, workspace=ws, num_ctas=num_ctas, flags=capi.TV_ATTN_WORKSPACE_ZEROED))
        assert int(ws[:16384].max()) == 0
    _check(c, *runs[0])
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


def test_captured_calls_follow_their_inputs():
    """Graph replays with lengths and tables changed in place; two graphs share a workspace in turn."""
    lens = [900, 33, 0, 2000]
    c = _case(lens, 8, 2, 128, "bf16", 16, 121, poison=False)
    ws = capi.alloc_workspace(capi.tv_decode_attn_workspace_size(8, 2, 128, torch.bfloat16))
    out, out2 = torch.empty_like(c["q"]), torch.empty_like(c["q"])

    def call(o, **opt):
        capi.tv_decode_attn(c["q"], c["k"], c["v"], c["table"], c["lens"], out=o, workspace=ws,
                            flags=capi.TV_ATTN_WORKSPACE_ZEROED, **opt)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        call(out)
    with torch.cuda.graph(graphs[1]):
        call(out2, window=64, softcap=20.0)
    for new in (lens, [1, 900, 16, 0], [0, 0, 0, 0], [899, 32, 7, 1999]):
        width = c["table"].shape[1] * 16
        c["lens"].copy_(torch.tensor([min(n, width) for n in new], dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want, _ = _run(c)
        assert torch.equal(out, want)
        want, _ = _run(c, window=64, softcap=20.0)
        assert torch.equal(out2, want)


def test_calls_on_two_streams():
    cases = [_case([3000, 50], 8, 2, 128, "bf16", 16, 131), _case([700] * 9, 4, 4, 64, "f32", 16, 132)]
    want = [_run(c)[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [capi.alloc_workspace(16 << 20) for _ in cases]
    outs = [[torch.empty_like(w) for _ in range(10)] for w in want]
    torch.cuda.synchronize()
    for i in range(10):
        for c, s, ws, o in zip(cases, streams, spaces, outs):
            capi.tv_decode_attn(c["q"], c["k"], c["v"], c["table"], c["lens"], out=o[i], workspace=ws, stream=s,
                                flags=capi.TV_ATTN_WORKSPACE_ZEROED)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


def test_a_call_on_another_stream_allocates_there():
    """Outputs and workspace that the call makes itself belong to the stream it is given: many calls in a row, with the
    current stream busy reusing freed memory, give what one call gives."""
    c = _case([3000, 50, 700], 8, 2, 128, "bf16", 16, 133)
    want, _ = _run(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        outs.append(capi.tv_decode_attn(c["q"], c["k"], c["v"], c["table"], c["lens"], stream=s))
        torch.full((8 << 20,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_cache_offsets_past_32_bits():
    Hkv, bs, D = 8, 64, 128
    nblk = (1 << 31) // (Hkv * bs * D) + 8
    k = torch.zeros(nblk, Hkv, bs, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[-6:].normal_()
    v[-6:].normal_()
    table = torch.arange(nblk - 6, nblk, dtype=torch.int32, device="cuda").view(2, 3)
    c = {"q": torch.randn(2, 32, D, device="cuda").to(torch.bfloat16), "k": k, "v": v, "table": table,
         "lens": torch.tensor([192, 100], dtype=torch.int32, device="cuda")}
    out, lse = _run(c)
    small = dict(c, k=k[-6:], v=v[-6:], table=table - (nblk - 6))
    _check(small, out, lse)


def test_many_requests():
    """More requests than CTAs, most of them short or unused."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, size=1500)
    lens[::7] = 0
    lens[700] = 2500
    c = _case(lens, 4, 2, 64, "bf16", 16, 141)
    out, lse = _run(c)
    _check(c, out, lse)


def test_an_empty_batch():
    c = _case([4], 4, 2, 64, "bf16", 16, 151)
    out = capi.tv_decode_attn(c["q"][:0], c["k"], c["v"], c["table"][:0], c["lens"][:0])
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_is_the_one_node_tree(dtype):
    """A plain step -- append the token, attend -- is tree attention of a one-node tree whose root is the token."""
    w = W.Workload("case", 4, 8, 2, 128, dtype, ("fixed", 0), 16, (0.7, 0.15), 1, 1, 161)
    inp = W.attention_inputs(w, device="cuda", seq_lens=[0, 15, 16, 333], reserve=1)
    mask = torch.ones(4, 1, dtype=torch.int64, device="cuda")
    want = capi.tv_tree_attn_verify(inp["q"], inp["k_cache"], inp["v_cache"], inp["block_table"], inp["seq_lens"],
                                    inp["k_tree"], inp["v_tree"], mask)
    kc, vc = inp["k_cache"].clone(), inp["v_cache"].clone()
    _, lens = capi.tv_kv_append(inp["k_tree"][:, 0], inp["v_tree"][:, 0], kc, vc, inp["block_table"], inp["seq_lens"])
    got = capi.tv_decode_attn(inp["q"][:, 0], kc, vc, inp["block_table"], lens)
    tol = 2e-2 if dtype == "bf16" else 1e-4  # the tree kernels' own
    assert float((got.float() - want[:, 0].float()).abs().max()) <= tol


def test_binding_checks_every_argument():
    """Each wrong type, shape, layout and place is refused by name before anything is launched."""
    c = _case([40, 9], 4, 2, 64, "bf16", 16, 171)
    good = dict(q=c["q"], k_cache=c["k"], v_cache=c["v"], block_table=c["table"], seq_lens=c["lens"])
    bad = dict(q=c["q"][:1], k_cache=c["k"].half(), v_cache=c["v"][:, :1], block_table=c["table"][:1],
               seq_lens=c["lens"].long(), out=torch.empty(2, 4, 64, device="cuda"),
               lse=torch.empty(2, 3, device="cuda"), slopes=torch.ones(3, device="cuda"),
               workspace=torch.zeros(100, dtype=torch.int32, device="cuda"), status=torch.zeros(1, device="cuda"))
    for name, x in bad.items():
        with pytest.raises(ValueError, match=name):
            capi.tv_decode_attn(**{**good, name: x})
    with pytest.raises(ValueError, match="contiguous rows"):
        capi.tv_decode_attn(**{**good, "q": c["q"].transpose(1, 2).contiguous().transpose(1, 2)})
    with pytest.raises(ValueError, match="k_cache"):
        capi.tv_decode_attn(**{**good, "k_cache": c["k"].cpu()})
    with pytest.raises(capi.TVError, match="workspace"):
        capi.tv_decode_attn(**good, workspace=torch.zeros(100, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, "bf16"), (16, 1, 256, "bf16"), (8, 8, 64, "bf16"), (4, 1, 64, "f32"),
                                            (8, 1, 256, "f32"), (2, 2, 128, "f32")])
@pytest.mark.parametrize("num_ctas", [0, 1, 3, 40])
def test_no_score_above_minus_infinity(Hq, Hkv, D, dtype, num_ctas):
    """Requests whose scores are all -inf (a product past float32, keys of -inf) have no weight anywhere: a zero row with
    lse -inf, as without a visible key; requests whole, cut in few and many pieces, and shared by warps.  The others are
    as they were."""
    lens = [700, 5000, 1, 20, 16, 3, 300]
    c = _case(lens, Hq, Hkv, D, dtype, 16, 77)
    want, wlse = _run(c, num_ctas=num_ctas)
    gone = [1, 3, 5, 6]
    c["q"][gone] = 1e20
    table = c["table"].cpu().numpy()
    for b in gone:
        for i in range((lens[b] + 15) // 16):
            n = min(16, lens[b] - 16 * i)
            c["k"][table[b, i], :, :n] = -float("inf") if b == 6 else -1e20
    out, lse = _run(c, num_ctas=num_ctas)
    assert (out[gone] == 0).all() and (lse[gone] == -np.inf).all()
    rest = [0, 2, 4]
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], wlse[rest])


def test_the_largest_caps_and_biases():
    """A cap far above every score changes nothing; a bias near float32's largest value leaves the last key alone."""
    for dtype in ("f32", "bf16"):
        c = _case([300, 17, 1], 4, 2, 64, dtype, 16, 79)
        want, wlse = _run(c)
        for cap in (1e30, 1e37, 1e38, 2.3e38):
            out, lse = _run(c, softcap=cap)
            # the cap's tanh and its two factors: 8 roundings of scores within 2^4
            assert (lse - wlse).abs().max() <= 8 * 2.0 ** -24 * 16
            u = torch.finfo(DT[dtype]).eps
            assert ((out - want).float().abs() <= u * want.float().abs() + 16 * 2.0 ** -24 * 16 * 4).all()
        out, lse = _run(c, slopes=torch.full((4,), 3.2e38, device="cuda"))
        for b, L in enumerate([300, 17, 1]):
            blk, slot = int(c["table"][b, (L - 1) // 16]), (L - 1) % 16
            assert torch.equal(out[b], c["v"][blk, :, slot].repeat_interleave(2, 0)) and lse[b].isfinite().all()


def test_numbers_past_32_bits_are_refused():
    """None of them is taken modulo 2^32; negative ones are the library's to refuse, as before."""
    c = _case([40, 9], 4, 2, 64, "bf16", 16, 173)
    for name in ("window", "n_sink", "num_ctas", "flags"):
        with pytest.raises(capi.TVError):
            capi.tv_decode_attn(c["q"], c["k"], c["v"], c["table"], c["lens"], **{name: -1})
    for name in ("window", "n_sink", "num_ctas", "flags"):
        for x in (1 << 32, (1 << 32) + 5, 1 << 31, -(1 << 32)):
            with pytest.raises((ValueError, capi.TVError), match=name):
                capi.tv_decode_attn(c["q"], c["k"], c["v"], c["table"], c["lens"], **{name: x})


def test_a_request_in_hundreds_of_pieces():
    """More than 512 pieces of one request: joined in runs of 20, the same bits each time, counters left zero."""
    c = _case([20000, 7], 1, 1, 256, "f32", 16, 2800)
    ws = capi.alloc_workspace(capi.tv_decode_attn_workspace_size(1, 1, 256, torch.float32, 700))
    runs = []
    for _ in range(3):
        runs.append(_run(c, workspace=ws, num_ctas=700, flags=capi.TV_ATTN_WORKSPACE_ZEROED))
        assert int(ws[:16384].max()) == 0
    _check(c, *runs[0])
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, "bf16"), (16, 1, 256, "bf16"), (8, 8, 64, "bf16"), (4, 1, 64, "f32")])
@pytest.mark.parametrize("num_ctas", [0, 1, 40])
def test_nan_reaches_its_own_rows_only(Hq, Hkv, D, dtype, num_ctas):
    """A NaN among a request's keys, or as a bias, makes its rows NaN; an infinite bias leaves the last key alone."""
    lens = [700, 5000, 1, 20, 16, 300]
    c = _case(lens, Hq, Hkv, D, dtype, 16, 78)
    want, wlse = _run(c, num_ctas=num_ctas)
    table = c["table"].cpu().numpy()
    for b, t in ((1, 4000), (3, 19), (4, 0)):
        c["k"][table[b, t // 16], :, t % 16] = float("nan")
    out, lse = _run(c, num_ctas=num_ctas)
    assert out[[1, 3, 4]].isnan().all() and lse[[1, 3, 4]].isnan().all()
    rest = [0, 2, 5]
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], wlse[rest])
    slopes = torch.zeros(Hq, device="cuda")
    slopes[0], slopes[-1] = float("inf"), float("nan")
    out, lse = _run(c, slopes=slopes, num_ctas=num_ctas)
    for b in rest:
        L = lens[b]
        assert torch.equal(out[b, 0], c["v"][table[b, (L - 1) // 16], 0, (L - 1) % 16]) and lse[b, 0].isfinite()
        assert out[b, -1].isnan().all() and lse[b, -1].isnan()
