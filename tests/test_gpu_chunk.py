"""GPU parity of tv_chunk_attn (a chunk of new tokens per request over the
paged cache) against the same attention in float64, on both kernels."""

import math

import numpy as np
import pytest
import torch

from gpu_helpers import to_np
from oracle import attention as OA
from speculative_decoding_tree_attn_gb300 import capi
from speculative_decoding_tree_attn_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
KERNELS = {"simt": capi.TV_ATTN_SIMT, "tcgen05": capi.TV_ATTN_TCGEN05, "auto": capi.TV_ATTN_AUTO}


def _case(lens, counts, Hq, Hkv, D, dtype, bs, seed=1, pad=0, fused=False, window=0, n_sink=0, poison=True, alibi=False,
          gain=1.0, **kw):
    """Caches of which only the slots that some row sees hold numbers (else NaN), blocks without such a slot at table
    entries outside the cache."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[dtype]
    lens, counts = np.asarray(lens, dtype=np.int64), np.asarray(counts, dtype=np.int64)
    total = lens + counts
    table, nblk = W.block_table_for(total, bs, seed, spare_blocks=1)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    kc, vc = randn(nblk, Hkv, bs, D).to(dt), randn(nblk, Hkv, bs, D).to(dt)
    if poison:
        seen = np.zeros((nblk, bs), dtype=bool)
        for b in range(lens.size):
            t = np.arange(total[b]) if counts[b] else np.zeros(0, dtype=np.int64)
            if window:
                t = t[(t > lens[b] - window) | (t < n_sink)]
            seen[table[b, t // bs], t % bs] = True
            blocks = np.setdiff1d(np.arange(table.shape[1]), t // bs)
            table[b, blocks] = np.where(blocks % 2, -1, 2 ** 31 - 1)
        dark = torch.from_numpy(~seen).cuda()[:, None, :, None]
        kc, vc = kc.masked_fill(dark, float("nan")), vc.masked_fill(dark, float("nan"))
    T = int(counts.sum()) + pad
    q = (gain * randn(T, Hq + (3 if fused else 0), D)).to(dt)[:, :Hq]
    slopes = torch.pow(2.0, -8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32) / Hq) if alibi else None
    return dict(q=q, kc=kc, vc=vc, table=torch.from_numpy(table.astype(np.int32)).cuda(),
                lens=torch.from_numpy(total.astype(np.int32)).cuda(), counts=counts,
                cu=torch.from_numpy(np.concatenate(([0], np.cumsum(counts))).astype(np.int32)).cuda(),
                opt=dict(window=window, n_sink=n_sink, slopes=slopes, **kw))


def _run(c, flags=0, **kw):
    out = torch.full((c["q"].shape[0], c["q"].shape[1], c["q"].shape[2]), 7.0, device="cuda", dtype=c["q"].dtype)
    lse = torch.full(out.shape[:2], 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.tv_chunk_attn(c["q"], c["kc"], c["vc"], c["table"], c["lens"], out=out, lse=lse, flags=flags, status=status,
                       **{"cu_new": c["cu"], **c["opt"], **kw})
    torch.cuda.synchronize()
    return out, lse, int(status)


def _dense(c, rows_of=None):
    """Per request: (first row, out, lse, sum p |v|, scale of a score's rounding) in float64."""
    o = c["opt"]
    Hq, D = c["q"].shape[1:]
    Hkv, bs = c["kc"].shape[1:3]
    G, at = Hq // Hkv, 0
    scale = 1.0 / math.sqrt(D) if o.get("scale") is None else o["scale"]
    for b, n in enumerate(c["counts"].tolist()):
        first, at = at, at + n
        L = int(c["lens"][b])
        if n == 0 or (rows_of is not None and b not in rows_of):
            continue
        t = torch.arange(L, device="cuda")
        pos = torch.arange(L - n, L, device="cuda")
        seen = t[None] <= pos[:, None]
        if o["window"]:
            seen &= (t[None] > pos[:, None] - o["window"]) | (t[None] < o["n_sink"])
        used = seen.any(dim=0)
        blk = c["table"][b].long()[t // bs]
        blk = torch.where(used, blk, 0)
        k = torch.where(used[:, None, None], c["kc"][blk, :, t % bs].double(), 0.0)
        v = torch.where(used[:, None, None], c["vc"][blk, :, t % bs].double(), 0.0)
        q = c["q"][first:at].double().view(n, Hkv, G, D)
        s = torch.einsum("nhgd,thd->hgnt", q, k) * scale
        size = torch.einsum("nhgd,thd->hgnt", q.abs(), k.abs()) * abs(scale)
        if o.get("softcap"):
            s = o["softcap"] * torch.tanh(s / o["softcap"])
        far = (t[None] - pos[:, None]).double()
        if o["slopes"] is not None:
            bias = o["slopes"].double().view(Hkv, G, 1, 1) * far
            s, size = s + bias, size + bias.abs() / (D + 8)
        s = torch.where(seen, s, -math.inf)
        size = torch.where(seen, size, 0.0).amax(dim=-1)
        m = s.amax(dim=-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        w = torch.exp(s - m)
        z = w.sum(dim=-1, keepdim=True)
        w = w / torch.where(z == 0, 1.0, z)
        lay = lambda x: x.permute(2, 0, 1, *range(3, x.dim())).reshape(n, Hq, *x.shape[3:])
        yield (first, lay(torch.einsum("hgnt,thd->hgnd", w, v)), lay((m + torch.log(z))[..., 0]),
               lay(torch.einsum("hgnt,thd->hgnd", w, v.abs())), lay(size), L)


def _check(c, out, lse, tensor_core, rows_of=None):
    """A score: D products and their float32 sum, scale, cap (8 half steps of its size) and bias, in all D + 8 half steps
    of the products' magnitudes; lse moves by the largest of them.  A weight moves by e^that, its sum by as much
    again; the exponential is good to 2^-21, sums over the keys to a half step an addition of tile sums (at most
    L / 32 + 64).  The tcgen05 kernel rounds weights to bf16 (half step 2^-8 at most, the sum keeps them unrounded),
    and outputs are rounded once."""
    u = torch.finfo(c["q"].dtype).eps / 2
    for first, ro, rl, pv, size, L in _dense(c, rows_of):
        n = ro.shape[0]
        es = size * (ro.shape[2] + 8) * 2.0 ** -24
        sums = 2.0 ** -21 + (L / 32 + 64) * 2.0 ** -24
        got, gl = out[first:first + n].double(), lse[first:first + n].double()
        live = rl > -math.inf
        assert torch.equal(gl > -math.inf, live)
        assert not live.any() or bool(((gl - rl).abs() <= es + 2 * sums + rl.abs() * 2.0 ** -22)[live].all()), \
            float((gl - rl).abs()[live].max())
        bound = (2 * es + 2 * sums + (2.0 ** -8 if tensor_core else 0.0))[..., None] * pv
        bound = bound + u * (ro.abs() + bound) + 2.0 ** -120
        err = (got - ro).abs()
        assert bool((err <= bound).all()), (float(err.max()), float((err / bound).max()))


SHAPES = [
    # lens before, counts, Hq, Hkv, D, dtype, block
    ([0], [1], 1, 1, 64, "f32", 16),
    ([0], [1], 4, 1, 128, "bf16", 16),
    ([1001], [17], 32, 8, 128, "bf16", 16),
    ([0, 15, 16, 17, 100], [1, 1, 1, 1, 1], 8, 2, 128, "bf16", 16),
    ([0, 3, 0, 40, 7], [17, 0, 64, 1, 0], 4, 4, 256, "bf16", 24),
    ([5, 0, 31], [300, 129, 2], 5, 1, 64, "f32", 1),
    ([1, 2], [33, 1000], 6, 3, 64, "bf16", 8),
    ([64, 127, 128, 129], [127, 128, 129, 255], 8, 2, 128, "bf16", 64),
    ([2048, 0], [257, 1025], 16, 2, 128, "bf16", 128),
    ([700, 1], [65, 200], 20, 4, 64, "bf16", 32),
    ([33], [500], 16, 1, 256, "f32", 7),
    ([0, 200, 9], [200, 3, 77], 14, 2, 128, "bf16", 256),
    ([50, 400], [70, 90], 48, 1, 128, "bf16", 24),
    ([10, 77], [40, 5], 130, 1, 64, "bf16", 16),
    ([300], [20], 200, 1, 64, "f32", 16),
    ([0] * 40, list(range(40)), 2, 2, 128, "bf16", 48),
    ([5000], [3], 8, 1, 128, "bf16", 16),
]


@pytest.mark.parametrize("Hq,Hkv,D,dtype,bs,stride", [(4, 1, 256, "f32", 16, 1), (4, 1, 128, "f32", 16, 1), (4, 1, 64, "bf16", 12, 1),
                                                     (130, 1, 64, "bf16", 16, 1), (4, 1, 128, "bf16", 16, 0)])
def test_shapes_without_a_tcgen05_kernel(Hq, Hkv, D, dtype, bs, stride):
    """Refused by name, and computed by the other kernel (the last: one query row for every token)."""
    c = _case([20], [30], Hq, Hkv, D, dtype, bs)
    if not stride:
        c["q"] = c["q"][:1].expand(30, Hq, D)
    with pytest.raises(capi.TVError) as e:
        _run(c, capi.TV_ATTN_TCGEN05)
    assert e.value.code == -4 and "tcgen05" in str(e.value)
    out, lse, status = _run(c)
    assert status == 0
    _check(dict(c, q=c["q"].contiguous()), out, lse, False)


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(s[1])}of{max(s[0])}_{s[2]}_{s[3]}_{s[4]}_{s[5]}_{s[6]}")
def test_matches_float64(shape, kernel):
    c = _case(*shape, pad=3, fused=True)
    out, lse, status = _run(c, KERNELS[kernel])
    assert status == 0
    _check(c, out, lse, kernel == "auto" and shape[5] == "bf16")
    n = int(np.sum(shape[1]))
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()  # rows behind the last request


@pytest.mark.parametrize("G,Hkv,D,bs", [(32, 3, 128, 16), (64, 2, 64, 32), (96, 2, 128, 16), (128, 2, 128, 64), (32, 2, 256, 16),
                                        (96, 1, 64, 24), (128, 3, 256, 16)])
@pytest.mark.parametrize("ctas", [0, 3, 40])
def test_wide_groups_on_tcgen05(G, Hkv, D, bs, ctas):
    """Groups of a multiple of 32 query heads: outputs in boxes of 32 heads of one token; 1 to 4 tokens an M tile, the last
    units partly filled, cut by other grids."""
    c = _case([700, 0, 13, 4000], [37, 70, 1, 5], G * Hkv, Hkv, D, "bf16", bs, seed=G, pad=2, fused=True, window=900, n_sink=3)
    out, lse, status = _run(c, capi.TV_ATTN_TCGEN05, num_ctas=ctas)
    assert status == 0
    _check(c, out, lse, True)
    assert (out[113:] == 7.0).all() and (lse[113:] == 7.0).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_lengths_past_the_table_are_clamped(dtype, D):
    """A length of more positions than the block table has counts as the table's."""
    c = _case([100, 90, 5], [28, 38, 40], 4, 2, D, dtype, 16, poison=False)
    assert c["table"].shape[1] == 8
    want, wl, _ = _run(dict(c, lens=torch.tensor([128, 128, 45], dtype=torch.int32, device="cuda")))
    for past in (129, 4000, 2 ** 31 - 1):
        out, lse, status = _run(dict(c, lens=torch.tensor([past, 128, 45], dtype=torch.int32, device="cuda")))
        assert status == 0 and torch.equal(out, want) and torch.equal(lse, wl)
    _check(c, want, wl, dtype == "bf16")


MASKS = [
    dict(window=1), dict(window=16), dict(window=100, n_sink=4), dict(window=129, n_sink=200), dict(window=5000, n_sink=3),
    dict(window=2 ** 31 - 1, n_sink=2 ** 31 - 1), dict(softcap=5.0), dict(softcap=0.01), dict(softcap=1e30),
    dict(alibi=True), dict(window=64, n_sink=17, softcap=20.0, alibi=True), dict(scale=-0.3), dict(scale=0.0),
    dict(n_sink=9),
]


@pytest.mark.parametrize("kernel", ["simt", "auto"])
@pytest.mark.parametrize("dtype,D,bs", [("bf16", 128, 16), ("bf16", 64, 64), ("f32", 64, 24), ("bf16", 256, 16)])
@pytest.mark.parametrize("mask", MASKS, ids=lambda m: "_".join(f"{k}{v}" for k, v in m.items()))
def test_masks_caps_and_biases(mask, dtype, D, bs, kernel):
    c = _case([0, 500, 37, 1000], [300, 90, 1, 260], 8, 2, D, dtype, bs, seed=2, gain=3.0, **mask)
    out, lse, status = _run(c, KERNELS[kernel])
    assert status == 0
    _check(c, out, lse, kernel == "auto" and dtype == "bf16")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [88.0, 50.0, 30.0, 5.0, 0.5])
def test_caps_of_small_scores(cap, D):
    """Scores far below the cap: the tcgen05 kernel's are within 2^-21 of the cap, however small they are, so lse is too and a
    weight within twice that; the CUDA-core kernel's are within the bounds of _check, which go by the score."""
    c = _case([40, 600], [200, 70], 8, 2, D, "bf16", 16, seed=11, gain=0.05, softcap=cap)
    out, lse, status = _run(c, capi.TV_ATTN_TCGEN05)
    assert status == 0
    u = 2.0 ** -8
    for first, ro, rl, pv, size, L in _dense(c):
        n = ro.shape[0]
        es = size * (D + 8) * 2.0 ** -24 + cap * 2.0 ** -21
        sums = 2.0 ** -21 + (L / 32 + 64) * 2.0 ** -24
        assert ((lse[first:first + n].double() - rl).abs() <= es + 2 * sums + rl.abs() * 2.0 ** -22).all()
        bound = (2 * es + 2 * sums + u)[..., None] * pv
        assert ((out[first:first + n].double() - ro).abs() <= bound + u * (ro.abs() + bound)).all()
    out, lse, status = _run(c, capi.TV_ATTN_SIMT)
    assert status == 0
    _check(c, out, lse, False)


def test_the_oracle_agrees():
    c = _case([3, 20], [5, 9], 4, 2, 64, "f32", 16, window=8, n_sink=2, softcap=4.0, alibi=True, poison=False)
    out, lse, _ = _run(c)
    ro, rl = OA.chunk_attention(to_np(c["q"]), to_np(c["kc"]), to_np(c["vc"]), c["table"].cpu().numpy(), [8, 29], [5, 9],
                                softcap=4.0, window=8, n_sink=2, slopes=to_np(c["opt"]["slopes"]))
    assert np.abs(to_np(out) - ro).max() < 1e-5 and np.abs(to_np(lse) - rl).max() < 1e-5


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("f32", 64)])
def test_rows_that_see_nothing(dtype, D):
    """A chunk longer than its sequence: its first tokens sit below 0; a sequence of length 0 and below."""
    c = _case([0, 0, 0, 0], [40, 9, 300, 20], 4, 1, D, dtype, 16)
    c["lens"] = torch.tensor([10, 0, 290, -5], dtype=torch.int32, device="cuda")
    out, lse, status = _run(c)
    assert status == 0
    for first, n in ((0, 30), (40, 9), (49, 10), (349, 20)):
        assert (out[first:first + n] == 0).all() and (lse[first:first + n] == -math.inf).all()
    c2 = dict(c, q=torch.cat((c["q"][30:40], c["q"][59:349])).contiguous(), counts=np.array([10, 0, 290, 0]),
              cu=torch.tensor([0, 10, 10, 300, 300], dtype=torch.int32, device="cuda"))
    _check(c2, torch.cat((out[30:40], out[59:349])), torch.cat((lse[30:40], lse[59:349])), dtype == "bf16")


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_scores_of_minus_infinity(dtype, D):
    """Keys of -inf under positive queries: without weight among others, zero rows alone."""
    c = _case([0, 0], [150, 30], 4, 1, D, dtype, 16, poison=False)
    c["q"] = c["q"].abs() + 0.1
    kc = c["kc"].clone()
    bs = 16
    for b, ts in ((0, range(100)), (1, range(30))):
        for t in ts:
            kc[c["table"][b, t // bs].long(), :, t % bs] = -math.inf
    c["kc"] = kc
    out, lse, _ = _run(c)
    assert (out[:100] == 0).all() and (lse[:100] == -math.inf).all()
    assert (out[150:] == 0).all() and (lse[150:] == -math.inf).all()
    want = dict(c, kc=torch.where(kc == -math.inf, torch.zeros_like(kc), kc))
    assert torch.isfinite(out[100:150]).all() and torch.isfinite(lse[100:150]).all()
    for j in (100, 149):  # only keys 100.. count
        t = torch.arange(100, j + 1, device="cuda")
        k = want["kc"][c["table"][0].long()[t // bs], 0, t % bs].double()
        s = c["q"][j].double() @ k.T / math.sqrt(D)
        assert (torch.logsumexp(s, -1) - lse[j].double()).abs().max() < 1e-4


def test_bad_blocks_count_as_zeros():
    for dtype, D in (("bf16", 128), ("f32", 64)):
        c = _case([100], [50], 4, 1, D, dtype, 16, poison=False)
        table = c["table"].clone()
        zero = int(set(range(c["kc"].shape[0])).difference(table.flatten().tolist()).pop())
        c["kc"][zero], c["vc"][zero] = 0, 0
        for entry in (-1, c["kc"].shape[0], 2 ** 31 - 1, -2 ** 31):
            table[0, 3] = entry
            out, lse, status = _run(dict(c, table=table))
            assert status == capi.TV_DEV_BAD_BLOCK
            table[0, 3] = zero
            _check(dict(c, table=table), out, lse, dtype == "bf16")


def test_bad_offsets():
    for dtype, D in (("bf16", 128), ("f32", 64)):
        c = _case([100, 7, 30, 2], [50, 20, 40, 9], 4, 1, D, dtype, 16, poison=False)
        want, wl, _ = _run(c)
        for cu, rows in (([0, 50, 70, 200, 119], [(0, 70)]), ([-1, 50, 70, 110, 119], [(50, 119)]),
                         ([0, 50, 45, 110, 119], [(110, 119), (0, 45)]), ([0, 50, 70, 110, 2 ** 31 - 1], [(0, 110)])):
            out, lse, status = _run(c, cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"))
            assert status & capi.TV_DEV_BAD_OFFSETS
            for a, e in rows:
                assert torch.equal(out[a:e], want[a:e]) and torch.equal(lse[a:e], wl[a:e])
        good, gl, status = _run(c)
        assert status == 0 and torch.equal(good, want) and torch.equal(gl, wl)


def test_without_offsets():
    c = _case([100, 7, 30], [20, 20, 20], 4, 2, 128, "bf16", 16)
    out, lse, _ = _run(c)
    out2, lse2, _ = _run(c, cu_new=None)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,D,bs", [("bf16", 128, 16), ("bf16", 64, 16), ("f32", 64, 16), ("bf16", 256, 16)])
def test_a_chunk_of_one_is_the_one_token_call(dtype, D, bs):
    c = _case([100, 7, 3000], [1, 1, 1], 8, 2, D, dtype, bs, window=900, n_sink=5)
    out, lse, _ = _run(c)
    lse1 = torch.empty_like(lse)
    one = capi.tv_decode_attn(c["q"].contiguous(), c["kc"], c["vc"], c["table"], c["lens"], window=900, n_sink=5, lse=lse1)
    _check(c, one, lse1, dtype == "bf16")
    _check(c, out, lse, dtype == "bf16")


def test_chunks_in_turn_are_the_whole_prompt():
    """A prompt at once, or in pieces that follow one another, and the same rows either way but for rounding."""
    for dtype, D in (("bf16", 128), ("f32", 64)):
        c = _case([0], [600], 8, 2, D, dtype, 16)
        out, lse, _ = _run(c)
        at = 0
        for n in (1, 128, 200, 7, 264):
            piece = dict(c, q=c["q"][at:at + n], counts=np.array([n]), lens=torch.tensor([at + n], dtype=torch.int32).cuda(),
                         cu=torch.tensor([0, n], dtype=torch.int32).cuda())
            o, l, _ = _run(piece)
            _check(piece, o, l, dtype == "bf16")
            assert (l - lse[at:at + n]).abs().max() < 1e-4
            at += n


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 40, 152, 333, 4096])
def test_any_grid(ctas, D):
    c = _case([900, 0, 2000, 40], [100, 300, 5, 1], 8, 2, D, "bf16", 16, seed=4)
    out, lse, status = _run(c, num_ctas=ctas)
    assert status == 0
    _check(c, out, lse, True)


@pytest.mark.parametrize("G", [1, 3, 5, 6, 7, 12, 20, 43])
@pytest.mark.parametrize("D,window", [(128, 0), (64, 700), (256, 0)])
def test_any_group_cut_anywhere(G, D, window):
    """Steps of 256 down to 2 tokens a unit, most of them no power of two: the runs of many grids meet without a gap."""
    c = _case([900, 0, 2000, 40], [100, 300, 5, 1], 2 * G, 2, D, "bf16", 16, seed=G, window=window, n_sink=70)
    for ctas in (1, 13, 152, 1000):
        out, lse, status = _run(c, num_ctas=ctas)
        assert status == 0
        _check(c, out, lse, True)


@pytest.mark.parametrize("D,G,bs", [(128, 4, 16), (64, 4, 64), (128, 16, 8), (256, 4, 16)])
def test_long_runs_of_a_cta(D, G, bs):
    """Few CTAs: hundreds of tiles each, half of an M tile pair idle for whole requests, and then not."""
    rng = np.random.default_rng(D + G)
    c = _case(rng.integers(500, 4000, size=24), rng.choice([1, 3, 30, 40, 70, 200], size=24), 2 * G, 2, D, "bf16", bs, seed=9)
    for ctas in (1, 3):
        out, lse, status = _run(c, num_ctas=ctas)
        assert status == 0
        _check(c, out, lse, True)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_an_output_on_a_16_byte_boundary(D):
    c = _case([30, 200], [40, 70], 8, 2, D, "bf16", 16)
    want, _, _ = _run(c)
    room = torch.zeros(c["q"].numel() + 8, device="cuda", dtype=torch.bfloat16)
    out = room[8:].view(c["q"].shape)
    capi.tv_chunk_attn(c["q"], c["kc"], c["vc"], c["table"], c["lens"], cu_new=c["cu"], out=out)
    assert out.data_ptr() % 32 == 16 and torch.equal(out, want) and not room[:8].any()


def test_scores_that_rise_along_the_keys():
    """Every tile's scores lie far above the last one's: the reference of the weights has to follow."""
    c = _case([0], [300], 4, 1, 128, "bf16", 16, poison=False)
    c["q"] = torch.ones_like(c["q"])
    ramp = torch.arange(300, device="cuda", dtype=torch.float32) * 0.25
    t = torch.arange(300, device="cuda")
    c["kc"][c["table"][0].long()[t // 16], :, t % 16] = ramp[:, None, None].expand(300, 1, 128).bfloat16()
    out, lse, status = _run(c)
    assert status == 0
    _check(c, out, lse, True)


def test_same_bits_again_and_counters_left_zero():
    c = _case([4000, 10, 900], [60, 300, 3], 8, 2, 128, "bf16", 16, seed=5)
    ws = capi.alloc_workspace(capi.tv_chunk_attn_workspace_size(8, 2, 128, torch.bfloat16))
    first = None
    for _ in range(20):
        out, lse, status = _run(c, capi.TV_ATTN_WORKSPACE_ZEROED, workspace=ws)
        assert status == 0 and not ws[:16384].any()
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    ws.fill_(255)  # without the flag the call clears what it counts in
    out, lse, _ = _run(c, workspace=ws)
    assert torch.equal(out, first[0]) and not ws[:16384].any()


@pytest.mark.parametrize("D,dtype,bs", [(64, "f32", 16), (128, "f32", 64), (256, "f32", 16), (128, "bf16", 20)])
def test_keys_shared_by_ctas_without_tcgen05(D, dtype, bs):
    """Few rows over many keys: right, the same bits again, counters left zero, also behind a call on tcgen05."""
    c = _case([5000, 0, 700], [3, 1, 40], 8, 2, D, dtype, bs, seed=D)
    other = _case([2000, 10], [30, 300], 8, 2, 128, "bf16", 16, seed=5)
    ws = capi.alloc_workspace(max(capi.tv_chunk_attn_workspace_size(8, 2, x["q"].shape[2], x["q"].dtype)
                                  for x in (c, other)))
    want, want_lse, status = _run(c)
    assert status == 0
    _check(c, want, want_lse, False)
    want_other = _run(other)[0]
    for _ in range(10):
        out, lse, status = _run(c, capi.TV_ATTN_WORKSPACE_ZEROED, workspace=ws)
        assert status == 0 and not ws[:16384].any()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        out, _, status = _run(other, capi.TV_ATTN_WORKSPACE_ZEROED, workspace=ws)
        assert status == 0 and torch.equal(out, want_other) and not ws[:16384].any()


@pytest.mark.parametrize("dtype,D,bs", [("f32", 64, 16), ("bf16", 64, 12)])
def test_counters_are_cleared_by_calls_that_cut_nothing(dtype, D, bs):
    """A workspace of garbage, then a call without the flag whose rows are many enough to share no keys: the calls behind
    it, which cut their units, take the counters as zero."""
    big = _case([0] * 40, [500] * 40, 8, 2, D, dtype, bs, seed=3, poison=False)
    cut = [_case([5000, 700], [3, 40], 8, 2, 64, "f32", 16, seed=4), _case([4000, 900], [60, 3], 8, 2, 128, "bf16", 16, seed=5)]
    want = [_run(c)[0] for c in cut]
    ws = capi.alloc_workspace(max(capi.tv_chunk_attn_workspace_size(8, 2, d, t) for d, t in
                                  ((D, DT[dtype]), (64, torch.float32), (128, torch.bfloat16))))
    ws.fill_(255)
    out, _, status = _run(big, workspace=ws)
    assert status == 0 and not ws[:16384].any()
    assert torch.equal(out, _run(big)[0])
    for c, w in zip(cut, want):
        out, _, status = _run(c, capi.TV_ATTN_WORKSPACE_ZEROED, workspace=ws)
        assert status == 0 and torch.equal(out, w) and not ws[:16384].any()


def test_one_workspace_for_different_calls():
    ws = capi.alloc_workspace(capi.tv_chunk_attn_workspace_size(16, 2, 128, torch.bfloat16))
    for seed, shape in enumerate((([5000], [3], 8, 1, 128, "bf16", 16), ([0], [700], 16, 2, 128, "bf16", 16),
                                  ([10, 3000], [9, 20], 4, 1, 64, "bf16", 16), ([0], [30], 4, 1, 64, "f32", 16))):
        c = _case(*shape, seed=seed)
        out, lse, status = _run(c, capi.TV_ATTN_WORKSPACE_ZEROED, workspace=ws)
        assert status == 0
        _check(c, out, lse, shape[5] == "bf16")


def test_captured_replayed_with_other_lengths_and_on_another_stream():
    c = _case([900, 40], [100, 7], 8, 2, 128, "bf16", 16, seed=6, poison=False)
    ws = capi.alloc_workspace(capi.tv_chunk_attn_workspace_size(8, 2, 128, torch.bfloat16))
    out, lse = torch.zeros_like(c["q"]), torch.zeros(c["q"].shape[:2], device="cuda")
    call = lambda **kw: capi.tv_chunk_attn(c["q"], c["kc"], c["vc"], c["table"], c["lens"], cu_new=c["cu"], out=out, lse=lse,
                                           workspace=ws, flags=capi.TV_ATTN_WORKSPACE_ZEROED, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check(c, out, lse, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, counts in (([1000, 47], [100, 7]), ([400, 47], [80, 27]), ([107, 30], [107, 0])):
        c["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        c["counts"] = np.array(counts)
        c["cu"].copy_(torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        _check(c, out, lse, True)


def test_two_calls_at_once():
    """Two streams, a workspace each, many times over."""
    cs = [_case([900, 40, 2000], [100, 300, 70], 8, 2, D, "bf16", 16, seed=D) for D in (128, 64)]
    want = [_run(c)[0] for c in cs]
    ws = [capi.alloc_workspace(capi.tv_chunk_attn_workspace_size(8, 2, c["q"].shape[2], torch.bfloat16)) for c in cs]
    outs, streams = [torch.zeros_like(w) for w in want], [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(30):
        for c, w, o, st in zip(cs, ws, outs, streams):
            capi.tv_chunk_attn(c["q"], c["kc"], c["vc"], c["table"], c["lens"], cu_new=c["cu"], out=o, workspace=w,
                               flags=capi.TV_ATTN_WORKSPACE_ZEROED, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_offsets_past_32_bits():
    """Blocks at the far end of a cache of more than 2^31 elements."""
    D, bs, Hkv = 128, 16, 8
    nblk = (1 << 31) // (Hkv * bs * D) + 40
    kc = torch.zeros(nblk, Hkv, bs, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    small = _case([100], [60], 16, 8, D, "bf16", bs, seed=7, poison=False)
    far = nblk - 1 - small["table"]
    kc[far.long().flatten()], vc[far.long().flatten()] = small["kc"][small["table"].long().flatten()], \
        small["vc"][small["table"].long().flatten()]
    want, wl, _ = _run(small)
    for flag in (0, capi.TV_ATTN_SIMT):
        out, lse, status = _run(dict(small, kc=kc, vc=vc, table=far.contiguous()), flag)
        assert status == 0
        _check(small, out, lse, True)
    assert torch.equal(_run(dict(small, kc=kc, vc=vc, table=far.contiguous()))[0], want)


def test_many_requests_of_a_few_tokens():
    rng = np.random.default_rng(8)
    c = _case(rng.integers(0, 200, size=700), rng.integers(0, 5, size=700), 8, 2, 128, "bf16", 16, seed=8)
    out, lse, status = _run(c)
    assert status == 0
    _check(c, out, lse, True)


def test_empty_batches():
    c = _case([5], [3], 4, 1, 128, "bf16", 16)
    out = capi.tv_chunk_attn(c["q"][:0], c["kc"], c["vc"], c["table"], c["lens"],
                             cu_new=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 128)
    capi.tv_chunk_attn(c["q"][:0], c["kc"], c["vc"], c["table"][:0], c["lens"][:0])


def test_a_prompt_to_its_first_token():
    """Norm and append, chunk attention, sampling, then the next token's step: against the same in float64."""
    from oracle import kvcache as OK
    from oracle import sampling as OS

    B, Hq, Hkv, D, bs, V = 3, 8, 2, 128, 16, 2000
    counts = np.array([37, 130, 1])
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    table, blocks = W.block_table_for(counts + 1, bs, 3)
    for dtype in (torch.float32, torch.bfloat16):
        kc, vc = (torch.full((blocks, Hkv, bs, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        rows, qw, kw = randn(168, Hq + 2 * Hkv, D).to(dtype), (1 + 0.1 * randn(D)).to(dtype), (1 + 0.1 * randn(D)).to(dtype)
        cs, tbl = capi.tv_rope_table(200, D), torch.from_numpy(table).cuda()
        cu = torch.tensor([0, 37, 167, 168], dtype=torch.int32, device="cuda")
        q, lens = capi.tv_kv_append_norm(rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], kc, vc, tbl, torch.zeros_like(cu[:B]),
                                         k_weight=kw, q=rows[:, :Hq], q_weight=qw, cos_sin=cs, cu_new=cu)
        out = capi.tv_chunk_attn(q, kc, vc, tbl, lens, cu_new=cu)
        head = randn(Hq * D, V) * 0.02
        logits = out[(cu[1:] - 1).long()].view(B, -1).float() @ head
        u, p = torch.tensor([0.2, 0.5, 0.8], device="cuda"), torch.full((B,), 0.9, device="cuda")
        tokens = capi.tv_token_sample(logits, u, top_p=p)
        lp = capi.tv_token_logprobs(logits[:, None], tokens[:, None])[0]
        step = randn(B, Hq + 2 * Hkv, D).to(dtype)
        q1, lens1 = capi.tv_kv_append_norm(step[:, Hq:Hq + Hkv], step[:, Hq + Hkv:], kc, vc, tbl, lens, k_weight=kw,
                                           q=step[:, :Hq], q_weight=qw, cos_sin=cs)
        out1 = capi.tv_decode_attn(q1, kc, vc, tbl, lens1)

        zero, r, s = np.zeros((blocks, Hkv, bs, D)), to_np(rows), to_np(step)
        args = dict(q_weight=to_np(qw), k_weight=to_np(kw), eps=1e-6, table=to_np(cs))
        okc, ovc, ol, oq = OK.append_normed(zero, zero, table, np.zeros(B, dtype=int), r[:, Hq:Hq + Hkv],
                                            r[:, Hq + Hkv:], counts, q=r[:, :Hq], **args)
        ref, _ = OA.chunk_attention(oq, okc, ovc, table, ol, counts)
        tol = 1e-4 if dtype == torch.float32 else 2e-2
        assert np.abs(to_np(out) - ref).max() < tol
        want, _ = OS.token_sample(to_np(logits), to_np(u), top_p=to_np(p))
        np.testing.assert_array_equal(tokens.cpu().numpy(), want)
        okc, ovc, ol, oq = OK.append_normed(okc, ovc, table, ol, s[:, Hq:Hq + Hkv], s[:, Hq + Hkv:], np.ones(B, dtype=int),
                                            q=s[:, :Hq], **args)
        ref, _ = OA.decode_attention(oq, okc, ovc, table, ol)
        assert np.abs(to_np(out1) - ref).max() < tol
        assert np.array_equal(lens1.cpu().numpy(), counts + 1) and (lp <= 0).all()
