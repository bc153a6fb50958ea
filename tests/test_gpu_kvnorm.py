"""GPU parity of tv_kv_append_norm (new tokens' K/V into the paged cache, keys
and queries normalised per head and rotated on the way) against the float64
oracle and, without the norm, bit for bit against tv_kv_append."""

import numpy as np
import pytest
import torch

from gpu_helpers import to_np
from oracle import kvcache as OK
from speculative_decoding_tree_attn_gb300 import capi
from speculative_decoding_tree_attn_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def _case(lens, counts, Hq, Hkv, D, dtype, bs, seed, rot=None, pad=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[dtype]
    lens, counts = np.asarray(lens, dtype=np.int32), np.asarray(counts, dtype=np.int32)
    table, nblk = W.block_table_for(lens + counts, bs, seed, spare_blocks=2)
    T = int(counts.sum()) + pad
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    c = {"k_cache": randn(nblk, Hkv, bs, D).to(dt), "v_cache": randn(nblk, Hkv, bs, D).to(dt),
         "table": torch.from_numpy(table).cuda(), "lens": torch.from_numpy(lens).cuda(), "counts": counts,
         "cu": torch.from_numpy(np.concatenate(([0], np.cumsum(counts))).astype(np.int32)).cuda()}
    rows = (scale * randn(T, Hq + 2 * Hkv, D)).to(dt)
    c["q"], c["k"], c["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    c["qw"], c["kw"] = (1 + 0.3 * randn(D)).to(dt), (1 + 0.3 * randn(D)).to(dt)
    c["cs"] = None if rot == 0 else capi.tv_rope_table(int((lens + counts).max()) + 1, rot or D)
    return c


def _append(c, pairs=False, norm=(True, True), **kw):
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    q, lens = capi.tv_kv_append_norm(c["k"], c["v"], kc, vc, c["table"], c["lens"], k_weight=c["kw"] if norm[1] else None,
                                     q=c["q"], q_weight=c["qw"] if norm[0] else None, eps=EPS, cos_sin=c["cs"],
                                     interleaved=pairs, **{"cu_new": c["cu"], **kw})
    torch.cuda.synchronize()
    return kc, vc, lens, q


def _held(got, want, size, dt):
    """One rounding to the type, and float32's: the sum of D <= 256 squares goes through at most 21 additions and a
    product (22 half steps), of which the root takes half; eps, root and division are a half step each, the two
    products another, so a normalised element is off by 16 * 2^-24 of itself at most; a rotation's product and sum
    by 2 * 2^-24 of |x1| + |x2| <= 2 size, which carry the 16 each."""
    u = torch.finfo(dt).eps / 2
    err = np.abs(to_np(got).astype(np.float64) - want)
    assert (err <= u * np.abs(want) * (1 + u) + 2 * 18 * 2.0 ** -24 * size * (1 + u)).all(), float(err.max())


def _check(c, kc, vc, lens, q, pairs=False, norm=(True, True)):
    okc, ovc, olens, oq = OK.append_normed(to_np(c["k_cache"]), to_np(c["v_cache"]), c["table"].cpu().numpy(),
                                           c["lens"].cpu().numpy(), to_np(c["k"]), to_np(c["v"]), c["counts"],
                                           q=to_np(c["q"]), q_weight=to_np(c["qw"]) if norm[0] else None,
                                           k_weight=to_np(c["kw"]) if norm[1] else None, eps=EPS,
                                           table=None if c["cs"] is None else to_np(c["cs"]), interleaved=pairs)
    dt, n = c["k_cache"].dtype, int(c["counts"].sum())
    np.testing.assert_array_equal(lens.cpu().numpy(), olens)
    np.testing.assert_array_equal(to_np(vc), ovc)
    _held(kc, okc, np.abs(okc).max(axis=-1, keepdims=True) * np.sqrt(2), dt)
    _held(q[:n], oq[:n], np.abs(oq[:n]).max(axis=-1, keepdims=True) * np.sqrt(2), dt)


@pytest.mark.parametrize("lens,counts,Hq,Hkv,D,dtype,bs,rot,pairs", [
    ([0], [1], 1, 1, 64, "f32", 16, 64, False),
    ([37], [1], 32, 8, 128, "bf16", 16, 128, False),
    ([0, 15, 16, 17, 100], [1, 1, 1, 1, 1], 8, 2, 128, "bf16", 16, 64, True),
    ([0, 3, 0, 40, 7], [17, 0, 64, 1, 0], 4, 4, 256, "bf16", 24, 48, False),
    ([5, 0, 31], [300, 129, 2], 5, 1, 16, "f32", 1, 16, True),
    ([1, 2], [33, 1000], 3, 3, 32, "bf16", 7, 16, False),
    ([0] * 70, list(range(70)), 6, 2, 64, "f32", 64, 48, True),
    ([2048], [2049], 64, 8, 128, "bf16", 64, 0, False),
    ([9, 1], [5, 3], 7, 1, 256, "f32", 5, 256, True),
])
def test_matches_the_oracle(lens, counts, Hq, Hkv, D, dtype, bs, rot, pairs):
    c = _case(lens, counts, Hq, Hkv, D, dtype, bs, 500 + D + bs, rot=rot, pad=3)
    q_out = torch.full((c["q"].shape[0], Hq, D), 7.0, device="cuda", dtype=DT[dtype])
    kc, vc, got, q = _append(c, pairs, q_out=q_out)
    _check(c, kc, vc, got, q, pairs)
    assert (q[int(np.sum(counts)):] == 7.0).all()  # rows behind the last request


@pytest.mark.parametrize("norm", [(True, False), (False, True)])
def test_one_of_the_two_normalised(norm):
    c = _case([3, 60], [40, 7], 8, 2, 128, "bf16", 16, 3)
    _check(c, *_append(c, norm=norm), norm=norm)


@pytest.mark.parametrize("dtype,D,T", [("f32", 64, 30), ("bf16", 128, 30), ("bf16", 64, 9000)])
def test_without_norm_the_bits_of_kv_append(dtype, D, T):
    c = _case([7, 100, 0], [T, T, T], 2, 1, D, dtype, 16, 9)
    kc, vc, lens, q = _append(c, norm=(False, False))
    kc2, vc2 = c["k_cache"].clone(), c["v_cache"].clone()
    q2, lens2 = capi.tv_kv_append(c["k"], c["v"], kc2, vc2, c["table"], c["lens"], cos_sin=c["cs"], q=c["q"], cu_new=c["cu"])
    for a, b in ((kc, kc2), (vc, vc2), (lens, lens2), (q, q2)):
        assert torch.equal(a, b)


def test_without_norm_and_rotation_the_bits_of_every_value():
    """All 65536 bf16 values as queries, keys and values: what is neither normalised nor rotated keeps its bits, as in
    tv_kv_append, but for the NaNs of queries and keys, which become one."""
    c = _case([3], [1024], 2, 1, 64, "bf16", 16, 14, rot=0)
    as_bits = lambda x: x.contiguous().view(torch.int16)
    one_nan = lambda x: torch.where(torch.isnan(x), torch.full_like(as_bits(x), 0x7fff), as_bits(x))
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(1024, 1, 64)
    rows = bits.expand(1024, 4, 64).contiguous().view(torch.bfloat16)
    c["q"], c["k"], c["v"] = rows[:, :2], rows[:, 2:3], rows[:, 3:]
    kc, vc, lens, q = _append(c, norm=(False, False))
    kc2, vc2 = c["k_cache"].clone(), c["v_cache"].clone()
    capi.tv_kv_append(c["k"], c["v"], kc2, vc2, c["table"], c["lens"], cu_new=c["cu"])
    assert torch.equal(as_bits(kc), one_nan(kc2)) and torch.equal(as_bits(vc), as_bits(vc2))
    assert torch.equal(as_bits(q), one_nan(c["q"]))
    c["cs"] = capi.tv_rope_table(1028, 32)  # the second half of a head is not rotated
    kc, vc, lens, q = _append(c, norm=(False, False))
    assert torch.equal(as_bits(q[..., 32:]), one_nan(c["q"][..., 32:]))


def test_rows_of_zeros_and_of_large_and_small_values():
    c = _case([0], [4], 2, 2, 64, "f32", 16, 12)
    rows = torch.empty(4, 6, 64, device="cuda").normal_()
    rows *= torch.tensor([0.0, 1e-18, 1.0, 1e18], device="cuda").view(4, 1, 1)
    c["q"], c["k"], c["v"] = rows[:, :2], rows[:, 2:4], rows[:, 4:]
    kc, vc, lens, q = _append(c)
    _check(c, kc, vc, lens, q)
    assert (q[0] == 0).all()


def test_queries_in_place_and_without_offsets():
    c = _case([9, 50], [6, 6], 4, 1, 64, "bf16", 16, 11, rot=32)
    kc, vc, lens, q = _append(c, pairs=True)
    q_in = c["q"].clone()
    kc2, vc2, lens2, q2 = _append(dict(c, q=q_in), pairs=True, q_out=q_in, cu_new=None)
    assert q2.data_ptr() == q_in.data_ptr()
    for a, b in ((kc, kc2), (vc, vc2), (lens, lens2), (q, q2)):
        assert torch.equal(a, b)


def test_bad_blocks_positions_and_offsets():
    c = _case([0, 10, 3], [20, 5, 4], 2, 1, 64, "bf16", 8, 21)
    table = c["table"].clone()
    table[0, 1] = 10 ** 6  # tokens 8 .. 15 of the first request
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc, lens, q = _append(dict(c, table=table), status=status)
    assert int(status) == capi.TV_DEV_OUT_OVERFLOW and lens.tolist() == [8, 15, 7]
    good = _append(c)
    assert torch.equal(q, good[3])
    hit = table[0, 1] != c["table"][0, 1]
    assert hit and torch.equal(kc[c["table"][0, 1]], c["k_cache"][c["table"][0, 1]])
    status.zero_()
    _, _, lens, _ = _append(dict(c, cs=c["cs"][:12].contiguous()), status=status)
    assert int(status) == capi.TV_DEV_BAD_POSITION and lens.tolist() == [12, 12, 7]
    status.zero_()
    cu = torch.tensor([0, 20, 19, 29], dtype=torch.int32, device="cuda")
    _, _, lens, _ = _append(c, cu_new=cu, status=status)
    assert int(status) & capi.TV_DEV_BAD_OFFSETS and lens.tolist()[1] == 10


def test_captured_and_on_another_stream():
    c = _case([0, 31], [40, 9], 4, 2, 128, "bf16", 16, 31)
    want = _append(c)
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    q_out, new = torch.zeros_like(want[3]), torch.zeros_like(c["lens"])
    call = lambda **kw: capi.tv_kv_append_norm(c["k"], c["v"], kc, vc, c["table"], c["lens"], k_weight=c["kw"], q=c["q"],
                                               q_weight=c["qw"], q_out=q_out, eps=EPS, cos_sin=c["cs"], cu_new=c["cu"],
                                               new_seq_lens=new, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((kc, vc, new, q_out), want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    kc.copy_(c["k_cache"]), vc.copy_(c["v_cache"]), q_out.zero_(), new.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((kc, vc, new, q_out), want):
        assert torch.equal(a, b)
