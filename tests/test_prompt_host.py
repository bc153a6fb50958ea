"""Checks of the prompt operators (append with norms, chunk attention,
sampling) that need no GPU: argument errors are reported before anything is
launched, and the oracle's definitions agree with independent ones."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import kvcache as OK
from oracle import sampling as OS
from speculative_decoding_tree_attn_gb300 import build as B
from speculative_decoding_tree_attn_gb300 import capi

FAKE = ctypes.c_void_p(4096)  # stands for a device buffer; never touched


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(capi.LIB_PATH):
        B.build()
    return capi.lib()


def _call(name, args, **change):
    """Status of the entry point with the named arguments changed."""
    return getattr(capi.lib(), name)(*{**args, **change}.values())


NORM = dict(q=FAKE, q_stride=256, q_weight=FAKE, q_out=FAKE, q_out_stride=256, Hq=4, k_new=FAKE, k_stride=64, k_weight=FAKE,
            v_new=FAKE, v_stride=64, eps=1e-6, cu_new=None, T=6, k_cache=FAKE, v_cache=FAKE, num_blocks=9, block_size=16,
            table=FAKE, max_blocks=4, seq_lens=FAKE, new_lens=ctypes.c_void_p(8192), cos_sin=FAKE, max_pos=100, rot_dim=64,
            interleaved=0, B=3, Hkv=1, head_dim=64, dtype=1, status=None, stream=None)


@pytest.mark.parametrize("change,code,text", [
    (dict(B=-1), -1, b"bad sizes"), (dict(T=-1), -1, b"bad sizes"), (dict(Hkv=0), -1, b"bad sizes"),
    (dict(Hq=0), -1, b"bad sizes"), (dict(max_pos=0), -1, b"bad sizes"), (dict(num_blocks=0), -1, b"bad sizes"),
    (dict(dtype=2), -4, b"dtype"), (dict(head_dim=48), -4, b"head_dim 48"), (dict(T=7), -1, b"multiple of B"),
    (dict(k_cache=None), -1, b"null"), (dict(v_new=None), -1, b"null"), (dict(seq_lens=None), -1, b"null"),
    (dict(q_out=None), -1, b"q_out"), (dict(q=None), -1, b"q_weight without q"),
    (dict(new_lens=FAKE), -1, b"alias"), (dict(new_lens=ctypes.c_void_p(4104)), -1, b"overlap"),
    (dict(k_stride=-64), -1, b"stride"), (dict(q_out_stride=128), -1, b"stride"), (dict(k_stride=65), -1, b"16 bytes"),
    (dict(k_new=ctypes.c_void_p(4098)), -1, b"16 bytes"), (dict(k_weight=ctypes.c_void_p(4104)), -1, b"16-byte"),
    (dict(q_weight=ctypes.c_void_p(4098)), -1, b"16-byte"),
    (dict(eps=-1e-6), -1, b"eps"), (dict(eps=float("nan")), -1, b"eps"), (dict(eps=float("inf")), -1, b"eps"),
    (dict(rot_dim=0), -1, b"rot_dim"), (dict(rot_dim=8), -1, b"rot_dim"), (dict(rot_dim=40), -1, b"rot_dim"),
    (dict(rot_dim=80), -1, b"rot_dim"), (dict(rot_dim=-16), -1, b"rot_dim"), (dict(interleaved=2), -1, b"interleaved"),
])
def test_append_norm_refuses_on_the_host(change, code, text):
    assert _call("tv_kv_append_norm", NORM, **change) == code
    assert text in capi.lib().tv_last_error() and b"tv_kv_append_norm" in capi.lib().tv_last_error()


def test_append_norm_of_an_empty_batch_does_nothing():
    assert _call("tv_kv_append_norm", NORM, B=0, T=0) == 0


CHUNK = dict(q=FAKE, q_stride=256, k_cache=FAKE, v_cache=FAKE, num_blocks=9, block_size=16, table=FAKE, max_blocks=4,
             seq_lens=FAKE, cu_new=FAKE, T=7, B=3, Hq=4, Hkv=2, head_dim=64, dtype=1, scale=0.125, softcap=0.0, window=0,
             n_sink=0, slopes=None, out=FAKE, lse=None, workspace=FAKE, workspace_bytes=64 << 20, num_ctas=8, flags=0,
             status=None, stream=None)


@pytest.mark.parametrize("change,code,text", [
    (dict(B=-1), -1, b"bad sizes"), (dict(T=-1), -1, b"bad sizes"), (dict(Hq=5), -1, b"bad sizes"),
    (dict(Hkv=0), -1, b"bad sizes"), (dict(window=-1), -1, b"bad sizes"), (dict(n_sink=-1), -1, b"bad sizes"),
    (dict(block_size=0), -1, b"bad sizes"), (dict(max_blocks=0), -1, b"bad sizes"), (dict(num_ctas=4097), -1, b"bad sizes"),
    (dict(num_ctas=-1), -1, b"bad sizes"), (dict(dtype=7), -4, b"dtype"), (dict(head_dim=32), -4, b"head_dim 32"),
    (dict(cu_new=None), -1, b"multiple of B"), (dict(Hq=70000, Hkv=70000), -4, b"65535"),
    (dict(softcap=-1.0), -1, b"softcap"), (dict(softcap=float("nan")), -1, b"softcap"), (dict(softcap=3e38), -1, b"softcap"),
    (dict(scale=float("inf")), -1, b"scale"), (dict(scale=3e38), -1, b"scale"), (dict(flags=3), -1, b"unknown flags"),
    (dict(flags=4), -1, b"unknown flags"), (dict(flags=64), -1, b"unknown flags"),
    (dict(q=None), -1, b"null"), (dict(out=None), -1, b"null"), (dict(table=None), -1, b"null"),
    (dict(seq_lens=None), -1, b"null"), (dict(q_stride=-256), -1, b"16 bytes"), (dict(q_stride=257), -1, b"16 bytes"),
    (dict(k_cache=ctypes.c_void_p(4104)), -1, b"16 bytes"), (dict(workspace=None), -5, b"workspace"),
    (dict(workspace_bytes=100), -5, b"workspace"), (dict(workspace=ctypes.c_void_p(4096 + 128)), -5, b"workspace"),
])
def test_chunk_refuses_on_the_host(change, code, text):
    assert _call("tv_chunk_attn", CHUNK, **change) == code
    assert text in capi.lib().tv_last_error()


def test_chunk_refuses_groups_past_its_grid():
    for change in (dict(Hq=1 << 22, Hkv=1), dict(Hq=65535 * 32 + 1, Hkv=1), dict(Hq=3 << 21, Hkv=2)):
        assert _call("tv_chunk_attn", CHUNK, q_stride=1 << 29, **change) == -4
        assert b"query heads per KV head" in capi.lib().tv_last_error()
    with pytest.raises(capi.TVError, match="query heads"):
        capi.tv_chunk_attn_workspace_size(1 << 22, 1, 64, torch.float32)


def test_chunk_of_nothing():
    assert _call("tv_chunk_attn", CHUNK, B=0) == 0
    assert _call("tv_chunk_attn", CHUNK, T=0) == 0


def test_chunk_workspace_size():
    n = [capi.tv_chunk_attn_workspace_size(8, 2, 128, torch.bfloat16, num_ctas=k) for k in (1, 152, 160)]
    assert n == sorted(n) and n[2] <= 64 << 20
    with pytest.raises(capi.TVError):
        capi.tv_chunk_attn_workspace_size(9, 2, 128, torch.bfloat16, num_ctas=1)


@pytest.mark.parametrize("name", ["window", "n_sink", "num_ctas", "flags"])
@pytest.mark.parametrize("x", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1])
def test_binding_refuses_numbers_past_32_bits(name, x):
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    cache, q = torch.zeros(3, 1, 16, 64), torch.zeros(2, 4, 64)
    with pytest.raises(ValueError, match=name + f" {x}"):
        capi.tv_chunk_attn(q, cache, cache, table, lens, **{name: x})


SAMPLE = dict(logits=FAKE, R=3, V=100, dtype=0, temperature=None, top_k=None, top_p=None, min_p=None, u=FAKE, tokens=FAKE,
              probs=None, status=None, stream=None)


@pytest.mark.parametrize("change,code,text", [
    (dict(R=-1), -1, b"bad sizes"), (dict(V=0), -1, b"bad sizes"), (dict(dtype=3), -4, b"dtype"),
    (dict(V=(1 << 20) + 1), -4, b"exceeds"), (dict(R=1 << 28), -4, b"2^28"), (dict(logits=None), -1, b"null"),
    (dict(u=None), -1, b"null"), (dict(tokens=None), -1, b"null"), (dict(logits=ctypes.c_void_p(4100)), -1, b"16-byte"),
    (dict(probs=ctypes.c_void_p(4104)), -1, b"16-byte"),
])
def test_sample_refuses_on_the_host(change, code, text):
    assert _call("tv_token_sample", SAMPLE, **change) == code
    assert text in capi.lib().tv_last_error()


def test_sample_of_nothing():
    assert _call("tv_token_sample", SAMPLE, R=0) == 0


def _weight_mantissa(x, m, temperature):
    """The arithmetic of the sampling kernel's weights, float32 operation by operation: w as (mantissa, s), w = mantissa
    2^(-43 - s).  A fused product and sum goes through float64, which holds the product exactly."""
    f = np.float32
    fma = lambda a, b, c: (np.float64(a) * np.float64(b) + np.float64(c)).astype(f)
    c = 1.4426950408889634074 / float(f(temperature))
    c1 = f(c)
    c2 = f(c - float(c1))
    dh = x - m
    back = dh - x
    dl = (x - (dh - back)) - (m + back)
    yh = dh * c1
    yl = fma(dh, c1, -yh) + fma(dh, c2, dl * c1)
    n = np.rint(yh * f(64))
    rh = fma(n, f(-2.0 ** -6), yh)
    hi, lo = f(0.693147182464599609375), f(-1.904654323148236e-09)
    th = rh * hi
    tl = fma(rh, hi, -th) + fma(rh, lo, yl * hi)
    t = th + tl
    q = t * t * fma(t, fma(t, fma(t, f(1 / 120), f(1 / 24)), f(1 / 6)), f(0.5))
    e = np.rint(th * f(2.0 ** 38)).astype(np.int64) + np.rint((tl + q) * f(2.0 ** 38)).astype(np.int64)
    powers = np.array([round(np.exp2(np.longdouble(j) / 64) * 2 ** 43) for j in range(64)], dtype=np.int64)
    ni = n.astype(np.int64)
    p = powers[ni & 63]
    return p + ((p >> 12) * e >> 26), -(ni >> 6), powers


def test_sampling_weights_bound():
    """A weight is good to 2^-36 of itself.  In units of 2^-39: q, below 2^-16.05, takes five float32 roundings (2.41) and
    its sum with tl a sixth (0.25); the two roundings to units of 2^-38 are one each (2); p >> 12 cuts 2^-31 of a factor of
    |e^t - 1| < 2^-7.5 (1.39); what tl gathers is 0.9 for weights down to 2^-126; the table and the last cut 0.1; all of it
    over e^-|t|, 7.1.  The table is the one in the source."""
    assert re.sub(r"\s", "", ",".join(f"{v}ull" for v in _weight_mantissa(np.zeros(1, np.float32), np.float32(0), 1.0)[2])) in \
        re.sub(r"\s", "", open(os.path.join(B.CSRC, "sample.cu")).read())
    rng = np.random.default_rng(5)
    worst = 0.0
    for temperature in (1.0, 0.6, 1.2, 1e-3, 0.013, 50.0, 1e9, 2.0 ** -30):
        for most in (0.02, 1.0, 20.0, 44.0, 126.0):  # log2 w down to
            for top in (0.0, 9.7, -3.3, 180.25):
                m = np.float32(top * temperature)
                t = float(np.float32(temperature))
                x = (m - rng.uniform(0.0, most * np.log(2.0) * t, size=20000)).astype(np.float32)
                x = np.concatenate((x, [m])).astype(np.float32)
                exact = (x.astype(np.longdouble) - np.longdouble(m)) / np.longdouble(t)
                with np.errstate(under="ignore"):
                    got, s, _ = _weight_mantissa(x, m, temperature)
                live = exact / np.log(np.longdouble(2)) > -126
                w = got.astype(np.longdouble) * np.exp2(np.longdouble(-43) - s)
                worst = max(worst, float((np.abs(w / np.exp(exact) - 1))[live].max()))
                assert w[-1] == 1
                assert ((got >= 2.0 ** 42.99) & (got < 2.0 ** 43.993)).all()
    assert 2.0 ** -39 < worst <= 2.0 ** -36, worst * 2.0 ** 39


def test_binding_names_what_it_refuses():
    t, lens, table = torch.zeros(2, 1, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    cache = torch.zeros(3, 1, 16, 64)
    for call in (lambda: capi.tv_kv_append_norm(t, t, cache, cache, table, lens),
                 lambda: capi.tv_chunk_attn(t, cache, cache, table, lens),
                 lambda: capi.tv_chunk_attn(t, cache, cache, table, [0, 0]),
                 lambda: capi.tv_token_sample(torch.zeros(2, 10), torch.zeros(2)),
                 lambda: capi.tv_token_sample(None, torch.zeros(2))):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()


def test_norm_oracle_against_torch():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((3, 2, 32)), rng.standard_normal(32)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (32,), torch.from_numpy(w), eps=1e-3).numpy()
    np.testing.assert_allclose(OK.norm_rows(x, w, 1e-3), want, atol=1e-14)


def test_rotation_oracle():
    """Halves over the whole head: the rotation that the tree uses.  Pairs: the same after a shuffle.  Part of the head:
    the rest as it was."""
    rng = np.random.default_rng(2)
    x, pos = rng.standard_normal((5, 2, 32)), np.array([0, 1, 7, 100, 5000])
    ang = pos[:, None] * 10000.0 ** (-np.arange(16) / 16)
    table = np.stack((np.cos(ang), np.sin(ang)), axis=1)
    halves = OK.turn_rows(x, table)
    np.testing.assert_allclose(halves, OA.rope(x, pos[:, None], 10000.0), atol=1e-12)
    shuffled = np.concatenate((x[..., 0::2], x[..., 1::2]), axis=-1)
    pairs = OK.turn_rows(x, table, interleaved=True)
    np.testing.assert_array_equal(np.concatenate((pairs[..., 0::2], pairs[..., 1::2]), axis=-1), OK.turn_rows(shuffled, table))
    part = OK.turn_rows(x, table[:, :, :8])
    np.testing.assert_array_equal(part[..., 16:], x[..., 16:])
    np.testing.assert_array_equal(part[..., :16], OK.turn_rows(x[..., :16], table[:, :, :8]))


def test_append_oracle_without_norm_is_the_append():
    rng = np.random.default_rng(3)
    lens, counts, D = np.array([0, 3, 9]), np.array([5, 1, 4]), 32
    table = rng.permutation(15).reshape(3, 5)
    kc, vc = rng.standard_normal((15, 2, 4, D)), rng.standard_normal((15, 2, 4, D))
    k, v, q = rng.standard_normal((10, 2, D)), rng.standard_normal((10, 2, D)), rng.standard_normal((12, 4, D))
    ang = np.arange(20)[:, None] * 10000.0 ** (-np.arange(16) / 16)
    got = OK.append_normed(kc, vc, table, lens, k, v, counts, q=q, table=np.stack((np.cos(ang), np.sin(ang)), axis=1))
    want = OK.append_tokens(kc, vc, table, lens, k, v, counts, q=q, rope_base=10000.0)
    for g, w in zip(got, want):
        np.testing.assert_allclose(g, w, atol=1e-12)


def test_chunk_oracle_against_torch():
    """One request: torch's own causal attention (a mask for the window and the kept first keys)."""
    rng = np.random.default_rng(4)
    L, n, Hq, Hkv, D, bs = 21, 8, 4, 2, 16, 4
    table = rng.permutation(6)[None]
    kc, vc, q = rng.standard_normal((6, Hkv, bs, D)), rng.standard_normal((6, Hkv, bs, D)), rng.standard_normal((n + 1, Hq, D))
    keys, values = (np.concatenate([c[i] for i in table[0]], axis=1)[:, :L].repeat(2, axis=0) for c in (kc, vc))
    for window, sink in ((0, 0), (5, 2)):
        out, lse = OA.chunk_attention(q, kc, vc, table, [L], [n], window=window, n_sink=sink)
        far = (np.arange(L - n, L)[:, None] - np.arange(L)[None])
        seen = (far >= 0) & ((window == 0) | (far < window) | (np.arange(L)[None] < sink))
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[:n].transpose(1, 0, 2).copy()), torch.from_numpy(keys), torch.from_numpy(values),
            attn_mask=torch.from_numpy(seen)).numpy().transpose(1, 0, 2)
        np.testing.assert_allclose(out[:n], want, atol=1e-13)
        assert (out[n] == 0).all() and (lse[n] == -np.inf).all()


def test_sampling_oracle():
    """The limits one by one on a small row, against what each says."""
    x = np.log(np.array([0.05, 0.4, 0.1, 0.1, 0.3, 0.05]))
    p = lambda **kw: (lambda w: w / w.sum())(OS.processed(x, **kw))
    np.testing.assert_allclose(p(), np.exp(x), atol=1e-15)
    np.testing.assert_allclose(p(temperature=0.5), np.exp(2 * x) / np.exp(2 * x).sum(), atol=1e-15)
    np.testing.assert_allclose(p(top_k=3), np.array([0, 0.4, 0.1, 0, 0.3, 0]) / 0.8, atol=1e-15)
    np.testing.assert_allclose(p(top_p=0.65), np.array([0, 0.4, 0, 0, 0.3, 0]) / 0.7, atol=1e-15)
    np.testing.assert_allclose(p(top_p=0.75), np.array([0, 0.4, 0.1, 0, 0.3, 0]) / 0.8, atol=1e-15)
    np.testing.assert_allclose(p(min_p=0.2), np.array([0, 0.4, 0.1, 0.1, 0.3, 0]) / 0.9, atol=1e-15)
    np.testing.assert_allclose(p(top_k=2, top_p=0.5), np.array([0, 1.0, 0, 0, 0, 0]), atol=1e-15)
    assert p(temperature=0.0).tolist() == [0, 1, 0, 0, 0, 0] and p(top_p=0.0).tolist() == [0, 1, 0, 0, 0, 0]
    u = np.array([0.0, 0.04, 0.06, 0.5, 0.96, 1.0])
    tokens, _ = OS.token_sample(np.tile(x, (6, 1)), u)
    assert tokens.tolist() == [0, 0, 1, 2, 5, 5]
    assert OS.token_sample(np.array([[1.0, np.nan]]), [0.5])[0].tolist() == [-1]
