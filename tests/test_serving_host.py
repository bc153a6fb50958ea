"""Checks of the serving operators (append, one-token attention, token log
probabilities) that need no GPU: argument errors are reported before anything
is launched, and the oracle's definitions agree with independent ones."""

import ctypes
import importlib.util
import os
import types

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import kvcache as OK
from oracle import logprobs as OL
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


APPEND = dict(q=FAKE, q_stride=256, q_out=FAKE, q_out_stride=256, Hq=4, k_new=FAKE, k_stride=64, v_new=FAKE,
              v_stride=64, cu_new=None, T=6, k_cache=FAKE, v_cache=FAKE, num_blocks=9, block_size=16, table=FAKE,
              max_blocks=4, seq_lens=FAKE, new_lens=ctypes.c_void_p(8192), cos_sin=FAKE, max_pos=100, B=3, Hkv=1,
              head_dim=64, dtype=1, status=None, stream=None)


@pytest.mark.parametrize("change,code,text", [
    (dict(B=-1), -1, b"bad sizes"), (dict(T=-1), -1, b"bad sizes"), (dict(Hkv=0), -1, b"bad sizes"),
    (dict(Hq=0), -1, b"bad sizes"), (dict(max_pos=0), -1, b"bad sizes"), (dict(num_blocks=0), -1, b"bad sizes"),
    (dict(dtype=2), -4, b"dtype"), (dict(head_dim=48), -4, b"head_dim 48"), (dict(T=7), -1, b"multiple of B"),
    (dict(k_cache=None), -1, b"null"), (dict(v_new=None), -1, b"null"), (dict(seq_lens=None), -1, b"null"),
    (dict(cos_sin=None), -1, b"cos_sin"), (dict(q_out=None), -1, b"cos_sin"),
    (dict(new_lens=FAKE), -1, b"alias"), (dict(k_stride=-64), -1, b"stride"), (dict(q_out_stride=128), -1, b"stride"),
    (dict(k_stride=65), -1, b"16 bytes"), (dict(k_new=ctypes.c_void_p(4098)), -1, b"16 bytes"),
])
def test_append_refuses_on_the_host(change, code, text):
    assert _call("tv_kv_append", APPEND, **change) == code
    assert text in capi.lib().tv_last_error()


@pytest.mark.parametrize("at", [4096 - 8, 4096 - 4, 4096 + 4, 4096 + 8])
def test_append_refuses_lengths_that_overlap(at):
    """Shifted views of one buffer: a request's new length would land where another's old one is read."""
    assert _call("tv_kv_append", APPEND, new_lens=ctypes.c_void_p(at)) == -1
    assert b"overlap" in capi.lib().tv_last_error()


def test_append_of_an_empty_batch_does_nothing():
    assert _call("tv_kv_append", APPEND, B=0, T=0) == 0


def test_binding_refuses_tensors_off_the_gpu():
    t = torch.zeros(2, 1, 64)
    cache, table, lens = torch.zeros(3, 1, 16, 64), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        capi.tv_kv_append(t, t, cache, cache, table, lens)


def test_append_oracle_is_the_commit_of_a_chain():
    """Appending a chain's rotated rows is committing the path 0, 1, .. of a tree holding those rows rotated."""
    rng = np.random.default_rng(3)
    Bn, N, Hkv, D, bs = 3, 5, 2, 32, 4
    lens, counts = np.array([0, 3, 9]), np.array([5, 1, 4])
    table = rng.permutation(15).reshape(3, 5)
    kc, vc = rng.standard_normal((15, Hkv, bs, D)), rng.standard_normal((15, Hkv, bs, D))
    kt, vt = rng.standard_normal((Bn, N, Hkv, D)), rng.standard_normal((Bn, N, Hkv, D))
    pos = lens[:, None] + np.arange(N)[None]
    path = np.tile(np.arange(N), (Bn, 1))
    want = OK.commit_path(kc, vc, table, lens, OA.rope(kt, pos[:, :, None]), vt, path, counts)
    rows = [np.concatenate([t[b, :counts[b]] for b in range(Bn)]) for t in (kt, vt)]
    got = OK.append_tokens(kc, vc, table, lens, rows[0], rows[1], counts, rope_base=10000.0)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)


DECODE = dict(q=FAKE, q_stride=256, k_cache=FAKE, v_cache=FAKE, num_blocks=9, block_size=16, table=FAKE, max_blocks=4,
              seq_lens=FAKE, B=3, Hq=4, Hkv=2, head_dim=64, dtype=1, scale=0.125, softcap=0.0, window=0, n_sink=0,
              slopes=None, out=FAKE, lse=None, workspace=FAKE, workspace_bytes=16 << 20, num_ctas=8, flags=0,
              status=None, stream=None)


@pytest.mark.parametrize("change,code,text", [
    (dict(B=-1), -1, b"bad sizes"), (dict(Hq=5), -1, b"bad sizes"), (dict(Hkv=0), -1, b"bad sizes"),
    (dict(window=-1), -1, b"bad sizes"), (dict(n_sink=-1), -1, b"bad sizes"), (dict(block_size=0), -1, b"bad sizes"),
    (dict(num_ctas=4097), -1, b"bad sizes"), (dict(num_ctas=-1), -1, b"bad sizes"),
    (dict(dtype=7), -4, b"dtype"), (dict(head_dim=32), -4, b"head_dim 32"),
    (dict(softcap=-1.0), -1, b"softcap"), (dict(softcap=float("nan")), -1, b"softcap"),
    (dict(softcap=float("inf")), -1, b"softcap"), (dict(scale=float("inf")), -1, b"scale"),
    (dict(flags=1), -1, b"unknown flags"), (dict(q=None), -1, b"null"), (dict(out=None), -1, b"null"),
    (dict(table=None), -1, b"null"), (dict(q_stride=-256), -1, b"16 bytes"), (dict(q_stride=257), -1, b"16 bytes"),
    (dict(k_cache=ctypes.c_void_p(4104)), -1, b"16 bytes"), (dict(workspace=None), -5, b"workspace"),
    (dict(workspace_bytes=100), -5, b"workspace"), (dict(workspace=ctypes.c_void_p(4096 + 128)), -5, b"workspace"),
])
def test_decode_refuses_on_the_host(change, code, text):
    assert _call("tv_decode_attn", DECODE, **change) == code
    assert text in capi.lib().tv_last_error()


@pytest.mark.parametrize("change,text", [(dict(softcap=3e38), b"softcap"), (dict(scale=3e38), b"scale"),
                                         (dict(scale=-3e38), b"scale")])
def test_decode_refuses_factors_past_the_log2_domain(change, text):
    """Their product with log2 e is no float32: a score of 0 would come out as NaN."""
    assert _call("tv_decode_attn", DECODE, **change) == -1
    assert text in capi.lib().tv_last_error()


def test_decode_of_an_empty_batch_does_nothing():
    assert _call("tv_decode_attn", DECODE, B=0) == 0


def test_decode_workspace_size():
    n = [capi.tv_decode_attn_workspace_size(8, 2, 128, torch.bfloat16, num_ctas=k) for k in (1, 152, 304)]
    assert n[0] >= 16384 and n == sorted(n) and n[2] <= 16 << 20
    with pytest.raises(capi.TVError):
        capi.tv_decode_attn_workspace_size(9, 2, 128, torch.bfloat16, num_ctas=1)


def test_decode_oracle_is_the_one_node_tree():
    """The token's K/V in the cache, or as the root of a one-node tree over the prefix: the same definition."""
    rng = np.random.default_rng(4)
    Bn, Hq, Hkv, D, bs = 3, 4, 2, 32, 4
    lens = np.array([0, 3, 9])
    table = rng.permutation(12).reshape(3, 4)
    kc, vc = rng.standard_normal((12, Hkv, bs, D)), rng.standard_normal((12, Hkv, bs, D))
    q = rng.standard_normal((Bn, Hq, D))
    kt, vt = rng.standard_normal((Bn, 1, Hkv, D)), rng.standard_normal((Bn, 1, Hkv, D))
    want, wlse = OA.tree_attention(q[:, None], kc, vc, table, lens, kt, vt, np.array([-1]), rotate=False)
    kc, vc, now, _ = OK.append_tokens(kc, vc, table, lens, kt[:, 0], vt[:, 0], np.ones(3, dtype=int))
    got, lse = OA.decode_attention(q, kc, vc, table, now)
    np.testing.assert_allclose(got, want[:, 0], rtol=0, atol=1e-13)
    np.testing.assert_allclose(lse, wlse[:, 0], rtol=0, atol=1e-13)


def test_decode_oracle_masks_caps_and_biases():
    """Against torch's own softmax over a dense mask."""
    rng = np.random.default_rng(5)
    L, Hq, D = 11, 2, 8
    k, v = rng.standard_normal((1, 1, 16, D)), rng.standard_normal((1, 1, 16, D))
    q = rng.standard_normal((1, Hq, D)) * 4
    slopes = np.array([0.5, 0.0625])
    got, lse = OA.decode_attention(q, k, v, np.array([[0]]), [L], softcap=3.0, window=4, n_sink=2, slopes=slopes)
    s = torch.from_numpy(q[0] @ k[0, 0, :L].T / np.sqrt(D))
    s = 3.0 * torch.tanh(s / 3.0) + torch.from_numpy(slopes)[:, None] * (torch.arange(L) - (L - 1))
    s[:, 2:7] = -float("inf")
    np.testing.assert_allclose(got[0], (torch.softmax(s, -1) @ torch.from_numpy(v[0, 0, :L])).numpy(), atol=1e-13)
    np.testing.assert_allclose(lse[0], torch.logsumexp(s, -1).numpy(), atol=1e-13)
    empty, elast = OA.decode_attention(q, k, v, np.array([[0]]), [0])
    assert (empty == 0).all() and (elast == -np.inf).all()


LOGPROBS = dict(logits=FAKE, tokens=FAKE, node=None, B=2, N=3, C=3, V=100, dtype=0, logprob=FAKE, entropy=FAKE, top_k=4,
                top_ids=FAKE, top_logprobs=FAKE, status=None, stream=None)


@pytest.mark.parametrize("change,code,text", [
    (dict(B=-1), -1, b"bad sizes"), (dict(N=0), -1, b"bad sizes"), (dict(V=0), -1, b"bad sizes"),
    (dict(C=4), -1, b"bad sizes"), (dict(C=-1), -1, b"bad sizes"), (dict(dtype=3), -4, b"dtype"),
    (dict(top_k=33), -1, b"top_k"), (dict(top_k=-1), -1, b"top_k"), (dict(V=3), -1, b"top_k"),
    (dict(logits=None), -1, b"null"), (dict(tokens=None), -1, b"null"), (dict(logprob=None), -1, b"null"),
    (dict(top_ids=None), -1, b"null"), (dict(top_logprobs=None), -1, b"null"),
    (dict(logits=ctypes.c_void_p(4100)), -1, b"16-byte"), (dict(B=1 << 30, C=3), -4, b"2^31"),
])
def test_logprobs_refuse_on_the_host(change, code, text):
    assert _call("tv_token_logprobs", LOGPROBS, **change) == code
    assert text in capi.lib().tv_last_error()


def test_logprobs_of_nothing():
    assert _call("tv_token_logprobs", LOGPROBS, B=0) == 0
    assert _call("tv_token_logprobs", LOGPROBS, C=0) == 0


def test_logprobs_oracle_against_torch():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((2, 3, 50)) * 3
    x[0, 1, ::3] = -np.inf
    x[1, 2, 4] = x[1, 2, 9] = 20.0
    tok = rng.integers(0, 50, size=(2, 3))
    tok[1, 0] = -1
    lp, ent, ids, top = OL.token_logprobs(x, tok, None, 5)
    t = torch.from_numpy(x)
    ref = torch.log_softmax(t, -1)
    want = torch.where(torch.from_numpy(tok) >= 0, ref.gather(-1, torch.from_numpy(tok).clamp(min=0)[..., None])[..., 0], 0.0)
    np.testing.assert_allclose(lp, want.numpy(), atol=1e-13)
    h = torch.special.entr(torch.softmax(t, -1)).sum(-1).numpy()
    h[1, 0] = 0
    np.testing.assert_allclose(ent, h, atol=1e-13)
    assert ids[1, 2, :2].tolist() == [4, 9] and (ids[1, 0] == -1).all() and (top[1, 0] == -np.inf).all()
    for b, n in ((0, 0), (0, 1), (0, 2), (1, 1)):
        v, i = torch.topk(ref[b, n], 5)
        assert ids[b, n].tolist() == i.tolist()
        np.testing.assert_allclose(top[b, n], v.numpy(), atol=1e-13)
    nan = OL.token_logprobs(np.full((1, 1, 4), -np.inf), np.array([[2]]), None, 2)
    assert np.isnan(nan[0]).all() and np.isnan(nan[1]).all() and nan[2][0, 0].tolist() == [0, 1]


def test_binding_names_what_it_refuses():
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    cache, q = torch.zeros(3, 1, 16, 64), torch.zeros(2, 4, 64)
    for call in (lambda: capi.tv_decode_attn(q, cache, cache, table, lens),
                 lambda: capi.tv_decode_attn(q, cache, cache, table, [0, 0]),
                 lambda: capi.tv_token_logprobs(torch.zeros(2, 3, 10), lens[:, None]),
                 lambda: capi.tv_token_logprobs(None, lens[:, None])):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()


def test_decode_oracle_without_any_weight():
    """Keys of -inf under positive queries: every score is -inf, a zero row as for an empty request."""
    k, v = np.full((2, 1, 16, 8), -np.inf), np.ones((2, 1, 16, 8))
    k[1] = 1.0
    out, lse = OA.decode_attention(np.ones((2, 2, 8)), k, v, np.array([[0], [1]]), [5, 5])
    assert (out[0] == 0).all() and (lse[0] == -np.inf).all()
    np.testing.assert_allclose(out[1], 1.0, atol=1e-15)


@pytest.mark.parametrize("name", ["window", "n_sink", "num_ctas", "flags"])
@pytest.mark.parametrize("x", [1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 31) - 1, -(1 << 32)])
def test_binding_refuses_numbers_past_32_bits(name, x):
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    cache, q = torch.zeros(3, 1, 16, 64), torch.zeros(2, 4, 64)
    with pytest.raises(ValueError, match=name + f" {x}"):
        capi.tv_decode_attn(q, cache, cache, table, lens, **{name: x})
    if name == "window":
        with pytest.raises(ValueError, match=f"top_k {x}"):
            capi.tv_token_logprobs(torch.zeros(2, 3, 10), lens[:, None], top_k=x)


def test_binding_without_torchs_raw_calls(monkeypatch):
    """A torch without the two private names: the public calls give device and stream."""
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("capi_public", capi.__file__)
    copy = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(copy)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=70 + dev))
    assert copy._current() == (3, 73)
