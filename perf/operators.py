"""The single-token serving operators as they are measured: appending keys and
values to the paged cache with the rotation on the way, attention of one new
token over that cache, and log probabilities of emitted tokens.

``run`` makes either the plain form of a case (elementary torch operations in
float32, rounded once at the end) or, with ``own`` set, the library's calls.
Lengths and accepted counts follow from a case's sizes alone, so ``work`` can
count them; the values come from the seed.
"""

import math
import zlib

import numpy as np
import torch

own = False

_ITEM = {"f32": 4, "bf16": 2}
_TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
_SCRATCH = 16 << 20  # the attention scratch a serving program reserves once


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def _append(name, B, Hq, Hkv, D, dtype, bs, lo, hi, new_lo, new_hi, pad=0):
    """B requests with lo..hi cached tokens each get new_lo..new_hi more (new_hi = 0: one each, no offsets);
    ``pad`` rows of the packed buffers lie behind the last request."""
    c = {"op": "append", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "bs": bs, "lo": lo, "hi": hi,
         "new_lo": new_lo, "new_hi": new_hi, "pad": pad}
    return dict(c, name=name) if name else c


def _decode(name, B, Hq, Hkv, D, dtype, bs, lo, hi, empty=0, softcap=0.0, window=0, sink=0, alibi=False):
    """B slots with lo..hi cached tokens each (the last ``empty`` slots unused, length 0)."""
    c = {"op": "decode", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "bs": bs, "lo": lo, "hi": hi,
         "empty": empty, "softcap": softcap, "window": window, "sink": sink, "alibi": alibi}
    return dict(c, name=name) if name else c


def _logprobs(name, B, N, C, V, dtype, K, path=False, masked=False):
    """Logits [B, N, V]; ``path``: C acceptance columns of which a part is padding, else column = row;
    ``masked``: half of the vocabulary excluded (-inf), as under a grammar."""
    c = {"op": "logprobs", "B": B, "N": N, "C": C, "V": V, "dtype": dtype, "K": K, "path": path, "masked": masked}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request's next token: latency of a single launch
        _append("append_b1", 1, 32, 8, 128, "bf16", 16, 512, 2048, 0, 0),
        # a full batch's next tokens
        _append("append_b256", 256, 32, 8, 128, "bf16", 16, 512, 2048, 0, 0),
        # a batch of prompts, packed, some behind a shared prefix, the buffers longer than the batch
        _append("append_prompts", 32, 32, 8, 128, "bf16", 16, 0, 64, 1, 1023, 37),
        # float32 prompts with narrow heads
        _append("append_prompts_f32", 7, 8, 8, 64, "f32", 16, 0, 100, 301, 999, 5),
        # one request's next token over its cache: latency, one (request, head) split over many SMs
        _decode("decode_b1", 1, 32, 8, 128, "bf16", 16, 1001, 1001),
        # the 64-request workload's prefixes
        _decode("decode_b64", 64, 32, 8, 128, "bf16", 16, 1024, 8192),
        # the long-context workload
        _decode("decode_long", 16, 64, 8, 128, "bf16", 64, 32768, 32768),
        # capped scores and a sliding window behind a few kept tokens, a bucket with unused slots
        _decode("decode_window_cap", 256, 32, 8, 128, "bf16", 16, 2048, 4096, 9, 30.0, 1024, 4),
        # float32 with a distance bias, narrow heads, one query head per KV head
        _decode("decode_f32_bias", 24, 16, 16, 64, "f32", 16, 100, 3000, alibi=True),
        # one request's accepted tokens out of its tree's logits
        _logprobs("logprobs_b1", 1, 10, 5, 32000, "f32", 5, path=True),
        # 64 requests' accepted paths out of 64-node trees
        _logprobs("logprobs_tree", 64, 64, 7, 32000, "f32", 20, path=True),
        # scoring a prompt over a large vocabulary
        _logprobs("logprobs_prompt", 1, 1999, 1999, 128000, "bf16", 5),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "logprobs"))
    if op == "append":
        D, Hkv, G = rng.choice((64, 128, 256)), rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8))
        dtype, bs = rng.choice(("bf16", "f32")), rng.choice((16, 24, 32, 64))
        B = _log_uniform(rng, 1, 256)
        hi = _log_uniform(rng, 16, 2048)
        room = (4 << 28) // (Hkv * D * _ITEM[dtype] * 2)  # cache tokens
        hi = max(16, min(hi, room // B))
        if rng.random() < 0.4:
            return _append(None, B, G * Hkv, Hkv, D, dtype, bs, hi // 4, hi, 0, 0)
        n = max(1, min(_log_uniform(rng, 1, 4096), (200 << 20) // ((G + 2) * Hkv * D * _ITEM[dtype] * B)))
        least = 0 if B >= 8 and n >= 3 else max(1, n // 3)  # in a large batch some requests may bring nothing
        return _append(None, B, G * Hkv, Hkv, D, dtype, bs, 0, hi, least, n, rng.randrange(0, 50))
    if op == "decode":
        D, Hkv, G = rng.choice((64, 128, 256)), rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 5, 8, 16))
        dtype, bs = rng.choice(("bf16", "bf16", "f32")), rng.choice((16, 24, 32, 64))
        B = _log_uniform(rng, 1, 256)
        room = (1 << 30) // (Hkv * D * _ITEM[dtype] * 2)
        hi = max(1, min(_log_uniform(rng, 1, 32768), room // B))
        window = _log_uniform(rng, 1, 4096) if rng.random() < 0.4 else 0
        return _decode(None, B, G * Hkv, Hkv, D, dtype, bs, max(1, hi // rng.choice((1, 4, 20))), hi,
                       rng.randrange(0, B) // 8, rng.choice((0.0, 0.0, 20.0, 50.0)), window,
                       rng.choice((0, 4, 17)) if window else 0, rng.random() < 0.3)
    V = _log_uniform(rng, 500, 200000)
    K = rng.choice((0, 1, 5, 20, 32))
    dtype = rng.choice(("bf16", "f32"))
    rows = max(1, min(_log_uniform(rng, 1, 4000), 250_000_000 // V))
    if rng.random() < 0.5 and rows >= 8:
        N = rng.choice((5, 10, 26, 64))
        return _logprobs(None, max(1, rows // N), N, min(N, rng.randrange(2, 9)), V, dtype, K, True,
                         rng.random() < 0.3)
    return _logprobs(None, 1, rows, rows, V, dtype, K, False, rng.random() < 0.3)


def _rng(case):
    """A generator that goes by the case's sizes only."""
    key = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    return np.random.RandomState(zlib.crc32(key.encode()) & 0x7FFFFFFF)


def _lens(case):
    """(cached lengths [B], new tokens [B]) of an append or decode case."""
    r = _rng(case)
    lens = r.randint(case["lo"], case["hi"] + 1, size=case["B"])
    if case["op"] == "decode":
        if case["empty"]:
            lens[-case["empty"]:] = 0
        return lens, None
    if not case["new_hi"]:
        return lens, np.ones(case["B"], dtype=np.int64)
    return lens, r.randint(case["new_lo"], case["new_hi"] + 1, size=case["B"])


def _accepted(case):
    """Emitted tokens per request of a path case (acceptance gives at least one)."""
    return _rng(case).randint(1, case["C"] + 1, size=case["B"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _pages(need_tokens, bs, r):
    """Block table of requests that own ceil(n / bs) randomly placed blocks each."""
    need = -(-np.asarray(need_tokens, dtype=np.int64) // bs)
    total = max(1, int(need.sum()))
    table = np.zeros((need.size, max(1, int(need.max()))), dtype=np.int32)
    cols = np.arange(table.shape[1])[None] < need[:, None]
    table[cols] = r.permutation(total)[:int(need.sum())].astype(np.int32)
    return torch.from_numpy(table).cuda(), total


def _rope_rows(n, D):
    """cos and sin of pos * 10000^(-2k/D), [n, 2, D/2], float64 rounded to float32."""
    k = torch.arange(D // 2, dtype=torch.float64, device="cuda")
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * torch.pow(10000.0, -2.0 * k / D)
    return torch.stack((torch.cos(ang), torch.sin(ang)), dim=1).float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    r = np.random.RandomState(int(seed) & 0x7FFFFFFF)
    dt = _TYPE[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = {"case": case}
    if case["op"] == "logprobs":
        B, N, C, V = case["B"], case["N"], case["C"], case["V"]
        logits = torch.randn(B, N, V, generator=g, device="cuda", dtype=torch.float32).mul_(math.sqrt(2.0))
        if case["masked"]:
            shut = torch.rand(V, generator=g, device="cuda") < 0.5
            shut[0] = False
            logits.masked_fill_(shut, -math.inf)
        s["logits"] = logits.to(dt)
        # emitted tokens: the likeliest one half of the time, else any
        if case["path"]:
            n = _accepted(case)
            node = np.full((B, C), -1, dtype=np.int32)
            for b in range(B):
                node[b, 1:n[b]] = np.sort(r.permutation(np.arange(1, N))[:n[b] - 1])
                node[b, 0] = 0
            s["node"] = torch.from_numpy(node).cuda()
            rows = s["node"].clamp(min=0).long()
        else:
            s["node"] = None
            rows = torch.arange(C, device="cuda").expand(B, C)
        best = s["logits"].argmax(dim=-1).gather(1, rows)
        anyone = torch.randint(0, V, (B, C), generator=g, device="cuda")
        tokens = torch.where(torch.rand(B, C, generator=g, device="cuda") < 0.5, best, anyone)
        if case["path"]:
            tokens = torch.where(s["node"] < 0, -1, tokens)
        s["tokens"] = tokens.to(torch.int32).contiguous()
        return s

    B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
    lens, new = _lens(case)
    s["seq_lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    s["table"], blocks = _pages(lens if new is None else lens + new, bs, r)
    s["k_cache"] = randn(blocks, Hkv, bs, D)
    s["v_cache"] = randn(blocks, Hkv, bs, D)
    if case["op"] == "append":
        total = int(new.sum())
        rows = total + case["pad"]
        s["total"] = total
        s["cu"] = None
        if case["new_hi"]:
            s["cu"] = torch.from_numpy(np.concatenate(([0], np.cumsum(new))).astype(np.int32)).cuda()
        # the three come out of one projection: heads of q, k and v side by side in a row
        qkv = randn(rows, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_out"] = torch.zeros(rows, Hq, D, dtype=dt, device="cuda")
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["cos_sin"] = _rope_rows(int((lens + new).max()) + 1, D)
        return s
    s["q"] = randn(B, Hq, D)
    s["slopes"] = None
    if case["alibi"]:  # the usual geometric slopes
        s["slopes"] = torch.pow(2.0, -8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32) / Hq)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(B, Hq, dtype=torch.float32, device="cuda")
    s["scratch"] = torch.zeros(_SCRATCH, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    case = s["case"]
    if own:
        from speculative_decoding_tree_attn_gb300 import capi

        if case["op"] == "append":
            capi.tv_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                              cos_sin=s["cos_sin"], q=s["q"], q_out=s["q_out"], cu_new=s["cu"],
                              new_seq_lens=s["new_lens"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["new_lens"]}
        if case["op"] == "decode":
            capi.tv_decode_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                                softcap=case["softcap"], window=case["window"], n_sink=case["sink"],
                                slopes=s["slopes"], out=s["out"], lse=s["lse"], workspace=s["scratch"],
                                flags=capi.TV_ATTN_WORKSPACE_ZEROED)
            return {"out": s["out"], "lse": s["lse"]}
        lp, ent, ids, top = capi.tv_token_logprobs(s["logits"], s["tokens"], node=s["node"], top_k=case["K"])
        return {"logprob": lp, "entropy": ent, "ids": ids, "top": top}
    return {"append": _run_append, "decode": _run_decode, "logprobs": _run_logprobs}[case["op"]](s)


def _rotated(x, rows, D):
    """x [T, H, D] in float32 turned by the table rows [T, 2, D/2]."""
    c, n = rows[:, None, 0], rows[:, None, 1]
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat((a * c - b * n, b * c + a * n), dim=-1)


def _run_append(s):
    case, total = s["case"], s["total"]
    D, bs, dt = case["D"], case["bs"], s["q"].dtype
    t = torch.arange(total, device="cuda")
    if s["cu"] is None:
        b, j = t, torch.zeros_like(t)
    else:
        cu = s["cu"].long()
        b = torch.bucketize(t, cu[1:], right=True)
        j = t - cu[b]
    pos = s["seq_lens"].long()[b] + j
    block, slot = s["table"].long()[b, pos // bs], pos % bs
    rows = s["cos_sin"][pos]
    s["k_cache"][block, :, slot] = _rotated(s["k"][:total].float(), rows, D).to(dt)
    s["v_cache"][block, :, slot] = s["v"][:total]
    s["q_out"][:total] = _rotated(s["q"][:total].float(), rows, D).to(dt)
    added = 1 if s["cu"] is None else s["cu"][1:] - s["cu"][:-1]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["seq_lens"] + added}


def _run_decode(s):
    case = s["case"]
    B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
    G, n = Hq // Hkv, s["table"].shape[1] * bs

    def rows(cache):
        return cache[s["table"].long()].transpose(1, 2).reshape(B, Hkv, n, D).float()

    x = torch.matmul(s["q"].float().view(B, Hkv, G, D), rows(s["k_cache"]).transpose(2, 3)) / math.sqrt(D)
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    t = torch.arange(n, device="cuda")
    L = s["seq_lens"].long()[:, None]
    if s["slopes"] is not None:
        x = x + s["slopes"].view(Hkv, G, 1) * (t - (L - 1)).float()[:, None, None]
    seen = t < L
    if case["window"]:
        seen = seen & ((t >= L - case["window"]) | (t < case["sink"]))
    x = torch.where(seen[:, None, None], x, -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    z = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, rows(s["v_cache"])) / torch.where(z == 0, 1.0, z)
    return {"out": out.reshape(B, Hq, D).to(s["q"].dtype), "lse": (m + torch.log(z)).reshape(B, Hq)}


def _run_logprobs(s):
    case = s["case"]
    B, N, C, V, K = case["B"], case["N"], case["C"], case["V"], case["K"]
    if s["node"] is None:
        x, ok = s["logits"][:, :C].reshape(B * C, V), s["tokens"].view(-1) >= 0
    else:
        ok = ((s["node"] >= 0) & (s["tokens"] >= 0)).view(-1)
        at = torch.arange(B, device="cuda")[:, None] * N + s["node"].clamp(min=0)
        x = s["logits"].view(B * N, V)[at.view(-1)]
    x = x.float()
    m = x.amax(dim=-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(dim=-1, keepdim=True)
    lse = m + torch.log(z)
    ent = torch.log(z) - torch.where(e > 0, e * (x - m), 0.0).sum(dim=-1, keepdim=True) / z
    lp = x.gather(1, s["tokens"].view(-1, 1).clamp(min=0).long()) - lse
    # one whole number orders a row: the value's bits in ascending order, then the lower index first
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits) * (1 << 31) + (V - 1 - torch.arange(V, device="cuda"))
    ids = V - 1 - (torch.topk(key, K, dim=-1).values & ((1 << 31) - 1))
    top = x.gather(1, ids) - lse
    ok = ok[:, None]
    return {"logprob": torch.where(ok, lp, 0.0).view(B, C), "entropy": torch.where(ok, ent, 0.0).view(B, C),
            "ids": torch.where(ok, ids, -1).to(torch.int32).view(B, C, K),
            "top": torch.where(ok, top, -math.inf).view(B, C, K)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        lens, new = _lens(case)
        D, bs = case["D"], case["bs"]
        kc, vc, qo = s["k_cache"].double(), s["v_cache"].double(), s["q_out"].double()
        start = 0
        for b in range(case["B"]):
            n, L = int(new[b]), int(lens[b])
            if n == 0:
                continue
            at = slice(start, start + n)
            start += n
            p = torch.arange(L, L + n, device="cuda")
            turn = torch.complex(*s["cos_sin"][L:L + n].double().unbind(1))[:, None]

            def turned(x):
                z = torch.complex(x[..., :D // 2].double(), x[..., D // 2:].double()) * turn
                return torch.cat((z.real, z.imag), dim=-1)

            block, slot = s["table"][b, p // bs].long(), p % bs
            kc[block, :, slot] = turned(s["k"][at])
            vc[block, :, slot] = s["v"][at].double()
            qo[at] = turned(s["q"][at])
        return {"q": qo, "k_cache": kc, "v_cache": vc, "lens": torch.from_numpy((lens + new).astype(np.int32))}
    if case["op"] == "decode":
        lens, _ = _lens(case)
        B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
        out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            L = int(lens[b])
            keep = [t for t in range(L) if not case["window"] or t >= L - case["window"] or t < case["sink"]]
            if not keep:
                continue
            t = torch.tensor(keep, device="cuda")
            block, slot = s["table"][b, t // bs].long(), t % bs
            k = s["k_cache"][block, :, slot].double().repeat_interleave(Hq // Hkv, dim=1)
            v = s["v_cache"][block, :, slot].double().repeat_interleave(Hq // Hkv, dim=1)
            x = torch.einsum("hd,thd->ht", s["q"][b].double(), k) * D ** -0.5
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            if s["slopes"] is not None:
                x = x - s["slopes"].double()[:, None] * (L - 1 - t).double()
            lse[b] = torch.logsumexp(x, dim=1)
            out[b] = torch.einsum("ht,thd->hd", torch.exp(x - lse[b][:, None]), v)
        return {"out": out, "lse": lse}
    B, N, C, V, K = case["B"], case["N"], case["C"], case["V"], case["K"]
    lp = torch.zeros(B, C, dtype=torch.float64, device="cuda")
    ent = torch.zeros(B, C, dtype=torch.float64, device="cuda")
    ids = torch.full((B, C, K), -1, dtype=torch.int32, device="cuda")
    top = torch.full((B, C, K), -math.inf, dtype=torch.float64, device="cuda")
    tokens = s["tokens"].cpu().numpy()
    node = np.tile(np.arange(C), (B, 1)) if s["node"] is None else s["node"].cpu().numpy()
    for b in range(B):
        for c in range(C):
            if node[b, c] < 0 or tokens[b, c] < 0:
                continue
            x = s["logits"][b, int(node[b, c])].double()
            logp = torch.log_softmax(x, dim=0)
            lp[b, c] = logp[int(tokens[b, c])]
            ent[b, c] = -torch.xlogy(logp.exp(), logp.exp()).sum()
            if K:
                order = torch.sort(x, descending=True, stable=True).indices[:K]
                ids[b, c] = order.to(torch.int32)
                top[b, c] = logp[order]
    return {"logprob": lp, "entropy": ent, "ids": ids, "top": top}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    if case["op"] == "append":
        _, new = _lens(case)
        n, e = int(new.sum()), _ITEM[case["dtype"]]
        heads = case["Hq"] + 2 * case["Hkv"]
        bytes_ = n * (2 * heads * case["D"] * e + 4 * case["D"]) + 8 * case["B"]
        return {"bytes": bytes_, "flops": 3 * n * case["D"] * (case["Hq"] + case["Hkv"])}
    if case["op"] == "decode":
        lens, _ = _lens(case)
        L = lens.astype(np.int64)
        if case["window"]:
            L = np.minimum(L, case["window"] + np.minimum(case["sink"], np.maximum(L - case["window"], 0)))
        keys, e = int(L.sum()), _ITEM[case["dtype"]]
        io = 2 * case["B"] * case["Hq"] * case["D"] * e + 4 * case["B"] * case["Hq"]
        return {"bytes": keys * case["Hkv"] * case["D"] * 2 * e + io, "flops": 4 * keys * case["Hq"] * case["D"]}
    rows = int(_accepted(case).sum()) if case["path"] else case["B"] * case["C"]
    n = rows * case["V"]
    return {"bytes": n * _ITEM[case["dtype"]] + case["B"] * case["C"] * (16 + 8 * case["K"]), "flops": 6 * n}
