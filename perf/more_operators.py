"""The operators of a prompt's way to its first token as they are measured:
queries and keys normalised per head, rotated and put into the paged cache,
attention of a chunk of new tokens over that cache, and sampling of a token
from a row of logits.

``run`` makes either the plain form of a case (elementary torch operations in
float32, sums of probabilities in float64, rounded once at the end) or, with
``own`` set, the library's calls.  Lengths follow from a case's sizes alone,
so ``work`` can count them; the values come from the seed.
"""

import math
import zlib

import numpy as np
import torch

own = False

_ITEM = {"f32": 4, "bf16": 2}
_TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
_SCRATCH = 96 << 20  # the attention scratch a serving program reserves once
_EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def _norm(name, B, Hq, Hkv, D, dtype, bs, lo, hi, new_lo, new_hi, pad=0, rot=0, pairs=False):
    """B requests with lo..hi cached tokens each get new_lo..new_hi more (new_hi = 0: one each, no offsets);
    ``rot`` leading elements of a head are rotated (0: all), ``pairs``: neighbours instead of halves;
    ``pad`` rows of the packed buffers lie behind the last request."""
    c = {"op": "norm", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "bs": bs, "lo": lo, "hi": hi,
         "new_lo": new_lo, "new_hi": new_hi, "pad": pad, "rot": rot or D, "pairs": pairs}
    return dict(c, name=name) if name else c


def _chunk(name, B, Hq, Hkv, D, dtype, bs, lo, hi, new_lo, new_hi, pad=0, softcap=0.0, window=0, sink=0, alibi=False):
    """Chunks of new_lo..new_hi tokens behind lo..hi cached ones, their own keys and values in the cache too."""
    c = {"op": "chunk", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "bs": bs, "lo": lo, "hi": hi,
         "new_lo": new_lo, "new_hi": new_hi, "pad": pad, "softcap": softcap, "window": window, "sink": sink,
         "alibi": alibi}
    return dict(c, name=name) if name else c


def _sample(name, R, V, dtype, k=0, p=0.0, min_p=0.0, temps=True, mixed=False, probs=False):
    """R rows of V logits; k, p, min_p: the requests' limits (0: none asks for that one); ``mixed``: only some
    requests ask for each and some are greedy; ``probs``: the processed distributions are wanted too."""
    c = {"op": "sample", "R": R, "V": V, "dtype": dtype, "k": k, "p": p, "min_p": min_p, "temps": temps,
         "mixed": mixed, "probs": probs}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a full batch's next tokens
        _norm("norm_b256", 256, 32, 8, 128, "bf16", 16, 512, 2048, 0, 0),
        # a batch of prompts, packed, some behind a shared prefix, the buffers longer than the batch
        _norm("norm_prompts", 32, 32, 8, 128, "bf16", 16, 0, 64, 1, 1023, 37),
        # float32 prompts, narrow heads of which a half is rotated in neighbouring pairs
        _norm("norm_pairs_f32", 7, 8, 8, 64, "f32", 16, 0, 100, 301, 999, 5, rot=32, pairs=True),
        # the last short piece of one prompt: latency, the cache split over many SMs
        _chunk("chunk_b1", 1, 32, 8, 128, "bf16", 16, 1001, 1001, 17, 17),
        # 64 conversations' next messages over what is cached of them
        _chunk("chunk_turns", 64, 32, 8, 128, "bf16", 16, 1024, 8192, 5, 300),
        # a batch of whole prompts, packed, the buffers longer than the batch
        _chunk("chunk_prompts", 32, 32, 8, 128, "bf16", 16, 0, 64, 1, 1023, 37),
        # the last quarter of a long prompt that is taken in pieces
        _chunk("chunk_long", 1, 64, 8, 128, "bf16", 64, 24576, 24576, 8192, 8192),
        # capped scores and a sliding window behind a few kept tokens
        _chunk("chunk_window_cap", 16, 32, 8, 128, "bf16", 16, 0, 6000, 100, 2047, 0, 30.0, 1024, 4),
        # float32 with a distance bias, narrow heads, one query head per KV head
        _chunk("chunk_f32_bias", 6, 16, 16, 64, "f32", 16, 0, 700, 33, 500, alibi=True),
        # one request's next token
        _sample("sample_b1", 1, 32000, "f32", 50, 0.95),
        # a drafter's rows: tokens and the distributions that acceptance compares them with
        _sample("sample_draft", 64, 32000, "f32", 0, 0.9, 0.01, probs=True),
        # a full batch over a large vocabulary, every request with its own settings
        _sample("sample_b256", 256, 128000, "bf16", 200, 0.95, 0.02, mixed=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "chunk", "sample"))
    if op == "norm":
        D, Hkv, G = rng.choice((64, 128, 256)), rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 5, 8))
        dtype, bs = rng.choice(("bf16", "f32")), rng.choice((16, 24, 32, 64))
        rot, pairs = rng.choice((D, D, D // 2, 48)), rng.random() < 0.4
        B = _log_uniform(rng, 1, 256)
        hi = _log_uniform(rng, 16, 2048)
        room = (4 << 28) // (Hkv * D * _ITEM[dtype] * 2)  # cache tokens
        hi = max(16, min(hi, room // B))
        if rng.random() < 0.4:
            return _norm(None, B, G * Hkv, Hkv, D, dtype, bs, hi // 4, hi, 0, 0, 0, rot, pairs)
        n = max(1, min(_log_uniform(rng, 1, 4096), (200 << 20) // ((G + 2) * Hkv * D * _ITEM[dtype] * B)))
        least = 0 if B >= 8 and n >= 3 else max(1, n // 3)  # in a large batch some requests may bring nothing
        return _norm(None, B, G * Hkv, Hkv, D, dtype, bs, 0, hi, least, n, rng.randrange(0, 50), rot, pairs)
    if op == "chunk":
        D, Hkv, G = rng.choice((64, 128, 128, 256)), rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 5, 8, 16))
        dtype, bs = rng.choice(("bf16", "bf16", "bf16", "f32")), rng.choice((16, 24, 32, 64))
        B = _log_uniform(rng, 1, 64)
        room = (1 << 29) // (Hkv * D * _ITEM[dtype] * 2)
        n = max(1, min(_log_uniform(rng, 1, 4096), room // B, (1 << 27) // (G * Hkv * D * B)))
        hi = max(0, min(_log_uniform(rng, 1, 16384) - 1, room // B - n))
        most = 1.5e11 if dtype == "f32" else 4e11 if D == 256 else 2e12  # products
        n = max(1, min(n, int(most / (4 * D * G * Hkv * B * (hi + n)))))
        window = _log_uniform(rng, 1, 4096) if rng.random() < 0.3 else 0
        return _chunk(None, B, G * Hkv, Hkv, D, dtype, bs, hi // rng.choice((1, 4, 20)), hi, max(1, n // 4), n,
                      rng.randrange(0, 50), rng.choice((0.0, 0.0, 0.0, 20.0, 50.0)), window,
                      rng.choice((0, 4, 17)) if window else 0, rng.random() < 0.2)
    V = _log_uniform(rng, 500, 200000)
    R = max(1, min(_log_uniform(rng, 1, 1000), 32_000_000 // V))
    return _sample(None, R, V, rng.choice(("bf16", "f32")), rng.choice((0, 1, 20, 200, 5000)),
                   rng.choice((0.0, 0.3, 0.9, 0.99)), rng.choice((0.0, 0.0, 0.05, 0.3)), rng.random() < 0.8,
                   rng.random() < 0.5, rng.random() < 0.4)


def _rng(case):
    """A generator that goes by the case's sizes only."""
    key = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    return np.random.RandomState(zlib.crc32(key.encode()) & 0x7FFFFFFF)


def _lens(case):
    """(cached lengths [B], new tokens [B]) of a norm or chunk case."""
    r = _rng(case)
    lens = r.randint(case["lo"], case["hi"] + 1, size=case["B"]).astype(np.int64)
    if not case["new_hi"]:
        return lens, np.ones(case["B"], dtype=np.int64)
    return lens, r.randint(case["new_lo"], case["new_hi"] + 1, size=case["B"]).astype(np.int64)


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


def _prepare_sample(case, s, g, r):
    R, V = case["R"], case["V"]
    # rows of different sharpness, as models give them
    spread = torch.from_numpy(r.uniform(1.5, 3.5, size=(R, 1)).astype(np.float32)).cuda()
    s["logits"] = (torch.randn(R, V, generator=g, device="cuda", dtype=torch.float32) * spread).to(_TYPE[case["dtype"]])
    s["u"] = torch.rand(R, generator=g, device="cuda", dtype=torch.float32)

    def asked(value, off, dtype):
        """The requests' limits: all the same, or up to it for some of them."""
        if not value:
            return None
        v = np.full(R, value, dtype=np.float64)
        if case["mixed"]:
            v *= r.uniform(0.5, 1.0, size=R)
            v[r.uniform(size=R) < 0.3] = off
        return torch.from_numpy(v.astype(dtype)).cuda()

    s["k"], s["p"], s["min_p"] = asked(case["k"], 0, np.int32), asked(case["p"], 1.0, np.float32), \
        asked(case["min_p"], 0.0, np.float32)
    s["t"] = None
    if case["temps"]:
        t = r.uniform(0.6, 1.2, size=R).astype(np.float32)
        if case["mixed"]:
            t[r.uniform(size=R) < 0.1] = 0.0
        s["t"] = torch.from_numpy(t).cuda()
    s["tokens"] = torch.zeros(R, dtype=torch.int32, device="cuda")
    s["probs"] = torch.zeros(R, V, dtype=torch.float32, device="cuda") if case["probs"] else None


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    r = np.random.RandomState(int(seed) & 0x7FFFFFFF)
    dt = _TYPE[case["dtype"]]
    s = {"case": case}
    if case["op"] == "sample":
        _prepare_sample(case, s, g, r)
        return s

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
    lens, new = _lens(case)
    s["lens"], s["new"], s["total"] = lens.tolist(), new.tolist(), int(new.sum())
    s["table"], blocks = _pages(lens + new, bs, r)
    s["k_cache"] = randn(blocks, Hkv, bs, D)
    s["v_cache"] = randn(blocks, Hkv, bs, D)
    s["cu"] = None
    if case["new_hi"]:
        s["cu"] = torch.from_numpy(np.concatenate(([0], np.cumsum(new))).astype(np.int32)).cuda()
    rows = s["total"] + case["pad"]
    if case["op"] == "norm":
        s["seq_lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        # the three come out of one projection: heads of q, k and v side by side in a row
        qkv = randn(rows, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_weight"] = (1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt)
        s["k_weight"] = (1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt)
        s["q_out"] = torch.zeros(rows, Hq, D, dtype=dt, device="cuda")
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["cos_sin"] = _rope_rows(int((lens + new).max()) + 1, case["rot"])
        return s
    s["seq_lens"] = torch.from_numpy((lens + new).astype(np.int32)).cuda()
    s["q"] = randn(rows, Hq, D)
    s["slopes"] = None
    if case["alibi"]:  # the usual geometric slopes
        s["slopes"] = torch.pow(2.0, -8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32) / Hq)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(rows, Hq, dtype=torch.float32, device="cuda")
    s["scratch"] = torch.zeros(_SCRATCH, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    case = s["case"]
    if own:
        from speculative_decoding_tree_attn_gb300 import capi

        if case["op"] == "norm":
            capi.tv_kv_append_norm(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                                   k_weight=s["k_weight"], q=s["q"], q_weight=s["q_weight"], q_out=s["q_out"],
                                   eps=_EPS, cos_sin=s["cos_sin"], interleaved=case["pairs"], cu_new=s["cu"],
                                   new_seq_lens=s["new_lens"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["new_lens"]}
        if case["op"] == "chunk":
            capi.tv_chunk_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], cu_new=s["cu"],
                               softcap=case["softcap"], window=case["window"], n_sink=case["sink"],
                               slopes=s["slopes"], out=s["out"], lse=s["lse"], workspace=s["scratch"],
                               flags=capi.TV_ATTN_WORKSPACE_ZEROED)
            return {"out": s["out"], "lse": s["lse"]}
        capi.tv_token_sample(s["logits"], s["u"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["min_p"],
                             tokens=s["tokens"], probs=s["probs"])
        return {"tokens": s["tokens"], "probs": s["probs"]} if case["probs"] else {"tokens": s["tokens"]}
    return {"norm": _run_norm, "chunk": _run_chunk, "sample": _run_sample}[case["op"]](s)


def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + _EPS) * w.float()


def _turned(x, rows, pairs):
    """x [T, H, D] with its leading elements turned by the table rows [T, 2, R/2]."""
    half = rows.shape[2]
    c, n = rows[:, None, 0], rows[:, None, 1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if pairs else (x[..., :half], x[..., half:2 * half])
    y = x.clone()
    if pairs:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * n, b * c + a * n
    else:
        y[..., :half], y[..., half:2 * half] = a * c - b * n, b * c + a * n
    return y


def _run_norm(s):
    case, total = s["case"], s["total"]
    bs, dt = case["bs"], s["q"].dtype
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
    s["k_cache"][block, :, slot] = _turned(_normed(s["k"][:total], s["k_weight"]), rows, case["pairs"]).to(dt)
    s["v_cache"][block, :, slot] = s["v"][:total]
    s["q_out"][:total] = _turned(_normed(s["q"][:total], s["q_weight"]), rows, case["pairs"]).to(dt)
    added = 1 if s["cu"] is None else s["cu"][1:] - s["cu"][:-1]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["seq_lens"] + added}


def _seen(case, pos, t):
    """Which keys t [L] the tokens at pos [n] see."""
    seen = t[None] <= pos[:, None]
    if case["window"]:
        seen = seen & ((t[None] > pos[:, None] - case["window"]) | (t[None] < case["sink"]))
    return seen


def _run_chunk(s):
    case = s["case"]
    Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
    G, at = Hq // Hkv, 0
    for b, (c, n) in enumerate(zip(s["lens"], s["new"])):
        L = c + n
        blocks = s["table"][b, :-(-L // bs)].long()
        k, v = (x[blocks].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].float() for x in (s["k_cache"], s["v_cache"]))
        t = torch.arange(L, device="cuda")
        step = max(1, (1 << 28) // (Hq * L))  # tokens whose scores are held at a time
        for j in range(0, n, step):
            e = min(n, j + step)
            q = s["q"][at + j:at + e].float().view(e - j, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
            x = (torch.matmul(q, k.transpose(1, 2)) / math.sqrt(D)).view(Hkv, G, e - j, L)
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            pos = c + torch.arange(j, e, device="cuda")
            if s["slopes"] is not None:
                x = x + s["slopes"].view(Hkv, G, 1, 1) * (t[None] - pos[:, None]).float()
            x = torch.where(_seen(case, pos, t), x, -math.inf)
            m = x.amax(dim=-1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            p = torch.exp(x - m)
            z = p.sum(dim=-1, keepdim=True)
            o = torch.matmul(p.view(Hkv, -1, L), v).view(Hkv, G, e - j, D) / torch.where(z == 0, 1.0, z)
            s["out"][at + j:at + e] = o.permute(2, 0, 1, 3).reshape(e - j, Hq, D).to(s["q"].dtype)
            s["lse"][at + j:at + e] = (m + torch.log(z)).permute(2, 0, 1, 3).reshape(e - j, Hq)
        at += n
    return {"out": s["out"], "lse": s["lse"]}


def _run_sample(s):
    """Probabilities and their sums in 64 bits: in 32 a long row's sum is off by more than a token's share."""
    x = s["logits"].float()
    R, V = x.shape
    t = s["t"].double()[:, None] if s["t"] is not None else torch.ones(R, 1, dtype=torch.float64, device="cuda")
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices  # equal logits: the lower index first
    y = x.double()
    y = y - y.amax(dim=-1, keepdim=True)
    w = torch.exp(torch.where(t > 0, y / torch.where(t > 0, t, 1.0), torch.where(y == 0, 0.0, -math.inf)))
    w = w.gather(1, order)
    rank = torch.arange(V, device="cuda")[None]
    keep = torch.where(t > 0, rank >= 0, rank == 0)  # without a temperature the likeliest alone
    if s["k"] is not None:
        keep = keep & ((s["k"][:, None] <= 0) | (rank < s["k"][:, None]))
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"].double()[:, None])
    if s["p"] is not None:
        w = torch.where(keep, w, 0.0)
        before = torch.cumsum(w, dim=-1) - w
        p = s["p"].double()[:, None]
        keep = keep & ((p >= 1.0) | (before < p * w.sum(dim=-1, keepdim=True)))
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    cdf = torch.cumsum(w, dim=-1)
    total = cdf[:, -1:]
    tokens = (cdf <= s["u"].double()[:, None] * total).sum(dim=-1)
    s["tokens"].copy_(tokens)
    if s["probs"] is None:
        return {"tokens": s["tokens"]}
    s["probs"].copy_(w / total)
    return {"tokens": s["tokens"], "probs": s["probs"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------


def _exact_norm(case, s):
    lens, new = _lens(case)
    bs, half = case["bs"], case["rot"] // 2
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

        def turned(x, w):
            x = x.double()
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + _EPS) * w.double()
            z = x[..., :2 * half]
            z = z.unflatten(-1, (half, 2)) if case["pairs"] else z.unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z.flatten(-2) if case["pairs"] else z.transpose(-1, -2).flatten(-2)
            return torch.cat((z, x[..., 2 * half:]), dim=-1)

        block, slot = s["table"][b, p // bs].long(), p % bs
        kc[block, :, slot] = turned(s["k"][at], s["k_weight"])
        vc[block, :, slot] = s["v"][at].double()
        qo[at] = turned(s["q"][at], s["q_weight"])
    return {"q": qo, "k_cache": kc, "v_cache": vc, "lens": torch.from_numpy((lens + new).astype(np.int32))}


def _exact_chunk(case, s):
    lens, new = _lens(case)
    Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
    out, lse = s["out"].double(), s["lse"].double()
    start = 0
    for b in range(case["B"]):
        n, L = int(new[b]), int(lens[b] + new[b])
        first = start
        start += n
        p = torch.arange(L, device="cuda")
        block, slot = s["table"][b, p // bs].long(), p % bs
        keys, values = s["k_cache"][block, :, slot].double(), s["v_cache"][block, :, slot].double()  # [L, Hkv, D]
        step = max(1, (1 << 26) // L)
        for j in range(0, n, step):
            e = min(n, j + step)
            far = (L - n + torch.arange(j, e, device="cuda"))[:, None] - p[None]  # how far back a key lies
            shut = far < 0
            if case["window"]:
                shut = shut | ((far >= case["window"]) & (p[None] >= case["sink"]))
            for h in range(Hq):
                x = s["q"][first + j:first + e, h].double() @ keys[:, h // (Hq // Hkv)].T * D ** -0.5
                if case["softcap"]:
                    x = torch.tanh(x / case["softcap"]) * case["softcap"]
                if s["slopes"] is not None:
                    x = x - s["slopes"][h].double() * far.double()
                x.masked_fill_(shut, -math.inf)
                z = torch.logsumexp(x, dim=1)
                lse[first + j:first + e, h] = z
                out[first + j:first + e, h] = x.sub_(z[:, None]).exp_() @ values[:, h // (Hq // Hkv)]
    return {"out": out, "lse": lse}


def _exact_sample(case, s):
    R, V = case["R"], case["V"]
    tokens = torch.zeros(R, dtype=torch.int32)
    probs = torch.zeros(R, V, dtype=torch.float64, device="cuda") if case["probs"] else None

    def of(name, i, off):
        return off if s[name] is None else float(s[name][i])

    for i in range(R):
        x = s["logits"][i].double()
        t, k, p, least = of("t", i, 1.0), int(of("k", i, 0)), of("p", i, 1.0), of("min_p", i, 0.0)
        if t == 0.0:
            kept = torch.nonzero(x == x.max())[:1, 0]
        else:
            # the likeliest k, then the probable enough, then as many as hold p of what is left
            kept = torch.argsort(x, descending=True, stable=True)
            if k > 0:
                kept = kept[:k]
            q = torch.softmax(x[kept] / t, dim=0)
            kept = kept[q >= least * q[0]]
            q = torch.softmax(x[kept] / t, dim=0)
            if p < 1.0:
                kept = kept[:1 + int((torch.cumsum(q, 0)[:-1] < p).sum())]
        kept = torch.sort(kept).values
        q = torch.softmax(x[kept] / (t or 1.0), dim=0)
        at = torch.searchsorted(torch.cumsum(q, 0), s["u"][i].double(), right=True)
        tokens[i] = int(kept[min(int(at), kept.numel() - 1)])
        if probs is not None:
            probs[i, kept] = q
    return {"tokens": tokens, "probs": probs} if case["probs"] else {"tokens": tokens}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "chunk": _exact_chunk, "sample": _exact_sample}[case["op"]](case, s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    e = _ITEM[case["dtype"]]
    if case["op"] == "norm":
        _, new = _lens(case)
        n = int(new.sum())
        heads = case["Hq"] + 2 * case["Hkv"]
        bytes_ = n * (2 * heads * case["D"] * e + 4 * case["rot"]) + 8 * case["B"]
        return {"bytes": bytes_, "flops": n * (4 * case["D"] + 3 * case["rot"]) * (case["Hq"] + case["Hkv"])}
    if case["op"] == "chunk":
        lens, new = _lens(case)
        pairs = keys = 0
        for c, n in zip(lens.tolist(), new.tolist()):
            p = np.arange(c, c + n, dtype=np.int64)
            first = np.maximum(0, p + 1 - case["window"]) if case["window"] else np.zeros_like(p)
            kept = np.minimum(case["sink"], first)
            pairs += int((p + 1 - first + kept).sum())
            keys += int(c + n - first[0] + kept[0])
        io = int(new.sum()) * case["Hq"] * (2 * case["D"] * e + 4)
        return {"bytes": keys * case["Hkv"] * case["D"] * 2 * e + io, "flops": 4 * pairs * case["Hq"] * case["D"]}
    n = case["R"] * case["V"]
    return {"bytes": n * (e + (4 if case["probs"] else 0)) + 24 * case["R"], "flops": 8 * n}
