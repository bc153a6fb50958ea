"""Oracle: commit of the accepted path's tree K/V to the paged cache, and
appending of new tokens' K/V (test infrastructure).

Definition followed
-------------------
"Build the tree attention mask that verifies a draft tree in one pass",
*What it costs.*: a serving system writes the tree's K/V to scratch and,
after verification, copies the accepted path into the cache.  "Tree
Verification" (stable-lab), *The Cost Side*: the accepted nodes' K/V rows
become the next step's prefix.

The accepted path of request b is ``path[b, 0 .. n_out[b] - 1]`` as the
acceptance step reports it: node ``path[b, 0]`` is the root (the last
accepted token of the previous step), and node ``path[b, j]`` sits at depth
j, i.e. at position ``L_b + j``.  Committing copies tree row
``path[b, j]`` (every KV head) into cache position ``L_b + j`` -- block
``block_table[b, (L_b + j) // block_size]``, slot
``(L_b + j) % block_size`` -- and the prefix length becomes
``L_b + n_out[b]``.  The tree keys are committed as given (the device path
stores them rotated at ``L_b + depth``, which is their cache position).
The token emitted after the last path node has no K/V yet: it is the next
step's root.

The pages define no failure; the library's reading (``stop_at_bad=True``):
a path step that cannot be committed -- a node outside the tree, a
position without a block in the table (or a table entry outside the
cache) -- ends the committed prefix there, so the prefix length never counts
a slot that was not written.
"""

from __future__ import annotations

import numpy as np

from .attention import rope


def commit_path(k_cache, v_cache, block_table, seq_lens, k_tree, v_tree, path, n_out, stop_at_bad=False):
    """Returns (k_cache', v_cache', seq_lens') with the accepted rows copied in.

    k_cache, v_cache [num_blocks, Hkv, block_size, D]; block_table
    [B, max_blocks]; seq_lens [B]; k_tree, v_tree [B, N, Hkv, D]; path
    [B, cols] node indices; n_out [B].  Raises if a position does not fit the
    block table, unless ``stop_at_bad``: then the first step that cannot be
    committed ends the request's commit (module docstring).
    """
    kc = np.array(k_cache, copy=True)
    vc = np.array(v_cache, copy=True)
    lens = np.array(seq_lens, dtype=np.int64, copy=True)
    bs = kc.shape[2]
    for b in range(lens.size):
        L = int(seq_lens[b])
        done = int(n_out[b])
        for j in range(int(n_out[b])):
            node = int(path[b, j])
            t = L + j
            fits = t // bs < block_table.shape[1] and 0 <= int(block_table[b, t // bs]) < kc.shape[0]
            if stop_at_bad and not (0 <= node < k_tree.shape[1] and fits):
                done = j
                break
            if t // bs >= block_table.shape[1]:
                raise ValueError(f"request {b}: position {t} beyond its block table")
            blk = int(block_table[b, t // bs])
            kc[blk, :, t % bs, :] = k_tree[b, node]
            vc[blk, :, t % bs, :] = v_tree[b, node]
        lens[b] = L + done
    return kc, vc, lens


def append_tokens(k_cache, v_cache, block_table, seq_lens, k_new, v_new, counts, q=None, rope_base=None,
                  max_pos=None):
    """New tokens' K/V appended to the paged cache: request b takes the next
    ``counts[b]`` rows of k_new / v_new [T, Hkv, D], row j at position
    ``L_b + j``, keys (and queries q [T, Hq, D]) rotated there when
    ``rope_base`` is given.  Returns (k_cache', v_cache', seq_lens', q').

    A token whose position is outside the rotary table (``max_pos`` rows) or
    without a valid block is not stored and ends the returned length; later
    tokens with a valid block are stored (their slots lie past the length).
    Queries past the table, and rows behind the last request, stay as given.
    """
    kc = np.array(k_cache, dtype=np.float64)
    vc = np.array(v_cache, dtype=np.float64)
    qo = None if q is None else np.array(q, dtype=np.float64)
    lens = np.array(seq_lens, dtype=np.int64, copy=True)
    bs = kc.shape[2]
    t = 0
    for b in range(lens.size):
        L, done = int(seq_lens[b]), None
        for j in range(int(counts[b])):
            pos = L + j
            ok = 0 <= L and (max_pos is None or pos < max_pos)
            if ok and qo is not None:
                qo[t] = rope(q[t], np.full(qo.shape[1], pos), rope_base)
            ok = ok and pos // bs < block_table.shape[1] and 0 <= int(block_table[b, pos // bs]) < kc.shape[0]
            if ok:
                blk = int(block_table[b, pos // bs])
                k = k_new[t] if rope_base is None else rope(k_new[t], np.full(kc.shape[1], pos), rope_base)
                kc[blk, :, pos % bs, :] = k
                vc[blk, :, pos % bs, :] = v_new[t]
            elif done is None:
                done = j
            t += 1
        lens[b] = L + (int(counts[b]) if done is None else done)
    return kc, vc, lens, qo


def norm_rows(x, weight, eps):
    """Rows x [..., D] divided by their root mean square (eps added to the mean square) and scaled by weight [D]."""
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def turn_rows(x, table, interleaved=False):
    """The leading R elements of rows x [T, H, D] turned by the angles' cos and sin, table [T, 2, R/2]: element i with
    i + R/2 or, interleaved, 2i with 2i + 1."""
    y = np.array(x, dtype=np.float64)
    half = table.shape[2]
    first, second = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                     else (slice(0, half), slice(half, 2 * half)))
    a, b = np.array(y[..., first]), np.array(y[..., second])
    c, s = (np.asarray(table, dtype=np.float64)[:, None, i] for i in (0, 1))
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y


def append_normed(k_cache, v_cache, block_table, seq_lens, k_new, v_new, counts, q=None, q_weight=None, k_weight=None,
                  eps=0.0, table=None, interleaved=False):
    """append_tokens of rows normalised per head (weights given) and turned by the rotary ``table`` [max_pos, 2, R/2]
    (None: not turned), every position within it.  Returns (k_cache', v_cache', seq_lens', q')."""
    counts = np.asarray(counts, dtype=np.int64)
    pos = np.concatenate([np.arange(L, L + n) for L, n in zip(seq_lens, counts)]).astype(np.int64)
    total = pos.size

    def done(x, weight):
        y = np.array(x, dtype=np.float64)
        z = y[:total] if weight is None else norm_rows(y[:total], weight, eps)
        y[:total] = z if table is None else turn_rows(z, np.asarray(table)[pos], interleaved)
        return y

    kc, vc, lens, _ = append_tokens(k_cache, v_cache, block_table, seq_lens, done(k_new, k_weight), v_new, counts)
    return kc, vc, lens, None if q is None else done(q, q_weight)
