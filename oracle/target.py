"""Plain statements of the target pass's operators over numpy arrays: the
4-bit KV cache, tree attention over it and the adjustment of target logits.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code
with the CUDA library.  Values that the definitions round (the cache's lo,
step and codes, the adjustment's fp32 operations) are computed in exactly
that precision, so results can be compared bit for bit; attention is in
64 bits.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
LIMIT = np.float32(57344.0)


def head_bytes(D: int) -> int:
    return D + D // 4


def _bit(D):
    """(byte, shift) of each channel's code within a head row's D / 2 bytes."""
    c = np.arange(D)
    bit = (c // 8) * 32 + 4 * ((c % 8) // 2) + 16 * (c % 2)
    return bit // 8, bit % 8


def kv4_groups(x):
    """(codes [..., D], step, lo [..., D / 32] fp16) of rows [..., D]."""
    x = np.asarray(x, np.float32)
    x = np.clip(np.where(np.isnan(x), np.float32(0), x), -LIMIT, LIMIT)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    lo = g.min(-1).astype(np.float16)
    step = ((g.max(-1) - g.min(-1)) * np.float32(1.0 / 15.0)).astype(np.float16)
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = np.float32(1.0) / step.astype(np.float32)
        at = np.rint((g - lo.astype(np.float32)[..., None]) * inv[..., None])
    code = np.where(step[..., None] > 0, np.clip(at, 0, 15), 0).astype(np.int64)
    return code.reshape(x.shape), step, lo


def kv4_rows(k, v):
    """Cache rows [T, Hkv * 5 D / 4] uint8 of k, v [T, Hkv, D]."""
    T, H, D = k.shape
    rows = np.zeros((T, H, head_bytes(D)), np.uint8)
    byte, shift = _bit(D)
    for i, x in enumerate((k, v)):
        code, step, lo = kv4_groups(x)
        codes = np.zeros((T, H, D // 2), np.int64)
        for c in range(D):
            codes[..., byte[c]] |= code[..., c] << shift[c]
        rows[..., i * D // 2:(i + 1) * D // 2] = codes
        meta = np.stack((step, lo), -1).reshape(T, H, -1)
        rows[..., D + i * D // 8:D + (i + 1) * D // 8] = np.ascontiguousarray(meta).view(np.uint8)
    return rows.reshape(T, -1)


def kv4_values(rows, H: int, D: int):
    """k, v [T, Hkv, D] fp64 that cache rows [T, bytes] stand for (exact)."""
    rows = np.ascontiguousarray(rows[:, :H * head_bytes(D)]).reshape(-1, H, head_bytes(D))
    byte, shift = _bit(D)
    out = []
    for i in range(2):
        code = (rows[..., i * D // 2:(i + 1) * D // 2][..., byte] >> shift) & 15
        meta = np.ascontiguousarray(rows[..., D + i * D // 8:D + (i + 1) * D // 8]).view(np.float16).astype(np.float64)
        out.append(meta[..., 1::2].repeat(GROUP, -1) + code * meta[..., 0::2].repeat(GROUP, -1))
    return out


def kv4_attention(q, rows, req_to_token, seq_lens, Hkv, scale, tree_mask=None, num_nodes=None):
    """Attention in 64 bits of q [B, N, Hq, D]: a dict of out [B, N, Hq, D],
    lse [B, N, Hq], and what error bounds need: mean_abs [B, N, Hq, D] (the
    weighted mean of |v|), dot_abs [B, N, Hq] (the largest |scale| sum |q| |k|
    of an attended position), part_abs (the largest |scale| (max |q| sum |k| +
    sum |q|)) and count [B, N, Hq] (attended positions).  Rows
    n >= num_nodes[b] are NaN.  A position whose slot is out of range is not
    attended; a request whose positions are out of range gives zeros."""
    q = np.asarray(q, np.float64)
    B, N, Hq, D = q.shape
    G = Hq // Hkv
    r = {"out": np.full((B, N, Hq, D), np.nan), "mean_abs": np.zeros((B, N, Hq, D)), "lse": np.full((B, N, Hq), np.nan),
         "dot_abs": np.zeros((B, N, Hq)), "part_abs": np.zeros((B, N, Hq)), "count": np.zeros((B, N, Hq), np.int64)}
    for b in range(B):
        nn = N if num_nodes is None else int(min(max(num_nodes[b], 0), N))
        s = int(seq_lens[b])
        r["out"][b, :nn], r["lse"][b, :nn] = 0.0, -np.inf
        if nn == 0 or s < 0 or s + nn > req_to_token.shape[1]:
            continue
        slot = req_to_token[b, :s + nn].astype(np.int64)
        there = (slot >= 0) & (slot < rows.shape[0])
        k, v = kv4_values(rows[np.where(there, slot, 0)], Hkv, D)
        see = np.ones((nn, s + nn), bool)
        see[:, s:] = np.tril(np.ones((nn, nn), bool)) if tree_mask is None else tree_mask[b, :nn, :nn] != 0
        see &= there
        for n in range(nn):
            at = np.flatnonzero(see[n])
            if at.size == 0:
                continue
            for h in range(Hkv):
                heads = slice(h * G, (h + 1) * G)
                kh, vh = k[at, h], v[at, h]
                score = (q[b, n, heads] @ kh.T) * scale
                m = score.max(-1, keepdims=True)
                p = np.exp(score - m)
                total = p.sum(-1, keepdims=True)
                r["out"][b, n, heads] = p @ vh / total
                r["mean_abs"][b, n, heads] = p @ np.abs(vh) / total
                r["lse"][b, n, heads] = (m + np.log(total))[:, 0]
                qa, ka = np.abs(q[b, n, heads]), np.abs(kh)
                r["dot_abs"][b, n, heads] = (qa @ ka.T).max(-1) * abs(scale)
                r["part_abs"][b, n, heads] = (qa.max(-1) * ka.sum(-1).max() + qa.sum(-1)) * abs(scale)
                r["count"][b, n, heads] = at.size
    return r


def adjust_logits(x, history=None, history_lens=None, prompt_lens=None, rep=None, freq=None, pres=None, draft=None,
                  tree_mask=None, bias_ids=None, bias_vals=None, allowed=None, allowed_row=None, num_nodes=None):
    """The adjusted fp32 values of logits x [B, N, V] (fp32 of their type),
    each operation in fp32; rows n >= num_nodes[b] are x."""
    f = np.float32
    x = np.asarray(x, f)
    B, N, V = x.shape
    out = x.copy()
    for b in range(B):
        nn = N if num_nodes is None else int(min(max(num_nodes[b], 0), N))
        r = f(1) if rep is None or not rep[b] > 0 else f(rep[b])
        fq, pr = (f(0) if t is None else f(t[b]) for t in (freq, pres))
        said, seen = np.zeros(V, np.int64), np.zeros(V, bool)
        if history is not None:
            n_h = history.shape[1] if history_lens is None else int(min(max(history_lens[b], 0), history.shape[1]))
            for i in range(n_h):
                t = int(history[b, i])
                if 0 <= t < V:
                    seen[t] = True
                    said[t] += prompt_lens is None or i >= prompt_lens[b]
        bias = {}
        if bias_ids is not None:
            for t, w in zip(bias_ids[b].tolist(), bias_vals[b]):
                if 0 <= t < V:
                    bias[t] = f(bias[t] + w) if t in bias else f(w)
        for n in range(nn):
            cnt, on = said.copy(), seen.copy()
            if draft is not None:
                for m in range(1, nn):
                    t = int(draft[b, m])
                    if (m <= n if tree_mask is None else tree_mask[b, n, m] != 0) and 0 <= t < V:
                        cnt[t] += 1
                        on[t] = True
            with np.errstate(all="ignore"):
                y = x[b, n].copy()
                y = np.where(on, np.where(y > 0, y / r, y * r), y)
                y = np.where(cnt > 0, y - cnt.astype(f) * fq - pr, y)
                for t, w in bias.items():
                    y[t] = y[t] + w
            if allowed is not None:
                row = b * N + n if allowed_row is None else int(allowed_row[b, n])
                if 0 <= row < allowed.shape[0]:
                    v = np.arange(V)
                    y = np.where((allowed[row][v // 32].astype(np.int64) >> (v % 32)) & 1, y, f(-np.inf))
            out[b, n] = y
    return out
