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


def kv4_attention(q, rows, req_to_token, seq_lens, Hkv, scale, tree_mask=None, num_nodes=None, window=None, sinks=0,
                  positions=None):
    """Attention in 64 bits of q [B, N, Hq, D]: a dict of out [B, N, Hq, D],
    lse [B, N, Hq], and what error bounds need: mean_abs [B, N, Hq, D] (the
    weighted mean of |v|), dot_abs [B, N, Hq] (the largest |scale| sum |q| |k|
    of an attended position), part_abs (the largest |scale| (max |q| sum |k| +
    sum |q|)) and count [B, N, Hq] (attended positions).  Rows
    n >= num_nodes[b] are NaN.  A position whose slot is out of range is not
    attended; a request whose positions are out of range gives zeros.  With a
    window a node at position P sees, of this, the positions below sinks and
    those above P - window; P is seq_len + positions[b, n] - positions[b, 0]
    (positions [B, N], seq_len + n without; taken into [seq_len, seq_len + n])."""
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
        if window is not None:
            at = np.arange(s + nn)
            if positions is not None:
                depth = np.asarray(positions[b, :nn], np.int64)
                at[s:] = s + np.clip(depth - depth[0], 0, np.arange(nn))
            see &= (at < sinks)[None] | (at[None] > at[s:, None] - window)
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


def kv4_weight_sums(q, lse, rows, req_to_token, seq_lens, Hkv, scale, accept_path=None, accept_length=None, prev=None):
    """In 64 bits, a dict of sums [B, max_ctx], prev plus the weights w that each
    position receives, touched (the entries that are written), and what error
    bounds need, sums over the weights: w itself, parts = w |scale| sum |q| (|lo|
    + |k - lo|), far = w |scale| max |q| sum (|lo| + |k - lo|), size = w (|score|
    + |lse|), and count, their number."""
    q = np.asarray(q, np.float64)
    B, N, Hq, D = q.shape
    ctx = req_to_token.shape[1]
    total = np.zeros((B, ctx)) if prev is None else np.asarray(prev, np.float64).copy()
    r = {"sums": total, "touched": np.zeros((B, ctx), bool), "count": np.zeros((B, ctx), np.int64)}
    for name in ("w", "parts", "far", "size"):
        r[name] = np.zeros((B, ctx))
    for b in range(B):
        s, R = int(seq_lens[b]), N if accept_length is None else int(accept_length[b]) + 1
        if s < 0 or R < 1 or R > N or s + R > ctx:
            continue
        r["touched"][b, :s + R] = True
        slot = req_to_token[b, :s + R].astype(np.int64)
        there = (slot >= 0) & (slot < rows.shape[0])
        mine = rows[np.where(there, slot, 0)]
        k, _ = kv4_values(mine, Hkv, D)
        meta = np.ascontiguousarray(mine[:, :Hkv * head_bytes(D)].reshape(-1, Hkv, head_bytes(D))[..., D:D + D // 8])
        lo = meta.view(np.float16).astype(np.float64)[..., 1::2].repeat(GROUP, -1)
        part = np.abs(lo) + np.abs(k - lo)
        for i in range(R):
            n = i if accept_path is None else int(accept_path[b, i])
            if not 0 <= n < N:
                continue
            see = there & (np.arange(s + R) <= s + i)
            for h in range(Hq):
                z = float(lse[b, n, h])
                if not np.isfinite(z):
                    continue
                kv, qa = h // (Hq // Hkv), np.abs(q[b, n, h])
                score = k[:, kv] @ q[b, n, h] * scale
                w = np.where(see, np.exp(score - z), 0.0)
                total[b, :s + R] += w
                r["w"][b, :s + R] += w
                r["parts"][b, :s + R] += w * (part[:, kv] @ qa) * abs(scale)
                r["far"][b, :s + R] += w * part[:, kv].sum(-1) * qa.max() * abs(scale)
                r["size"][b, :s + R] += w * (np.abs(score) + abs(z))
                r["count"][b, :s + R] += see
    return r


def evict(sums, seq_lens, req_to_token, page, budget, limit, sinks, recent, rows=None):
    """A dict of what eviction leaves: kept, freed (a list), new_kv_len, table,
    sums and pool."""
    r = {"table": req_to_token.copy(), "sums": np.asarray(sums, np.float32).copy(),
         "pool": None if rows is None else rows.copy(), "freed": []}
    B, ctx = sums.shape
    r["kept"], r["new_kv_len"] = np.full((B, budget), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n = int(seq_lens[b])
        r["new_kv_len"][b] = n if 0 <= n <= ctx else -1
        if not limit < n <= ctx:
            continue
        value = np.where(np.isnan(sums[b, :n]), -np.inf, sums[b, :n])
        middle = sorted(range(sinks, n - recent), key=lambda p: (-value[p], p))[:budget - sinks - recent]
        kept = np.array(list(range(sinks)) + sorted(middle) + list(range(n - recent, n)))
        r["kept"][b], r["new_kv_len"][b] = kept, budget
        r["sums"][b, :n] = 0
        r["sums"][b, :budget] = sums[b, kept]
        slot = req_to_token[b]
        if page == 1:
            gone = np.ones(n, bool)
            gone[kept] = False
            r["freed"] += slot[:n][gone].tolist()
            r["table"][b, :budget] = slot[kept]
        else:
            r["freed"] += [max(-1, int(slot[p]) // page) for p in range(-(-budget // page) * page, n, page)]
            if rows is not None:
                ok = lambda s: 0 <= s < rows.shape[0]  # noqa: E731
                for i, p in enumerate(kept):
                    if ok(slot[p]) and ok(slot[i]):
                        r["pool"][slot[i]] = rows[slot[p]]
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
