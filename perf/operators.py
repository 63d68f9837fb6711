"""Cases of the target pass's operators: the 4-bit KV cache (append and read
back), tree attention over it, and the adjustment of the target logits.

Each case names one operator ("op") and its sizes.  ``run`` computes it in
elementary torch operations (``own`` false) or with the framework's calls
(``own`` true); ``exact`` states the same results in 64 bits.

Cache rows.  A pool row (slot) holds, per KV head, the codes of K (D/2
bytes), the codes of V (D/2 bytes), then the fp16 pairs (step, lo) of K's
groups of 32 channels and of V's: 5 D / 4 bytes.  Eight channels share a
little-endian 32-bit word, channel 2j in bits [4j, 4j + 4) and channel 2j + 1
16 bits higher.  A code c stands for lo + c * step.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 32          # channels that share (step, lo)
LIMIT = 57344.0     # values beyond it saturate: every code's value is finite in fp16
FIFTEENTH = 1.0 / 15.0
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)  # bit of channel e in its word
DEVICE = "cuda"

ATTENTION = {"op": "attention", "tree": True, "page": 16}
CACHE = {"op": "cache", "page": 16}
LOGITS = {"op": "logits", "history": 1024, "bias": 64, "grammar": 0.5}


def listed():
    return [
        # one request decoding one token over a short context: latency alone
        dict(ATTENTION, name="attention_one_token", B=1, N=1, Hq=32, Hkv=8, D=128, ctx_min=777, ctx_max=777),
        # a decode batch at the step benchmark's context lengths
        dict(ATTENTION, name="attention_decode_batch", B=128, N=1, Hq=32, Hkv=8, D=128, ctx_min=16, ctx_max=2048),
        # few requests over long contexts: the work has to be split along the cache
        dict(ATTENTION, name="attention_long_context", B=4, N=1, Hq=64, Hkv=8, D=128, ctx_min=60001, ctx_max=131001),
        # greedy verification of 16-node trees, small heads, one page size that no tile divides
        dict(ATTENTION, name="attention_tree_16", B=64, N=16, Hq=12, Hkv=4, D=64, ctx_min=0, ctx_max=2047, page=5),
        # stochastic verification of 64-node trees, the step benchmark's largest tree batch
        dict(ATTENTION, name="attention_tree_64", B=128, N=64, Hq=32, Hkv=8, D=128, ctx_min=16, ctx_max=2048),
        # single tokens written into the cache, as each decode step does
        dict(CACHE, name="cache_decode_batch", B=128, N=1, Hkv=8, D=128, dtype="bf16", ctx_min=16, ctx_max=2048),
        # the nodes of 64-node trees written before their verification
        dict(CACHE, name="cache_tree_64", B=128, N=64, Hkv=8, D=128, dtype="bf16", ctx_min=16, ctx_max=2048),
        # long prompts of an odd length from an fp32 projection, small heads
        dict(CACHE, name="cache_prompt", B=7, N=8191, Hkv=4, D=64, dtype="f32", ctx_min=0, ctx_max=1023),
        # one request decoding one token: latency alone
        dict(LOGITS, name="logits_one_row", B=1, N=1, V=32000, dtype="bf16", history=300),
        # fp32 logits of short chains over a vocabulary of an odd size
        dict(LOGITS, name="logits_chain_odd", B=96, N=5, V=50257, dtype="f32"),
        # every node under a grammar, long histories
        dict(LOGITS, name="logits_tree_16", B=64, N=16, V=32000, dtype="bf16", history=8000, grammar=1.0),
        # the step benchmark's largest target logits
        dict(LOGITS, name="logits_tree_64", B=128, N=64, V=128256, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the listed ranges, no larger than the largest."""
    op = rng.choice(("attention", "cache", "logits"))
    most = {"attention": work(listed()[4]), "cache": work(listed()[6]), "logits": work(listed()[11])}[op]
    if op == "attention":
        Hkv, ctx = rng.choice((1, 2, 3, 4, 8)), _log_int(rng, 1, 131000)
        case = dict(ATTENTION, B=_log_int(rng, 1, 128), N=_log_int(rng, 1, 64), Hkv=Hkv,
                    Hq=Hkv * rng.choice((1, 2, 3, 4, 5, 8)), D=rng.choice((64, 128)), ctx_min=rng.randrange(0, ctx + 1),
                    ctx_max=ctx, page=rng.choice((1, 5, 16, 64)), tree=rng.random() < 0.7)
    elif op == "cache":
        case = dict(CACHE, B=_log_int(rng, 1, 128), N=_log_int(rng, 1, 8191), Hkv=rng.choice((1, 2, 3, 4, 8)),
                    D=rng.choice((64, 128)), dtype=rng.choice(("bf16", "f32")), ctx_min=rng.randrange(0, 16),
                    ctx_max=_log_int(rng, 16, 2048), page=rng.choice((1, 5, 16, 64)))
    else:
        case = dict(LOGITS, B=_log_int(rng, 1, 128), N=_log_int(rng, 1, 64), V=_log_int(rng, 32, 152000),
                    dtype=rng.choice(("bf16", "f32")), history=_log_int(rng, 1, 8000), bias=rng.randrange(0, 200),
                    grammar=rng.choice((0.0, 0.5, 1.0)))
        case["bias"] = min(case["bias"], case["V"])

    def too_large(c):
        w = work(c)
        slots = c["B"] * (c.get("ctx_max", 0) + c["N"]) * c.get("Hkv", 0) * c.get("D", 0)
        return w["bytes"] > most["bytes"] or w["flops"] > max(most["flops"], 1) or slots > 6e8

    while too_large(case) and case["B"] > 1:
        case["B"] = max(1, case["B"] // 2)
    while too_large(case):
        case["N"] = max(1, case["N"] // 2)
    return case


# ------------------------------------------------------------------- inputs

def _lengths(case, g):
    """[B] int32 context lengths, evenly spread over the case's range in an
    order that the seed gives: their sum is the case's alone."""
    B = case["B"]
    at = torch.arange(B, device=DEVICE, dtype=torch.float64) / max(1, B - 1) if B > 1 else torch.ones(1, device=DEVICE)
    n = (case["ctx_min"] + at * (case["ctx_max"] - case["ctx_min"])).round().to(torch.int32)
    return n[torch.randperm(B, generator=g, device=DEVICE)].contiguous()


def _slot_table(case, g):
    """req_to_token [B, max_ctx] over a shuffled pool of pages, and the
    number of slots."""
    B, ps = case["B"], case["page"]
    pages = -(-(case["ctx_max"] + case["N"]) // ps)
    perm = torch.randperm(B * pages, generator=g, device=DEVICE).to(torch.int32)
    pos = torch.arange(pages * ps, device=DEVICE, dtype=torch.int32)
    table = perm.view(B, pages)[:, (pos // ps).long()] * ps + pos % ps
    return table.contiguous(), B * pages * ps


def _tree_mask(case, g):
    """[B, N, N] uint8: 1 iff column m is n or an ancestor of n (parents are
    drawn among the four nodes before, or each node hangs on the last)."""
    B, N = case["B"], case["N"]
    mask = torch.zeros((B, N, N), dtype=torch.uint8, device=DEVICE)
    mask[:, 0, 0] = 1
    rows = torch.arange(B, device=DEVICE)
    back = torch.randint(1, 5, (B, N), generator=g, device=DEVICE) if case["tree"] else torch.ones(
        (B, N), dtype=torch.int64, device=DEVICE)
    for n in range(1, N):
        mask[:, n] = mask[rows, (n - back[:, n]).clamp(min=0)]
        mask[:, n, n] = 1
    return mask


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 7919 + 17)
    return {"attention": _prepare_attention, "cache": _prepare_cache, "logits": _prepare_logits}[case["op"]](case, g)


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device=DEVICE) * std


def _prepare_attention(case, g):
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    table, slots = _slot_table(case, g)
    # K has a few strong channels in each head, as projections have; V has none
    strong = 1.0 + 3.0 * (torch.rand((1, Hkv, D), generator=g, device=DEVICE) < 0.05)
    pool = torch.empty((slots, Hkv * 5 * D // 4), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 27) // (Hkv * D))
    for a in range(0, slots, step):
        n = min(step, slots - a)
        pool[a:a + n] = _quantise(_normal((n, Hkv, D), g) * strong, _normal((n, Hkv, D), g))
    return {"case": case, "pool": pool, "table": table, "lens": _lengths(case, g),
            "q": _normal((B, N, Hq, D), g, 1.5).to(torch.bfloat16), "mask": _tree_mask(case, g),
            "scale": 1.0 / math.sqrt(D)}


def _prepare_cache(case, g):
    B, N, Hkv, D = (case[k] for k in ("B", "N", "Hkv", "D"))
    dtype = DTYPES[case["dtype"]]
    table, slots = _slot_table(case, g)
    # K and V lie beside one another in the projection's output
    kv = _normal((B, N, 2, Hkv, D), g).to(dtype)
    return {"case": case, "pool": torch.zeros((slots, Hkv * 5 * D // 4), dtype=torch.uint8, device=DEVICE),
            "table": table, "lens": _lengths(case, g), "k": kv[:, :, 0], "v": kv[:, :, 1]}


def _prepare_logits(case, g):
    B, N, V, H, M = (case[k] for k in ("B", "N", "V", "history", "bias"))
    # text repeats itself: ids crowd towards the front of the vocabulary
    ids = lambda *shape: (torch.rand(shape, generator=g, device=DEVICE) ** 4 * V).to(torch.int32).clamp(max=V - 1)  # noqa: E731
    logits = torch.empty((B, N, V), dtype=DTYPES[case["dtype"]], device=DEVICE)
    for b in range(B):
        logits[b] = _normal((N, V), g, 3.0)
    state = {"case": case, "logits": logits, "history": ids(B, H), "draft": ids(B, N),
             "mask": _tree_mask({"B": B, "N": N, "tree": True}, g),
             "history_lens": torch.randint(H // 2, H + 1, (B,), generator=g, device=DEVICE, dtype=torch.int32),
             "prompt_lens": torch.randint(0, H // 2 + 1, (B,), generator=g, device=DEVICE, dtype=torch.int32),
             "rep": 1.0 + 0.5 * torch.rand(B, generator=g, device=DEVICE),
             "freq": 0.5 * torch.rand(B, generator=g, device=DEVICE),
             "pres": 0.5 * torch.rand(B, generator=g, device=DEVICE)}
    # each request's bias list names distinct ids
    first = torch.randint(0, V, (B, 1), generator=g, device=DEVICE)
    apart = max(1, V // max(1, M))
    state["bias_ids"] = ((first + torch.arange(M, device=DEVICE) * apart) % V).to(torch.int32).contiguous()
    state["bias_vals"] = _normal((B, M), g, 4.0)
    # a share of the requests decodes under a grammar: each of its nodes has a
    # row of allowed ids, from a handful to almost all
    words = (V + 31) // 32
    held = torch.rand((B, 1), generator=g, device=DEVICE) < case["grammar"]
    row = torch.where(held, torch.arange(B * N, device=DEVICE).view(B, N), -1)
    dense = torch.randint(-2**31, 2**31, (B * N, words), generator=g, device=DEVICE, dtype=torch.int64)
    for _ in range(3):
        more = torch.randint(-2**31, 2**31, (B * N, words), generator=g, device=DEVICE, dtype=torch.int64)
        keep = torch.rand((B * N, 1), generator=g, device=DEVICE) < 0.5
        dense = torch.where(keep, dense & more, dense | more)
    state["allowed"], state["allowed_row"] = dense.to(torch.int32), row.to(torch.int32).contiguous()
    return state


# -------------------------------------------------------------- plain forms

def _groups(x):
    """codes [..., D] int64 and (step, lo) [..., D / 32] fp16 of rows [..., D]."""
    x = torch.nan_to_num(x.float(), nan=0.0).clamp(-LIMIT, LIMIT)
    x = x.reshape(*x.shape[:-1], -1, GROUP)
    lo = x.amin(-1).half()
    step = ((x.amax(-1) - x.amin(-1)) * FIFTEENTH).half()
    at = (x - lo.float()[..., None]) * torch.reciprocal(step.float())[..., None]
    code = torch.where(step[..., None] > 0, at.round().clamp(0, 15), torch.zeros_like(at)).to(torch.int64)
    return code.flatten(-2), step, lo


def _quantise(k, v):
    """Pool rows [T, Hkv * 5 D / 4] uint8 of k, v [T, Hkv, D]."""
    parts, metas = [], []
    shifts = torch.tensor(SHIFTS, device=k.device, dtype=torch.int64)
    for x in (k, v):
        code, step, lo = _groups(x)
        word = (code.reshape(*code.shape[:-1], -1, 8) << shifts).sum(-1)
        word = torch.where(word >= 2**31, word - 2**32, word).to(torch.int32)
        parts.append(word.contiguous().view(torch.uint8))
        metas.append(torch.stack((step, lo), -1).flatten(-2).contiguous().view(torch.uint8))
    return torch.cat(parts + metas, -1).flatten(1)


def _values(rows, Hkv, D):
    """k, v [..., Hkv, D] fp32 that pool rows [..., bytes] stand for."""
    rows = rows.reshape(*rows.shape[:-1], Hkv, 5 * D // 4)
    shifts = torch.tensor(SHIFTS, device=rows.device, dtype=torch.int32)
    got = []
    for i in range(2):
        word = rows[..., i * D // 2:(i + 1) * D // 2].contiguous().view(torch.int32)
        code = ((word[..., None] >> shifts) & 15).flatten(-2).float()
        meta = rows[..., D + i * D // 8:D + (i + 1) * D // 8].contiguous().view(torch.float16).float()
        step, lo = (meta[..., j::2].repeat_interleave(GROUP, -1) for j in (0, 1))
        got.append(lo + code * step)
    return got


def _plain_attention(s):
    c = s["case"]
    B, N, Hq, Hkv, D = (c[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    L = s["table"].shape[1]
    k, v = _values(s["pool"][s["table"].long()], Hkv, D)                    # [B, L, Hkv, D]
    q = s["q"].float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]             # [B, Hkv, N * G, L]
    pos = torch.arange(L, device=q.device)
    node = pos - s["lens"][:, None].long()                                  # [B, L]
    inside = s["mask"].gather(2, node.clamp(0, N - 1)[:, None, :].expand(B, N, L)) != 0
    seen = (node < 0)[:, None, :] | (inside & (node < N)[:, None, :])       # [B, N, L]
    seen = seen[:, None, :, None, :].expand(B, Hkv, N, Hq // Hkv, L).reshape(score.shape)
    score = torch.where(seen, score, float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = torch.matmul(p / p.sum(-1, keepdim=True), v.permute(0, 2, 1, 3))    # [B, Hkv, N * G, D]
    return o.view(B, Hkv, N, -1, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(torch.bfloat16)


def _plain_cache(s):
    c = s["case"]
    B, N, Hkv, D = (c[k] for k in ("B", "N", "Hkv", "D"))
    at = s["lens"][:, None].long() + torch.arange(N, device=DEVICE)
    slot = s["table"].gather(1, at).long()
    s["pool"][slot.flatten()] = _quantise(s["k"].reshape(-1, Hkv, D), s["v"].reshape(-1, Hkv, D))
    k, v = _values(s["pool"][slot], Hkv, D)
    return {"k": k.to(s["k"].dtype), "v": v.to(s["v"].dtype)}


def _adjust(x, count, seen, rep, freq, pres, bias):
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - count * freq
    x = x - (count > 0) * pres
    return x + bias


def _plain_logits(s):
    c = s["case"]
    B, N, V = c["B"], c["N"], c["V"]
    at = torch.arange(s["history"].shape[1], device=DEVICE)
    told = at < s["history_lens"][:, None]
    answered = told & (at >= s["prompt_lens"][:, None])
    ids = s["history"].long()
    count = torch.zeros((B, V), device=DEVICE).scatter_add_(1, ids, answered.float())
    seen = torch.zeros((B, V), device=DEVICE).scatter_add_(1, ids, told.float()) > 0
    bias = torch.zeros((B, V), device=DEVICE).scatter_(1, s["bias_ids"].long(), s["bias_vals"])
    one = lambda name: s[name][:, None, None]  # noqa: E731
    x = s["logits"].float()
    got = _adjust(x, count[:, None], seen[:, None], one("rep"), one("freq"), one("pres"), bias[:, None])
    # the tokens of a node's path (without the root, which the history has)
    tok = s["draft"].long()
    path = s["mask"].float()
    path[:, :, 0] = 0
    extra = torch.matmul(path, (tok[:, :, None] == tok[:, None, :]).float())   # [B, N, N]: of node m's token
    col = tok[:, None, :].expand(B, N, N)
    base = count.gather(1, tok)[:, None, :] + extra
    was = seen.gather(1, tok)[:, None, :] | (extra > 0)
    fixed = _adjust(x.gather(2, col), base, was, one("rep"), one("freq"), one("pres"), bias.gather(1, tok)[:, None, :])
    got.scatter_(2, col, fixed)
    bits = (s["allowed"][..., None] >> torch.arange(32, device=DEVICE, dtype=torch.int32)) & 1
    allowed = bits.flatten(1)[:, :V].bool()
    row = s["allowed_row"].long()
    free = (row < 0)[..., None] | allowed[row.clamp(min=0)]
    return torch.where(free, got, float("-inf")).to(s["logits"].dtype)


def _own(s):
    import speculative_decoding_draft_select_gb300 as sd
    c = s["case"]
    if c["op"] == "attention":
        return sd.spec_kv4_attention(s["q"], s["pool"], s["table"], s["lens"], c["Hkv"], tree_mask=s["mask"],
                                     scale=s["scale"])
    if c["op"] == "cache":
        sd.spec_kv4_append(s["k"], s["v"], s["pool"], s["table"], s["lens"])
        k, v = sd.spec_kv4_gather(s["pool"], s["table"], s["lens"], c["N"], c["Hkv"], c["D"], dtype=s["k"].dtype)
        return {"k": k, "v": v}
    return sd.spec_adjust_logits(s["logits"], history=s["history"], history_lens=s["history_lens"],
                                 prompt_lens=s["prompt_lens"], rep_penalty=s["rep"], freq_penalty=s["freq"],
                                 pres_penalty=s["pres"], draft_token=s["draft"], tree_mask=s["mask"],
                                 bias_ids=s["bias_ids"], bias_vals=s["bias_vals"], allowed=s["allowed"],
                                 allowed_row=s["allowed_row"], out=torch.empty_like(s["logits"]))


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "cache": _plain_cache, "logits": _plain_logits}[state["case"]["op"]](state)


# --------------------------------------------------------------------- work

def work(case):
    B, N = case["B"], case["N"]
    if case["op"] == "logits":
        size = 2 if case["dtype"] == "bf16" else 4
        words = B * N * ((case["V"] + 31) // 32) * case["grammar"]
        return {"bytes": 2 * B * N * case["V"] * size + 4 * words + B * (0.75 * case["history"] * 4 + 8 * case["bias"])
                + B * N * (8 + N), "flops": 0}
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "cache":
        size = 2 if case["dtype"] == "bf16" else 4
        # k and v read, their rows written and read, k and v written
        return {"bytes": B * N * (Hkv * (4 * D * size + 2 * 5 * D // 4) + 4), "flops": 0}
    ctx = case["ctx_max"] if B == 1 else (case["ctx_min"] + case["ctx_max"]) / 2
    return {"bytes": B * ((ctx + N) * (Hkv * 5 * D // 4 + 4) + 2 * N * case["Hq"] * D * 2 + N * N),
            "flops": 4 * B * N * case["Hq"] * D * (ctx + N)}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """run()'s results in 64 bits, request by request."""
    s = prepare(case, seed)
    return {"attention": _exact_attention, "cache": _exact_cache, "logits": _exact_logits}[case["op"]](case, s)


def _decode64(row, Hkv, D):
    """k, v [T, Hkv, D] in 64 bits of pool rows [T, bytes], byte by byte."""
    byte = row.view(-1, Hkv, 5 * D // 4).to(torch.int64)
    channel = torch.arange(D, device=row.device)
    pair, odd = (channel % 8) // 2, channel % 2
    at = channel // 8 * 4 + odd * 2 + pair // 2
    found = []
    for first, meta in ((0, D), (D // 2, D + D // 8)):
        code = (byte[:, :, first + at] >> (4 * (pair % 2))) & 15
        half = byte[:, :, meta:meta + D // 8].to(torch.uint8).contiguous().view(torch.float16).double()
        found.append(half[:, :, channel // GROUP * 2 + 1] + code * half[:, :, channel // GROUP * 2])
    return found


def _exact_attention(case, s):
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device=DEVICE)
    for b in range(B):
        n = int(s["lens"][b])
        k, v = _decode64(s["pool"][s["table"][b, :n + N].long()], Hkv, D)
        see = torch.cat((torch.ones((N, n), dtype=torch.bool, device=DEVICE), s["mask"][b] != 0), 1)
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            score = torch.einsum("nhd,ld->hnl", s["q"][b, :, heads].double(), k[:, h]) * s["scale"]
            p = torch.softmax(score.masked_fill(~see, float("-inf")), -1)
            out[b, :, heads] = torch.einsum("hnl,ld->nhd", p, v[:, h])
    return out


def _exact_cache(case, s):
    """The values that the rows stand for: lo and step are fp16 by the
    cache's definition, the codes whole numbers."""
    found = {}
    for name in ("k", "v"):
        x = s[name].double().unflatten(-1, (-1, GROUP))
        lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
        step = ((hi.float() - lo.float()) * FIFTEENTH).half().double()
        lo = lo.half().double()
        # the codes are whole numbers of a 32-bit product by definition
        code = ((x.float() - lo.float()) * (1.0 / step.float())).round().clamp(0, 15).double()
        found[name] = (lo + code * step).flatten(-2)
    return found


def _exact_logits(case, s):
    B, N, V = case["B"], case["N"], case["V"]
    out = torch.empty((B, N, V), dtype=torch.float64, device=DEVICE)
    bit = torch.arange(V, device=DEVICE)
    for b in range(B):
        h = s["history"][b, :int(s["history_lens"][b])].long()
        p = int(s["prompt_lens"][b])
        said = torch.bincount(h[p:], minlength=V)
        known = torch.bincount(h, minlength=V) > 0
        tok = s["draft"][b].long()
        count = said.repeat(N, 1)
        on = s["mask"][b].long()
        on[:, 0] = 0
        count.scatter_add_(1, tok.repeat(N, 1), on)
        known = known | (count > 0)
        x = s["logits"][b].double()
        r, f, a = (s[name][b].double() for name in ("rep", "freq", "pres"))
        x = torch.where(known & (x > 0), x / r, torch.where(known, x * r, x)) - f * count - a * (count > 0).double()
        x.index_add_(1, s["bias_ids"][b].long(), s["bias_vals"][b].double().repeat(N, 1))
        row = s["allowed_row"][b].long()
        ok = (s["allowed"][row.clamp(min=0)][:, bit // 32] >> (bit % 32).int()) & 1
        out[b] = x.masked_fill((ok == 0) & (row >= 0)[:, None], float("-inf"))
    return out
