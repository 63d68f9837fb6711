"""Cases of the operators that bound a long cache: attention with a sliding
window and sinks over the 4-bit KV cache, the attention weights summed for
every cached position, and the eviction of the positions with the smallest
sums.

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

GROUP = 32          # channels that share (step, lo)
FIFTEENTH = 1.0 / 15.0
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)  # bit of channel e in its word
DEVICE = "cuda"

WINDOW = {"op": "window", "tree": True, "page": 16, "sinks": 4}
SUMS = {"op": "sums", "page": 16, "commit": False}
EVICT = {"op": "evict", "sinks": 4}


def listed():
    return [
        # one request decoding one token far into its text: latency alone
        dict(WINDOW, name="window_one_token", B=1, N=1, Hq=32, Hkv=8, D=128, ctx_min=5000, ctx_max=5000, window=1024),
        # a decode batch, contexts from below the window to several times it
        dict(WINDOW, name="window_decode_batch", B=128, N=1, Hq=32, Hkv=8, D=128, ctx_min=16, ctx_max=8192, window=2048),
        # verification of 16-node trees: small heads, sizes that no tile divides
        dict(WINDOW, name="window_tree_16", B=64, N=16, Hq=12, Hkv=4, D=64, ctx_min=0, ctx_max=2047, page=5, sinks=7,
             window=509),
        # verification of the largest tree batch
        dict(WINDOW, name="window_tree_64", B=128, N=64, Hq=32, Hkv=8, D=128, ctx_min=16, ctx_max=8192, window=1024),
        # one request after one token: latency alone
        dict(SUMS, name="sums_one_token", B=1, N=1, Hq=32, Hkv=8, D=128, ctx_min=777, ctx_max=777),
        # a decode batch, each step's token
        dict(SUMS, name="sums_decode_batch", B=128, N=1, Hq=32, Hkv=8, D=128, ctx_min=16, ctx_max=2048),
        # after the verification of 64-node trees: the nodes of each accepted path
        dict(SUMS, name="sums_tree_commit", B=128, N=64, Hq=32, Hkv=8, D=128, ctx_min=16, ctx_max=2048, commit=True),
        # the last tokens of long prompts look back over the whole prompt
        dict(SUMS, name="sums_long_prompt", B=4, N=32, Hq=32, Hkv=8, D=128, ctx_min=60001, ctx_max=131001),
        # one request, its slots relabelled: latency alone
        dict(EVICT, name="evict_one", B=1, ctx_min=1500, ctx_max=1500, budget=1024, limit=1024, recent=128, page=1, row=0),
        # a batch whose longer half is cut, payload moved in pages
        dict(EVICT, name="evict_batch", B=128, ctx_min=16, ctx_max=2048, budget=768, limit=1024, recent=128, page=16,
             row=4096),
        # long prompts cut to a quarter, slots relabelled
        dict(EVICT, name="evict_long", B=4, ctx_min=60001, ctx_max=131001, budget=32768, limit=32768, recent=1024, page=1,
             row=0),
        # narrow rows, pages and sizes that nothing divides
        dict(EVICT, name="evict_pages_5", B=37, ctx_min=0, ctx_max=4093, budget=777, limit=1001, recent=129, sinks=3,
             page=5, row=320),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the listed ranges, no larger than the largest."""
    op = rng.choice(("window", "sums", "evict"))
    if op == "evict":
        ctx = _log_int(rng, 2, 131000)
        budget = _log_int(rng, 1, ctx)
        sinks = min(rng.choice((0, 1, 3, 4, 16)), budget)
        case = dict(EVICT, B=_log_int(rng, 1, 128), ctx_min=rng.randrange(0, ctx + 1), ctx_max=ctx, budget=budget,
                    limit=budget + rng.choice((0, 1, budget // 4)), sinks=sinks,
                    recent=min(_log_int(rng, 1, 1024) - 1, budget - sinks), page=rng.choice((1, 1, 5, 16, 64)), row=0)
        if case["page"] > 1:
            case["row"] = 16 * _log_int(rng, 5, 256)
    else:
        Hkv, ctx = rng.choice((1, 2, 3, 4, 8)), _log_int(rng, 1, 131000)
        case = dict(WINDOW if op == "window" else SUMS, B=_log_int(rng, 1, 128), N=_log_int(rng, 1, 64), Hkv=Hkv,
                    Hq=Hkv * rng.choice((1, 2, 3, 4, 5, 8)), D=rng.choice((64, 128)), ctx_min=rng.randrange(0, ctx + 1),
                    ctx_max=ctx, page=rng.choice((1, 5, 16, 64)))
        if op == "window":
            case.update(tree=rng.random() < 0.7, sinks=rng.choice((0, 1, 4, 7, 64)), window=_log_int(rng, 1, 4096))
        else:
            case.update(commit=rng.random() < 0.6)
    most = [work(c) for c in listed() if c["op"] == op]

    def too_large(c):
        w = work(c)
        held = c["B"] * (c["ctx_max"] + c.get("N", 0))
        wide = c["row"] if op == "evict" else c["Hkv"] * c["D"]
        # what the plain form holds at a time: scores, or decoded K
        seen = 0 if op == "evict" else c["B"] * min(c["ctx_max"], c.get("window", 1 << 30)) * max(
            c["N"] * c["Hq"], wide)
        return (w["bytes"] > max(m["bytes"] for m in most) or w["flops"] > max(max(m["flops"] for m in most), 1)
                or held * wide > 1.4e9 or seen > 6e8)

    while too_large(case) and case["B"] > 1:
        case["B"] = max(1, case["B"] // 2)
    while too_large(case) and case.get("N", 1) > 1:
        case["N"] = max(1, case["N"] // 2)
    while too_large(case):
        for name in ("ctx_min", "ctx_max", "budget", "limit", "sinks", "recent"):
            if name in case:
                case[name] = case[name] // 2
        if op == "evict":
            case["budget"], case["limit"] = max(1, case["budget"]), max(1, case["limit"], case["budget"])
    return case


# ------------------------------------------------------------------- inputs

def _lengths(case, g):
    """[B] int32 context lengths, evenly spread over the case's range in an
    order that the seed gives: their sum is the case's alone."""
    B = case["B"]
    at = torch.arange(B, device=DEVICE, dtype=torch.float64) / max(1, B - 1) if B > 1 else torch.ones(1, device=DEVICE)
    n = (case["ctx_min"] + at * (case["ctx_max"] - case["ctx_min"])).round().to(torch.int32)
    return n[torch.randperm(B, generator=g, device=DEVICE)].contiguous()


def _slot_table(case, g, more):
    """req_to_token [B, max_ctx] over a shuffled pool of pages, and the
    number of slots."""
    B, ps = case["B"], case["page"]
    pages = -(-max(1, case["ctx_max"] + more) // ps)
    perm = torch.randperm(B * pages, generator=g, device=DEVICE).to(torch.int32)
    pos = torch.arange(pages * ps, device=DEVICE, dtype=torch.int32)
    table = perm.view(B, pages)[:, (pos // ps).long()] * ps + pos % ps
    return table.contiguous(), B * pages * ps


def _tree(case, g):
    """tree_mask [B, N, N] uint8 (1 iff column m is n or an ancestor of n) and
    depths [B, N] (parents are drawn among the four nodes before, or each node
    hangs on the last)."""
    B, N = case["B"], case["N"]
    mask = torch.zeros((B, N, N), dtype=torch.uint8, device=DEVICE)
    mask[:, 0, 0] = 1
    rows = torch.arange(B, device=DEVICE)
    back = torch.randint(1, 5, (B, N), generator=g, device=DEVICE) if case["tree"] else torch.ones(
        (B, N), dtype=torch.int64, device=DEVICE)
    for n in range(1, N):
        mask[:, n] = mask[rows, (n - back[:, n]).clamp(min=0)]
        mask[:, n, n] = 1
    return mask, mask.sum(2, dtype=torch.int32) - 1


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device=DEVICE) * std


def _cache(slots, Hkv, D, g):
    """Pool rows of random K and V: K has a few strong channels in each head,
    as projections have; V has none."""
    strong = 1.0 + 3.0 * (torch.rand((1, Hkv, D), generator=g, device=DEVICE) < 0.05)
    pool = torch.empty((slots, Hkv * 5 * D // 4), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 27) // (Hkv * D))
    for a in range(0, slots, step):
        n = min(step, slots - a)
        pool[a:a + n] = _quantise(_normal((n, Hkv, D), g) * strong, _normal((n, Hkv, D), g))
    return pool


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 7919 + 29)
    return {"window": _prepare_window, "sums": _prepare_sums, "evict": _prepare_evict}[case["op"]](case, g)


def _prepare_window(case, g):
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    table, slots = _slot_table(case, g, N)
    mask, depth = _tree(case, g)
    lens = _lengths(case, g)
    return {"case": case, "pool": _cache(slots, Hkv, D, g), "table": table, "lens": lens, "mask": mask,
            "positions": (lens[:, None] + depth).contiguous(), "scale": 1.0 / math.sqrt(D),
            "q": _normal((B, N, Hq, D), g, 1.5).to(torch.bfloat16)}


def _prepare_sums(case, g):
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    table, slots = _slot_table(case, g, N)
    s = {"case": case, "pool": _cache(slots, Hkv, D, g), "table": table, "lens": _lengths(case, g),
         "q": _normal((B, N, Hq, D), g, 1.5).to(torch.bfloat16), "scale": 1.0 / math.sqrt(D),
         # what earlier steps have left
         "prev": torch.rand(table.shape, generator=g, device=DEVICE) ** 4 * 8.0,
         "out": torch.zeros(table.shape, device=DEVICE)}
    # accepted paths: the root and up to six nodes behind it (all rows without a verification)
    path = torch.rand((B, N), generator=g, device=DEVICE)
    path[:, 0] = -1.0
    length = torch.randint(0, min(7, N), (B,), generator=g, device=DEVICE) if case["commit"] else torch.full(
        (B,), N - 1, device=DEVICE)
    path = path.argsort(1).argsort(1)  # a random order of the nodes with the root first
    kept = path <= length[:, None]
    s["path"] = torch.where(kept, torch.arange(N, device=DEVICE), N).sort(1).values.clamp(max=N - 1).to(torch.int32)
    s["accepted"] = length.to(torch.int32)
    # the rows' lse, as the attention of the same rows has left it
    s["lse"] = torch.zeros((B, N, Hq), device=DEVICE)
    for b in range(B):
        n = int(s["lens"][b])
        rows = s["path"][b, :int(length[b]) + 1].long()
        R = rows.numel()
        k = _values(s["pool"][table[b, :n + R].long()], Hkv, D, 1)[0]          # [n + R, Hkv, D]
        q = s["q"][b, rows].float().view(R, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        score = torch.matmul(q, k.permute(1, 2, 0)).view(Hkv, R, Hq // Hkv, n + R) * s["scale"]
        hidden = torch.arange(n + R, device=DEVICE) > n + torch.arange(R, device=DEVICE)[:, None]
        score.masked_fill_(hidden[None, :, None], float("-inf"))
        s["lse"][b, rows] = torch.logsumexp(score, -1).permute(1, 0, 2).reshape(R, Hq)
    return s


def _prepare_evict(case, g):
    B = case["B"]
    table, slots = _slot_table(case, g, 0)
    lens = _lengths(case, g)
    # sums fall off steeply and differ by many powers of two; some positions were never looked at
    sums = torch.exp(_normal(table.shape, g, 3.0))
    sums = torch.where(torch.rand(table.shape, generator=g, device=DEVICE) < 0.02, 0.0, sums)
    state = {"case": case, "table": table, "lens": lens, "sums": sums, "after": torch.zeros_like(sums), "pool": None}
    if case["row"]:
        state["pool"] = torch.randint(0, 256, (slots, case["row"]), generator=g, device=DEVICE, dtype=torch.uint8)
    cap = B * max(1, table.shape[1] // case["page"])
    state["out"] = {"kept": torch.zeros((B, case["budget"]), dtype=torch.int32, device=DEVICE),
                    "freed": torch.zeros((cap,), dtype=torch.int32, device=DEVICE),
                    "num_freed": torch.zeros((1,), dtype=torch.int32, device=DEVICE),
                    "new_kv_len": torch.zeros((B,), dtype=torch.int32, device=DEVICE)}
    return state


# -------------------------------------------------------------- plain forms

def _groups(x):
    """codes [..., D] int64 and (step, lo) [..., D / 32] fp16 of rows [..., D]."""
    x = x.reshape(*x.shape[:-1], -1, GROUP)
    lo = x.amin(-1).half()
    step = ((x.amax(-1) - x.amin(-1)) * FIFTEENTH).half()
    at = (x - lo.float()[..., None]) * torch.reciprocal(step.float())[..., None]
    return at.round().clamp(0, 15).to(torch.int64).flatten(-2), step, lo


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


def _values(rows, Hkv, D, parts=2):
    """k, v [..., Hkv, D] fp32 that pool rows [..., bytes] stand for (the
    first ``parts`` of them)."""
    rows = rows.reshape(*rows.shape[:-1], Hkv, 5 * D // 4)
    shifts = torch.tensor(SHIFTS, device=rows.device, dtype=torch.int32)
    got = []
    for i in range(parts):
        word = rows[..., i * D // 2:(i + 1) * D // 2].contiguous().view(torch.int32)
        code = ((word[..., None] >> shifts) & 15).flatten(-2).float()
        meta = rows[..., D + i * D // 8:D + (i + 1) * D // 8].contiguous().view(torch.float16).float()
        step, lo = (meta[..., j::2].repeat_interleave(GROUP, -1) for j in (0, 1))
        got.append(lo + code * step)
    return got


def _plain_window(s):
    c = s["case"]
    B, N, Hq, Hkv, D, S, W = (c[k] for k in ("B", "N", "Hq", "Hkv", "D", "sinks", "window"))
    W0 = min(W - 1, c["ctx_max"])                                           # context positions of the root's window
    lens, depth = s["lens"].long()[:, None], (s["positions"] - s["lens"][:, None]).long()
    # the sinks, the window before the root, the nodes
    pos = torch.cat((torch.arange(S, device=DEVICE).expand(B, S), lens - W0 + torch.arange(W0, device=DEVICE),
                     lens + torch.arange(N, device=DEVICE)), 1)             # [B, L]
    L = pos.shape[1]
    kind = torch.cat((torch.zeros(S, device=DEVICE), torch.ones(W0, device=DEVICE), torch.full((N,), 2.0, device=DEVICE)))
    context = ((kind == 0) & (pos < lens)) | ((kind == 1) & (pos >= S))
    at = torch.where(kind < 2, pos, lens + depth[:, torch.arange(L, device=DEVICE).sub(S + W0).clamp(min=0)])
    near = (at[:, None, :] > s["positions"].long()[:, :, None] - W) | (at < S)[:, None, :]     # [B, N, L]
    on = torch.zeros((B, N, L), dtype=torch.bool, device=DEVICE)
    on[:, :, S + W0:] = s["mask"] != 0
    seen = near & (on | context[:, None, :])
    slot = s["table"].gather(1, pos.clamp(0, s["table"].shape[1] - 1)).long()
    k, v = _values(s["pool"][slot], Hkv, D)                                 # [B, L, Hkv, D]
    q = s["q"].float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]             # [B, Hkv, N * G, L]
    score = score.view(B, Hkv, N, Hq // Hkv, L).masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(B, Hkv, -1, L)
    o = torch.matmul(p, v.permute(0, 2, 1, 3))                              # [B, Hkv, N * G, D]
    return o.view(B, Hkv, N, -1, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(torch.bfloat16)


def _plain_sums(s):
    c = s["case"]
    B, N, Hq, Hkv, D = (c[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    L = s["table"].shape[1]
    R = min(7, N) if c["commit"] else N                                     # rows of an accepted path at most
    row = s["path"][:, :R].long()
    q = s["q"].float().gather(1, row[:, :, None, None].expand(B, R, Hq, D))
    lse = s["lse"].gather(1, row[:, :, None].expand(B, R, Hq)).view(B, R, Hkv, G)
    i, pos = torch.arange(R, device=DEVICE), torch.arange(L, device=DEVICE)
    lens = s["lens"].long()[:, None, None]
    seen = (pos <= lens + i[:, None]) & (i[:, None] <= s["accepted"].long()[:, None, None])    # [B, R, L]
    total = torch.zeros((B, L), device=DEVICE)
    for h in range(Hkv):
        rows = s["pool"][:, h * (5 * D // 4):(h + 1) * (5 * D // 4)]
        k = _values(rows[s["table"].long()], 1, D, 1)[0][:, :, 0]           # [B, L, D]
        score = torch.matmul(q[:, :, h * G:(h + 1) * G].reshape(B, R * G, D), k.transpose(1, 2)) * s["scale"]
        w = torch.exp(score.view(B, R, G, L) - lse[:, :, h, :, None])
        total += torch.where(seen[:, :, None], w, 0.0).sum((1, 2))
    inside = pos <= lens[:, 0] + s["accepted"].long()[:, None]
    s["out"].copy_(torch.where(inside, s["prev"] + total, s["out"]))
    return s["out"]


def _plain_evict(s):
    c, out = s["case"], s["out"]
    B, budget, S, recent, ps = (c[k] for k in ("B", "budget", "sinks", "recent", "page"))
    lens, table = s["lens"].long(), s["table"]
    L = table.shape[1]
    pos = torch.arange(L, device=DEVICE).expand(B, L)
    cut = lens > c["limit"]                                                 # [B]: requests that lose positions
    inside = pos < lens[:, None]
    held = (pos < S) | (pos >= lens[:, None] - recent)
    rank = torch.where(inside, torch.where(held, float("inf"), s["sums"]), float("-inf"))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :budget]
    keep = torch.zeros((B, L), dtype=torch.bool, device=DEVICE).scatter_(1, order, True)
    keep = torch.where(cut[:, None], keep, inside)
    width = min(budget, L)
    kept = torch.sort(order, dim=1).values                                  # [B, width]
    out["kept"].fill_(-1)
    out["kept"][:, :width] = torch.where(cut[:, None], kept, -1).to(torch.int32)
    new = torch.where(cut, budget, lens)
    out["new_kv_len"].copy_(new)
    s["after"].copy_(torch.where(inside, torch.where(cut[:, None], 0.0, s["sums"]), s["after"]))
    s["after"][:, :width] = torch.where(cut[:, None], s["sums"].gather(1, kept), s["after"][:, :width])
    if ps == 1:
        gone = inside & ~keep
        freed = table[gone]
        table[:, :width] = torch.where(cut[:, None], table.gather(1, kept), table[:, :width])
    else:
        page = torch.arange(-(-L // ps), device=DEVICE).expand(B, -1)
        gone = cut[:, None] & (page >= -(-new // ps)[:, None]) & (page < -(-lens // ps)[:, None])
        freed = (table[:, ::ps] // ps)[gone]
        rows = s["pool"][table.gather(1, kept)[cut].long()]
        s["pool"][table[:, :width][cut].long()] = rows
    out["num_freed"].fill_(freed.numel())
    out["freed"][:freed.numel()] = freed
    return _evict_outputs(s)


def _evict_outputs(s):
    got = dict(s["out"], table=s["table"], sums=s["after"])
    if s["pool"] is not None:
        got["pool"] = s["pool"]
    return got


def _own(s):
    import speculative_decoding_draft_select_gb300 as sd
    c = s["case"]
    if c["op"] == "window":
        return sd.spec_kv4_attention_window(s["q"], s["pool"], s["table"], s["lens"], c["Hkv"], c["sinks"], c["window"],
                                            positions=s["positions"], tree_mask=s["mask"], scale=s["scale"])
    if c["op"] == "sums":
        return sd.spec_kv4_weight_sums(s["q"], s["lse"], s["pool"], s["table"], s["lens"], c["Hkv"],
                                       accept_path=s["path"], accept_length=s["accepted"], prev=s["prev"], out=s["out"],
                                       scale=s["scale"])
    sd.spec_evict_slots(s["sums"], s["lens"], s["table"], c["page"], c["budget"], limit=c["limit"], sinks=c["sinks"],
                        recent=c["recent"], kv_pool=s["pool"], sums_out=s["after"], out=s["out"])
    return _evict_outputs(s)


def run(state):
    if own:
        return _own(state)
    return {"window": _plain_window, "sums": _plain_sums, "evict": _plain_evict}[state["case"]["op"]](state)


# --------------------------------------------------------------------- work

def _spread(case):
    """The case's context lengths, as _lengths spreads them."""
    B = case["B"]
    if B == 1:
        return [case["ctx_max"]]
    return [round(case["ctx_min"] + i / (B - 1) * (case["ctx_max"] - case["ctx_min"])) for i in range(B)]


def work(case):
    lens = _spread(case)
    B = case["B"]
    if case["op"] == "evict":
        total = 0
        for n in lens:
            # sums read and written
            total += 8 * n + 8
            if n > case["limit"]:
                # the slots read, the kept positions written; then new slots and freed ones, or rows moved
                total += 4 * n + 4 * case["budget"]
                if case["page"] == 1:
                    total += 4 * n
                else:
                    total += 4 * (n - case["budget"]) // case["page"]
                    total += 2 * max(0, case["budget"] - case["sinks"]) * case["row"]
        return {"bytes": total, "flops": 0}
    N, Hq, Hkv, D = (case[k] for k in ("N", "Hq", "Hkv", "D"))
    if case["op"] == "sums":
        rows = (min(7, N) + 1) / 2 if case["commit"] else N
        held = sum(lens) + B * rows
        return {"bytes": held * (Hkv * (D // 2 + D // 8) + 4 + 8) + B * rows * Hq * (2 * D + 4),
                "flops": 2 * held * rows * Hq * D}
    held = sum(min(n, case["sinks"] + case["window"] - 1) for n in lens) + B * N
    return {"bytes": held * (Hkv * 5 * D // 4 + 4) + B * (2 * N * Hq * D * 2 + N * N + 4 * N),
            "flops": 4 * held * N * Hq * D}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """run()'s results in 64 bits, request by request."""
    s = prepare(case, seed)
    return {"window": _exact_window, "sums": _exact_sums, "evict": _exact_evict}[case["op"]](case, s)


def _decode64(row, Hkv, D, which):
    """[T, Hkv, D] in 64 bits, K (which 0) or V (1) of pool rows [T, bytes],
    byte by byte."""
    byte = row.view(-1, Hkv, 5 * D // 4).to(torch.int64)
    channel = torch.arange(D, device=row.device)
    pair, odd = (channel % 8) // 2, channel % 2
    at = channel // 8 * 4 + odd * 2 + pair // 2
    code = (byte[:, :, which * D // 2 + at] >> (4 * (pair % 2))) & 15
    meta = D + which * D // 8
    half = byte[:, :, meta:meta + D // 8].to(torch.uint8).contiguous().view(torch.float16).double()
    return half[:, :, channel // GROUP * 2 + 1] + code * half[:, :, channel // GROUP * 2]


def _exact_window(case, s):
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device=DEVICE)
    for b in range(B):
        n = int(s["lens"][b])
        where = s["positions"][b].long()                                    # of the nodes
        first = torch.arange(n, device=DEVICE)
        first = first[(first < case["sinks"]) | (first > n - case["window"])]
        rows = s["pool"][torch.cat((s["table"][b, first], s["table"][b, n:n + N])).long()]
        k, v = _decode64(rows, Hkv, D, 0), _decode64(rows, Hkv, D, 1)
        at = torch.cat((first, where))
        see = torch.cat((torch.ones((N, first.numel()), dtype=torch.bool, device=DEVICE), s["mask"][b] != 0), 1)
        see &= (at < case["sinks"])[None] | (where[:, None] - at[None] < case["window"])
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            score = torch.einsum("nhd,ld->hnl", s["q"][b, :, heads].double(), k[:, h]) * s["scale"]
            p = torch.softmax(score.masked_fill(~see, float("-inf")), -1)
            out[b, :, heads] = torch.einsum("hnl,ld->nhd", p, v[:, h])
    return out


def _exact_sums(case, s):
    Hq, Hkv, D = (case[k] for k in ("Hq", "Hkv", "D"))
    out = s["out"].double()
    for b in range(case["B"]):
        n, R = int(s["lens"][b]), int(s["accepted"][b]) + 1
        row = s["path"][b, :R].long()
        k = _decode64(s["pool"][s["table"][b, :n + R].long()], Hkv, D, 0)
        out[b, :n + R] = s["prev"][b, :n + R].double()
        for h in range(Hq):
            score = s["q"][b, row, h].double() @ k[:, h // (Hq // Hkv)].T * s["scale"]
            w = torch.exp(score - s["lse"][b, row, h].double()[:, None]).tril(n)
            out[b, :n + R] += w.sum(0)
    return out


def _exact_evict(case, s):
    """Whole numbers and copies: the lists of each request put together on the host."""
    budget, ps = case["budget"], case["page"]
    table, pool = s["table"].clone(), None if s["pool"] is None else s["pool"].clone()
    after = s["after"].double()
    kept = torch.full_like(s["out"]["kept"], -1)
    new, freed = [], []
    for b in range(case["B"]):
        n = int(s["lens"][b])
        sums = s["sums"][b, :n].double()
        if n <= case["limit"]:
            new.append(n)
            after[b, :n] = sums
            continue
        first, last = case["sinks"], n - case["recent"]
        middle = torch.arange(first, last, device=DEVICE)
        # by falling sums, equal ones by rising position
        middle = middle[torch.argsort(-sums[first:last], stable=True)][:budget - case["sinks"] - case["recent"]]
        at = torch.cat((torch.arange(first, device=DEVICE), middle.sort().values, torch.arange(last, n, device=DEVICE)))
        kept[b] = at.to(torch.int32)
        new.append(budget)
        after[b, :budget], after[b, budget:n] = sums[at], 0.0
        if ps == 1:
            lost = torch.ones(n, dtype=torch.bool, device=DEVICE)
            lost[at] = False
            freed.append(s["table"][b, :n][lost])
            table[b, :budget] = s["table"][b, at]
        else:
            freed.append(s["table"][b, torch.arange(-(-budget // ps) * ps, n, ps, device=DEVICE)] // ps)
            pool[s["table"][b, :budget].long()] = s["pool"][s["table"][b, at].long()]
    everything = torch.cat(freed) if freed else torch.zeros(0, dtype=torch.int32, device=DEVICE)
    gone = s["out"]["freed"].clone()
    gone[:everything.numel()] = everything
    out = {"kept": kept, "freed": gone, "num_freed": torch.full_like(s["out"]["num_freed"], everything.numel()),
           "new_kv_len": torch.tensor(new, dtype=torch.int32, device=DEVICE), "table": table, "sums": after}
    if pool is not None:
        out["pool"] = pool
    return out
