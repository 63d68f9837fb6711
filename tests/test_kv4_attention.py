"""spec_kv4_attention against attention in 64 bits over the same cache rows.

The bounds count roundings (half a step, relative: fp16 2^-11, fp32 2^-24,
bf16 2^-8; below fp16's normal range 2^-25 absolute).  A score
scale sum_D q k takes k in fp16, q in fp16 after a division by a power of two
near its row's largest element, and D products, D sums and a few factors in
fp32:
  |dx| <= E = dot_abs (2^-11 + (2 D + 8) 2^-24) + part_abs 2^-25.
A weight exp(x - max) is then off by a factor 1 + d, |d| <= e^E - 1 + 2^-20
(the exponential's approximation, fp32 products), its fp16 form by 2^-11 more
(the sum that divides does not have this one), v by 2^-11, sums of n terms by
n 2^-24 each.  A quotient of sums whose non-negative weights are off by a
relative a in the numerator and b in the denominator moves by at most
(a + b) / (1 - b) mean|v|.  The result rounds to bf16."""
import ctypes
import math

import numpy as np
import pytest
import torch

import speculative_decoding_draft_select_gb300 as sd
from oracle import target as ref
from speculative_decoding_draft_select_gb300.build import build


def slot_table(rng, B, max_ctx, page):
    pages = -(-max_ctx // page)
    perm = rng.permutation(B * pages).reshape(B, pages)
    pos = np.arange(max_ctx)
    return np.ascontiguousarray(perm[:, pos // page] * page + pos % page, np.int32), B * pages * page


def tree_masks(rng, B, N):
    mask = np.zeros((B, N, N), np.uint8)
    mask[:, 0, 0] = 1
    for b in range(B):
        for n in range(1, N):
            mask[b, n] = mask[b, rng.integers(0, n)]
            mask[b, n, n] = 1
    return mask


def make_case(seed, B, N, Hq, Hkv, D, lens, page=16, spread=1.5, tree=True):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    table, slots = slot_table(rng, B, max(1, int(lens.max()) + N), page)
    k = rng.normal(0, 1, (slots, Hkv, D)).astype(np.float32) + rng.normal(0, 1, (1, Hkv, D)).astype(np.float32)
    v = rng.normal(0, 1, (slots, Hkv, D)).astype(np.float32)
    return {"rows": ref.kv4_rows(k, v), "table": table, "lens": lens, "Hkv": Hkv, "scale": D ** -0.5,
            "mask": tree_masks(rng, B, N) if tree else None,
            "q": torch.from_numpy(rng.normal(0, spread, (B, N, Hq, D)).astype(np.float32)).to(torch.bfloat16)}


def run(c, q=None, lse=True, **kw):
    q = c["q"].cuda() if q is None else q
    got_lse = torch.full(c["q"].shape[:3], 77.0, device="cuda") if lse else None
    out = sd.spec_kv4_attention(q, torch.from_numpy(c["rows"]).cuda(), torch.from_numpy(c["table"]).cuda(),
                                torch.from_numpy(c["lens"]).cuda(), c["Hkv"], scale=c["scale"], lse=got_lse,
                                tree_mask=None if c["mask"] is None else torch.from_numpy(c["mask"]).cuda(), **kw)
    return out, got_lse


def expected(c, num_nodes=None):
    return ref.kv4_attention(c["q"].float().numpy(), c["rows"], c["table"], c["lens"], c["Hkv"], c["scale"],
                             tree_mask=c["mask"], num_nodes=num_nodes)


def score_error(r, D):
    return r["dot_abs"] * (2.0**-11 + (2 * D + 8) * 2.0**-24) + r["part_abs"] * 2.0**-25


def check(out, lse, r, rows=None):
    """rows: a boolean [B, N] of the rows that count (all by default)."""
    D = out.shape[-1]
    rows = np.ones(out.shape[:2], bool) if rows is None else rows
    E = score_error(r, D)
    n = r["count"]
    below = np.expm1(E) + 2.0**-20 + n * 2.0**-24
    above = below + 2 * 2.0**-11 * (1 + below)
    move = ((above + below) / np.maximum(1 - below, 0.01))[..., None] * r["mean_abs"] + 2.0**-25
    bound = move + 2.0**-8 * (np.abs(r["out"]) + move)
    got = out.float().cpu().numpy().astype(np.float64)
    off = np.abs(got - r["out"]) - bound
    assert (off[rows] <= 0).all(), f"worst excess {np.nanmax(off[rows])}, bound there {bound[rows].flat[np.nanargmax(off[rows])]}"
    if lse is not None:
        w, g = r["lse"][rows], lse.cpu().numpy()[rows].astype(np.float64)
        assert np.array_equal(np.isneginf(w), np.isneginf(g))
        fine = np.isfinite(w)
        slack = (E + 2.0**-20 + n * 2.0**-24)[rows] + 2.0**-22 * (np.abs(r["lse"][rows]) + 24)
        assert (np.abs(g[fine] - w[fine]) <= slack[fine]).all()


# ------------------------------------------------------------------------ CPU

def test_reference_by_hand():
    """Two positions of equal score: the mean of their values; an empty row."""
    k = np.zeros((2, 1, 64), np.float32)
    v = np.stack((np.full((1, 64), 1.0), np.full((1, 64), 3.0))).astype(np.float32)
    rows = ref.kv4_rows(k, v)
    mask = np.array([[[1, 0], [1, 1]]], np.uint8)
    r = ref.kv4_attention(np.ones((1, 2, 1, 64)), rows, np.array([[0, 1]], np.int32), [0], 1, 1.0, tree_mask=mask)
    assert np.allclose(r["out"][0, 0], 1.0) and np.allclose(r["out"][0, 1], 2.0)
    assert np.allclose(r["lse"][0, :, 0], [0.0, math.log(2.0)])
    r = ref.kv4_attention(np.ones((1, 2, 1, 64)), rows, np.array([[0, 1]], np.int32), [0], 1, 1.0, tree_mask=mask * 0)
    assert (r["out"] == 0).all() and np.isneginf(r["lse"]).all()


def test_host_checks():
    build()
    lib, null = sd.lib(), None
    assert sd.spec_kv4_attention_ws_size(1, 1, 8, 8, 128) >= 1
    for bad in ((0, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 1, 8, 3, 128), (1, 1, 8, 8, 80), (1, 1, 0, 8, 64)):
        assert lib.spec_kv4_attention_ws_size(*bad) == 0

    def call(B=1, N=1, Hq=2, Hkv=1, D=64, q=null, qs=128, pool=null, slots=8, stride=80, lens=null, table=null, ctx=8,
             scale=1.0, out=null, ws=null, wsb=0):
        return lib.spec_kv4_attention(B, N, Hq, Hkv, D, q, qs, pool, slots, stride, null, lens, table, ctx, null, scale,
                                      out, null, null, ws, wsb, null)
    assert call(B=-1) == -1 and call(N=-1) == -1 and call(Hkv=0) == -1 and call(Hq=3, Hkv=2) == -1 and call(Hq=0) == -1
    assert call(ctx=0) == -1 and call(slots=0) == -1 and call(scale=float("inf")) == -1 and call(scale=float("nan")) == -1
    assert call(D=96) == -2 and call(N=2049) == -2 and call(B=65536) == -2 and call(Hq=4097 * 1) == -2
    assert call(qs=127) == -1 and call(stride=64) == -1 and call(stride=88) == -2 and call(qs=132) == -2
    assert call(B=0) == 0 and call(N=0) == 0 and call() == -1
    if not torch.cuda.is_available():  # made-up addresses: only where nothing could run
        p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4104)
        a = dict(q=p, pool=p, lens=p, table=p, out=p, ws=p, wsb=1 << 40)
        for name in ("q", "pool", "out"):
            assert call(**{**a, name: odd}) == -2
        assert call(**{**a, "ws": odd}) == -1
        assert call(**{**a, "wsb": 64}) == -4
        assert call(**{**a, "ws": null}) == -1


def test_binding_refuses_host_tensors():
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 8), dtype=torch.int32)
    with pytest.raises(ValueError):
        sd.spec_kv4_attention(q, torch.zeros((8, 80), dtype=torch.uint8), i, i[0, :1], 1)


# ------------------------------------------------------------------------ GPU

@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    return sd.lib()


SHAPES = [
    # B, N, Hq, Hkv, D, lens, page
    (1, 1, 1, 1, 64, [0], 1), (1, 1, 1, 1, 128, [1], 1), (3, 1, 8, 8, 128, [15, 16, 17], 16),
    (4, 1, 32, 8, 128, [62, 63, 64, 65], 16), (2, 1, 16, 1, 64, [200, 3], 5), (2, 3, 15, 3, 64, [127, 400], 7),
    (1, 1, 17, 1, 128, [300], 4), (2, 5, 8, 2, 128, [0, 130], 16), (2, 8, 4, 1, 64, [500, 1], 16),
    (1, 16, 12, 4, 64, [777], 5), (2, 33, 1, 1, 128, [0, 61], 16), (1, 64, 8, 2, 128, [190], 16),
    (2, 64, 8, 1, 64, [63, 129], 64), (1, 70, 5, 1, 128, [257], 16), (40, 2, 2, 2, 64, list(range(40)), 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,Hq,Hkv,D,lens,page", SHAPES)
@pytest.mark.parametrize("tree", [True, False])
def test_matches_64_bits(gpu, B, N, Hq, Hkv, D, lens, page, tree):
    c = make_case(B + N * 3 + Hq * 7 + D, B, N, Hq, Hkv, D, lens, page, tree=tree)
    stats = sd.new_stats()
    out, lse = run(c, stats=stats)
    check(out, lse, expected(c))
    assert int(stats.sum()) == 0
    again, _ = run(c, lse=False)
    assert torch.equal(out, again)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(1, 4), (3, 8), (9, 8)])
def test_long_context_cut_between_ctas(gpu, N, G):
    """One KV head, one request: every CTA holds a part of one segment."""
    c = make_case(N, 1, N, G, 1, 128, [30011], page=16, spread=0.7)
    out, lse = run(c)
    check(out, lse, expected(c))


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(1, 8), (16, 4), (64, 4)])
def test_ragged_batch(gpu, N, G):
    """Requests from one position to thousands: segments whole and cut."""
    c = make_case(N + G, 7, N, 2 * G, 2, 64, [0, 1, 2500, 64, 0, 700, 63], page=5)
    out, lse = run(c)
    check(out, lse, expected(c))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [2, 40])
def test_rows_that_attend_to_nothing(gpu, N):
    c = make_case(3, 3, N, 4, 2, 64, [0, 0, 5], page=1)
    c["mask"][0, N - 1] = 0   # no context and nothing on the mask: zeros
    c["mask"][1] = 0
    c["mask"][2, 1] = 0       # the context alone
    out, lse = run(c)
    check(out, lse, expected(c))
    assert (out[0, N - 1] == 0).all() and (out[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 48])
def test_extremes_in_masked_places(gpu, N):
    """Masked nodes hold the largest values of the format, and q is tiny,
    huge, zero, NaN or infinite in rows of its own."""
    c = make_case(4, 1, N, 2, 1, 128, [20], page=1)
    k, v = ref.kv4_values(c["rows"], 1, 128)
    c["mask"][:, :, N - 1] = 0
    at = c["table"][0, 20 + N - 1]
    k[at], v[at] = 57344.0, -57344.0
    k[at, 0, ::2] = -57344.0
    c["rows"] = ref.kv4_rows(k, v)
    c["q"][0, 0, 0] *= 1e-30
    c["q"][0, 1, 0] *= 1e-3
    c["q"][0, 1, 1] = 0
    c["q"][0, 2, 0] *= 400.0
    r = expected(c)
    out, lse = run(c)
    check(out, lse, r)
    c["q"][0, 2, 1, 5] = float("nan")
    c["q"][0, 0, 1, 9] = float("inf")
    got, _ = run(c)
    other = torch.ones(c["q"].shape[:3], dtype=torch.bool)
    other[0, 2, 1] = other[0, 0, 1] = False
    assert torch.equal(got.cpu()[other], out.cpu()[other])  # a bad row spoils no other
    assert torch.isnan(got[0, 2, 1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [4, 24])
def test_padded_batch_and_bad_requests(gpu, N):
    B = 6
    c = make_case(5, B, N, 4, 2, 64, [30, 9, 40, 64, 12, 3], page=4)
    nodes = np.array([N, 0, 2, -1, N + 5, 1], np.int32)
    c["lens"][2], c["lens"][4] = -7, c["table"].shape[1] - N + 1
    c["table"][0, 3], c["table"][0, 29], c["table"][5, 1] = -1, c["rows"].shape[0], 2**31 - 1
    stats = sd.new_stats()
    out = torch.full((B, N, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    got, lse = run(c, num_nodes=torch.from_numpy(nodes).cuda(), out=out, stats=stats)
    live = np.arange(N)[None] < np.clip(nodes, 0, N)[:, None]
    check(got, lse, expected(c, nodes), live)
    dead = torch.from_numpy(~live)
    assert (got.cpu()[dead] == 5).all() and (lse.cpu()[dead] == 77).all()  # left as they were
    assert int(stats[sd.STATS["bad_request"]]) == 2 + 3  # two requests, three slots
    assert int(stats.sum()) == 5


@pytest.mark.gpu
def test_strided_q_and_a_layer_of_a_wider_slot(gpu):
    c = make_case(6, 2, 5, 6, 2, 64, [33, 70], page=16)
    B, N, Hq, D = c["q"].shape
    fused = torch.zeros((B, N, Hq + 4, D), dtype=torch.bfloat16, device="cuda")
    fused[:, :, :Hq] = c["q"].cuda()
    want, _ = run(c)
    got, _ = run(c, q=fused[:, :, :Hq])
    assert torch.equal(want, got)
    row = c["rows"].shape[1]
    wide = torch.full((c["rows"].shape[0], 3 * row), 255, dtype=torch.uint8, device="cuda")
    wide[:, row:2 * row] = torch.from_numpy(c["rows"]).cuda()
    got = sd.spec_kv4_attention(c["q"].cuda(), wide[:, row:2 * row], torch.from_numpy(c["table"]).cuda(),
                                torch.from_numpy(c["lens"]).cuda(), 2, scale=c["scale"],
                                tree_mask=torch.from_numpy(c["mask"]).cuda())
    assert torch.equal(want, got)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 20])
def test_slots_past_two_gigabytes(gpu, N):
    H, D, ctx = 64, 128, 100
    c = make_case(7, 1, N, H, H, D, [ctx], page=1)
    row = c["rows"].shape[1]
    slots = (5 << 30) // row
    pool = torch.zeros((slots, row), dtype=torch.uint8, device="cuda")
    c2 = dict(c, table=(slots - 1 - c["table"]).astype(np.int32))
    pool[torch.from_numpy(c2["table"][0].astype(np.int64)).cuda()] = torch.from_numpy(c["rows"][c["table"][0]]).cuda()
    want, _ = run(c)
    got = sd.spec_kv4_attention(c["q"].cuda(), pool, torch.from_numpy(c2["table"]).cuda(),
                                torch.from_numpy(c["lens"]).cuda(), H, scale=c["scale"],
                                tree_mask=torch.from_numpy(c["mask"]).cuda())
    assert torch.equal(want, got)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 16])
def test_captured_replayed_and_concurrent(gpu, N):
    c = make_case(8, 3, N, 8, 2, 128, [100, 257, 31], page=16)
    q, rows, table, lens = (torch.from_numpy(t).cuda() if isinstance(t, np.ndarray) else t.cuda()
                            for t in (c["q"], c["rows"], c["table"], c["lens"]))
    mask = torch.from_numpy(c["mask"]).cuda()
    size = sd.spec_kv4_attention_ws_size(3, N, 8, 2, 128)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def step(o=out, w=ws):
        return sd.spec_kv4_attention(q, rows, table, lens, 2, scale=c["scale"], tree_mask=mask, out=o, ws=w)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for shift in (-20, 0):  # the captured launch follows the lengths on the device
        d = dict(c, lens=c["lens"] + shift)
        lens.copy_(torch.from_numpy(d["lens"]))
        ws.fill_(255)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(out, None, expected(d))
    # two calls at once, each with its workspace
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, w2 = torch.empty_like(out), torch.empty_like(ws)
    for _ in range(5):
        with torch.cuda.stream(side):
            step(o2, w2)
        step()
    torch.cuda.synchronize()
    assert torch.equal(out, o2)
    check(out, None, expected(c))


@pytest.mark.gpu
def test_binding_checks(gpu):
    c = make_case(9, 2, 3, 4, 2, 64, [5, 6], page=1)
    q, rows, table, lens = c["q"].cuda(), torch.from_numpy(c["rows"]).cuda(), torch.from_numpy(c["table"]).cuda(), \
        torch.from_numpy(c["lens"]).cuda()
    ok = dict(q=q, kv_pool=rows, req_to_token=table, seq_lens=lens, num_kv_heads=2)
    for bad in ({"q": q.float()}, {"q": q.transpose(1, 2)}, {"num_kv_heads": 3}, {"num_kv_heads": 4}, {"kv_pool": rows[:, :64]},
                {"kv_pool": rows.int()}, {"req_to_token": table[:1]}, {"req_to_token": table.t()}, {"seq_lens": lens[:1]},
                {"tree_mask": torch.ones((2, 3, 2), dtype=torch.uint8, device="cuda")},
                {"tree_mask": torch.ones((2, 3, 3), dtype=torch.bool, device="cuda")}, {"num_nodes": lens[:1]},
                {"out": torch.empty((2, 3, 4, 32), dtype=torch.bfloat16, device="cuda")}, {"lse": torch.empty(3, device="cuda")},
                {"ws": torch.empty(16, dtype=torch.uint8, device="cuda")}, {"scale": float("nan")},
                {"q": q[..., 1:33]}):
        with pytest.raises((ValueError, sd.SpecError)):
            sd.spec_kv4_attention(**{**ok, **bad})
    empty = sd.spec_kv4_attention(**{**ok, "q": q[:, :0]})
    assert empty.shape == (2, 0, 4, 64)


def test_refused_scales_and_overlaps():
    build()
    lib, null = sd.lib(), None

    def call(scale=1.0, q=null, out=null, ptr=null, N=2, qs=128):
        return lib.spec_kv4_attention(1, N, 2, 1, 64, q, qs, ptr, 8, 80, null, ptr, ptr, 8, null, scale, out, null, null,
                                      ptr, 1 << 40, null)
    assert call(0.0) == -1 and call(-0.125) == -1 and call(-math.inf) == -1
    assert call(2.0 ** -21) == -2 and call(2.0 ** 21) == -2
    if not torch.cuda.is_available():  # made-up addresses: only where nothing could run
        a = dict(ptr=ctypes.c_void_p(4096))
        at = lambda x: ctypes.c_void_p(4096 * 16 + x)  # noqa: E731
        assert call(q=at(0), out=at(0), **a) == -1            # in place
        assert call(q=at(0), out=at(2 * 256 - 16), **a) == -1  # q's last 16 bytes
        assert call(q=at(2 * 256 - 16), out=at(0), **a) == -1  # out's last 16 bytes
        assert call(q=at(0), out=at(256), qs=256, **a) == -1   # between q's rows and into the last


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 12, 24, 48])
@pytest.mark.parametrize("scale", [2.0 ** -20, 1.0, 2.0 ** 20])
def test_smallest_and_largest_scales(gpu, N, scale):
    # the largest with q as much smaller, so that scores stay where softmax is not a choice
    c = make_case(77 + N, 2, N, 4, 2, 64, [5, 130], page=5)
    c["scale"] = scale
    c["q"] = (c["q"].float() * (2.0 ** -23 if scale > 1 else 2.0 ** -3)).to(torch.bfloat16)
    out, lse = run(c)
    check(out, lse, expected(c))


@pytest.mark.gpu
@pytest.mark.parametrize("N,Hq,lens", [(1, 1, 6), (3, 4, 5), (5, 4, 4), (9, 16, 300)])
def test_few_requests_far_apart_in_the_largest_batch(gpu, N, Hq, lens):
    """65535 requests of which five have nodes: the skipped ones cost no wait its limit and are left as they were."""
    B, live = 65535, [0, 1, 40000, 65533, 65534]
    c = make_case(91, len(live), N, Hq, 1, 64, [lens] * len(live), page=1)
    nodes = torch.zeros(B, dtype=torch.int32, device="cuda")
    nodes[live] = N
    seq = torch.zeros(B, dtype=torch.int32, device="cuda")
    seq[live] = torch.from_numpy(c["lens"]).cuda()
    table = torch.zeros((B, c["table"].shape[1]), dtype=torch.int32, device="cuda")
    table[live] = torch.from_numpy(c["table"]).cuda()
    mask = torch.zeros((B, N, N), dtype=torch.uint8, device="cuda")
    mask[live] = torch.from_numpy(c["mask"]).cuda()
    q = torch.zeros((B, N, Hq, 64), dtype=torch.bfloat16, device="cuda")
    q[live] = c["q"].cuda()
    out = torch.full_like(q, 7.0)
    stats = sd.new_stats("cuda")
    sd.spec_kv4_attention(q, torch.from_numpy(c["rows"]).cuda(), table, seq, 1, tree_mask=mask, num_nodes=nodes, out=out,
                          scale=c["scale"], stats=stats)
    assert stats.sum().item() == 0
    check(out[live], None, expected(c))
    out[live] = 7.0
    assert bool((out == 7.0).all())


# rows per KV head by kernel: up to 8, up to 16, one accumulator, two
KERNELS = [(1, 4), (3, 2), (3, 5), (12, 1), (24, 1), (48, 2), (48, 4)]


def never_appended(rows, slots, D):
    """Bytes in `slots` that no append wrote: NaN, infinities, and finite (step, lo) whose values leave fp16."""
    head = rows.reshape(rows.shape[0], -1, D + D // 4)
    kinds = [(np.nan, np.nan), (np.inf, 0.0), (0.0, -np.inf), (np.inf, -np.inf), (60000.0, 0.0), (-60000.0, -60000.0),
             (1.0, np.nan), (7000.0, 57344.0)]
    for i, slot in enumerate(slots):
        head[slot] = 255
        if i:
            head[slot, :, D:] = np.tile(np.array(kinds[i % len(kinds)], np.float16), D // 16).view(np.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", KERNELS)
@pytest.mark.parametrize("D", [64, 128])
def test_masked_nodes_that_were_never_appended(gpu, N, G, D):
    """A padded tree without num_nodes: columns that the mask hides from every row."""
    c = make_case(N + G + D, 2, N, 2 * G, 2, D, [20, 173], page=1)
    hidden = [0] if N == 1 else list(range(1, N))[-8:]
    c["mask"][:, :, hidden] = 0
    c["mask"][1, hidden[-1]] = 0  # and a row of the context alone
    never_appended(c["rows"], [c["table"][b, c["lens"][b] + n] for n in hidden for b in range(2)], D)
    with np.errstate(invalid="ignore"):
        r = expected(c)
    out, lse = run(c)
    check(out, lse, r)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", KERNELS)
@pytest.mark.parametrize("peak", [1.0, 0.7, 1.3])
@pytest.mark.parametrize("power", [20, 24, 25, 26, 27, 28, 30, 33, 60, 126, 127])
def test_largest_q(gpu, N, G, power, peak):
    """q up to bf16's largest.  K differs in one channel alone: two positions far apart hold the largest, so one row's
    result is the mean of these two and, with q's sign turned, that of all others; every other weight is below 2^-1000."""
    D, ctx = 64, 700
    c = make_case(power, 1, N, G, 1, D, [ctx], page=1)
    k, v = ref.kv4_values(c["rows"], 1, D)
    k[:] = 0
    k[:, 0, 0] = 0.5 * peak
    k[c["table"][0, [5, ctx - 9]], 0, 0] = peak
    k[c["table"][0, ctx:], 0, 0] = 0.75 * peak  # the nodes are neither
    c["rows"] = ref.kv4_rows(k, v)
    q = torch.zeros_like(c["q"])
    q[0, :, :, 0] = 2.0 ** power
    q[0, -1, -1, 0] = -(2.0 ** power) * (1.9921875 if power == 127 else 1.0)
    c["q"] = q
    r = expected(c)
    out, lse = run(c)
    # equal scores are equal in any precision and the others do not count: no error of scores
    check(out, None, dict(r, dot_abs=0 * r["dot_abs"], part_abs=0 * r["part_abs"]))
    # k in fp16 and a few fp32 operations; log2 of the weights' sum (2^10 at most), held 2^15, is absolute
    slack = np.abs(r["lse"]) * (2.0**-11 + 2.0**-20) + 24
    assert (np.abs(lse.cpu().numpy().astype(np.float64) - r["lse"]) <= slack).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", KERNELS)
def test_nan_in_q_is_nan_in_both_results(gpu, N, G):
    c = make_case(41 + N, 1, N, G, 1, 64, [333], page=1)
    want, want_lse = run(c)
    c["q"][0, N - 1, G - 1, 7] = float("nan")
    out, lse = run(c)
    assert torch.isnan(out[0, N - 1, G - 1]).all() and torch.isnan(lse[0, N - 1, G - 1])
    other = torch.ones((1, N, G), dtype=torch.bool, device="cuda")
    other[0, N - 1, G - 1] = False
    assert torch.equal(out[other], want[other]) and torch.equal(lse[other], want_lse[other])


def test_division_by_the_number_of_heads():
    """The kernels' row / heads as a product with ceil(2^40 / heads), over every number of heads and the rows around
    each multiple up to 2^23."""
    for G in (*range(1, 70), 127, 128, 129, 1000, 2047, 4093, 4094, 4095, 4096):
        inv = ((1 << 40) + G - 1) // G
        n = np.arange(0, min((1 << 23) // G + 1, 2049), dtype=np.int64) * G
        r = np.concatenate((n, n + G - 1, n + G // 2))
        r = r[r < 1 << 23]
        assert np.array_equal(r * inv >> 40, r // G)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", KERNELS)
def test_large_q_over_small_k(gpu, N, G):
    """Large elements of q whose scores stay moderate: the bounds mean something in every row."""
    D = 128
    c = make_case(31 + N, 2, N, G, 1, D, [61, 200], page=5)
    k, v = ref.kv4_values(c["rows"], 1, D)
    c["rows"] = ref.kv4_rows(k * 2.0**-9, v)
    c["q"] = (c["q"].float() * 400).to(torch.bfloat16)
    r = expected(c)
    assert np.expm1(score_error(r, D)).max() < 0.1
    out, lse = run(c)
    check(out, lse, r)


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,Hq,Hkv,D,lens", [(2, 129, 2, 1, 64, [0, 130]), (1, 200, 4, 2, 128, [61]),
                                               (2, 300, 3, 1, 64, [33, 257]), (1, 257, 1, 1, 128, [1000]),
                                               (2, 128, 2, 1, 128, [5, 127])])
@pytest.mark.parametrize("tree", [True, False])
def test_more_nodes_than_a_tile(gpu, B, N, Hq, Hkv, D, lens, tree):
    c = make_case(N + D, B, N, Hq, Hkv, D, lens, page=5, tree=tree)
    nodes = np.array([N, N - 70][:B], np.int32)
    for nn in (None, nodes):
        out, lse = run(c, num_nodes=None if nn is None else torch.from_numpy(nn).cuda())
        live = np.arange(N)[None] < (nodes if nn is not None else np.full(B, N))[:, None]
        check(out, lse, expected(c, nn), live)


@pytest.mark.gpu
def test_most_nodes_and_heads(gpu):
    """2048 nodes of 4095 query heads on one KV head: 2^23 - 2048 rows.  Each node sees itself alone."""
    N, Hq, D = 2048, 4095, 64
    rng = np.random.default_rng(17)
    v = rng.normal(0, 1, (N, 1, D)).astype(np.float32)
    rows = ref.kv4_rows(v, v)
    q = torch.empty((1, N, Hq, D), dtype=torch.bfloat16, device="cuda").normal_()
    out = sd.spec_kv4_attention(q, torch.from_numpy(rows).cuda(), torch.arange(N, dtype=torch.int32, device="cuda")[None],
                                torch.zeros(1, dtype=torch.int32, device="cuda"), 1,
                                tree_mask=torch.eye(N, dtype=torch.uint8, device="cuda")[None])
    want = torch.from_numpy(ref.kv4_values(rows, 1, D)[1]).cuda()  # [N, 1, D] fp64
    # v and its weight in fp16, the exponential's 2^-20 and the division; then bf16
    move = want.abs() * (2 * 2.0**-11 + 2.0**-18) + 2.0**-25
    bound = move + 2.0**-8 * (want.abs() + move)
    for n in range(0, N, 256):
        off = (out[0, n:n + 256].double() - want[n:n + 256]).abs()
        assert bool((off <= bound[n:n + 256]).all())


def test_no_workspace_for_sizes_that_are_refused():
    build()
    size = sd.lib().spec_kv4_attention_ws_size
    assert size(65535, 1, 8, 8, 128) > 0 and size(1, 2048, 8, 8, 128) > 0 and size(1, 1, 4096, 1, 64) > 0
    for bad in ((65536, 1, 8, 8, 128), (1, 2049, 8, 8, 128), (1, 1, 4097, 1, 64), (1, 1, 514, 257, 64)):
        assert size(*bad) == 0
        with pytest.raises(sd.SpecError):
            sd.spec_kv4_attention_ws_size(*bad)
