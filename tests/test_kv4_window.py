"""spec_kv4_attention_window against windowed attention in 64 bits over the same
cache rows.  The bounds are those of the attention over the whole cache
(test_kv4_attention.py derives them); count is the number of positions seen."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_draft_select_gb300 as sd
from oracle import target as ref
from speculative_decoding_draft_select_gb300.build import build

from test_kv4_attention import check, make_case


def depths(mask):
    return mask.sum(2).astype(np.int32) - 1


def run(c, sinks, window, positions="tree", q=None, lse=True, **kw):
    q = c["q"].cuda() if q is None else q
    if isinstance(positions, str):
        positions = None if c["mask"] is None else c["lens"][:, None] + depths(c["mask"])
    got_lse = torch.full(c["q"].shape[:3], 77.0, device="cuda") if lse else None
    out = sd.spec_kv4_attention_window(
        q, torch.from_numpy(c["rows"]).cuda(), torch.from_numpy(c["table"]).cuda(), torch.from_numpy(c["lens"]).cuda(),
        c["Hkv"], sinks, window, positions=None if positions is None else torch.from_numpy(positions.astype(np.int32)).cuda(),
        scale=c["scale"], lse=got_lse, tree_mask=None if c["mask"] is None else torch.from_numpy(c["mask"]).cuda(), **kw)
    return out, got_lse


def expected(c, sinks, window, positions="tree", num_nodes=None):
    if isinstance(positions, str):
        positions = None if c["mask"] is None else c["lens"][:, None] + depths(c["mask"])
    return ref.kv4_attention(c["q"].float().numpy(), c["rows"], c["table"], c["lens"], c["Hkv"], c["scale"],
                             tree_mask=c["mask"], num_nodes=num_nodes, window=window, sinks=sinks, positions=positions)


# ------------------------------------------------------------------------ CPU

def test_reference_by_hand():
    """Values 0..5 of equal score; a chain of two nodes at 4 and 5."""
    k = np.zeros((6, 1, 64), np.float32)
    v = np.repeat(np.arange(6, dtype=np.float32)[:, None, None], 64, 2)
    rows, table = ref.kv4_rows(k, v), np.arange(6, dtype=np.int32)[None]
    q = np.ones((1, 2, 1, 64))
    r = ref.kv4_attention(q, rows, table, [4], 1, 1.0, window=2, sinks=1)
    assert np.allclose(r["out"][0, 0], (0 + 3 + 4) / 3) and np.allclose(r["out"][0, 1], (0 + 4 + 5) / 3)
    # the second node hangs beside the first: both at position 4
    r = ref.kv4_attention(q, rows, table, [4], 1, 1.0, window=2, tree_mask=np.eye(2, dtype=np.uint8)[None],
                          positions=np.array([[4, 4]]))
    assert np.allclose(r["out"][0, 0], 3.5) and np.allclose(r["out"][0, 1], 4.0)
    # a position too large is taken as the second node's deepest, 5
    far = ref.kv4_attention(q, rows, table, [4], 1, 1.0, window=2, positions=np.array([[0, 99]]))
    assert np.allclose(far["out"][0, 0], 3.5) and np.allclose(far["out"][0, 1], 4.5)


def test_host_checks():
    build()
    lib, null = sd.lib(), None

    def call(B=1, N=1, Hq=2, Hkv=1, D=64, q=null, qs=128, pool=null, slots=8, stride=80, lens=null, table=null, ctx=8,
             sinks=0, window=1, scale=1.0, out=null, ws=null, wsb=0):
        return lib.spec_kv4_attention_window(B, N, Hq, Hkv, D, q, qs, pool, slots, stride, null, lens, null, table, ctx,
                                             null, sinks, window, scale, out, null, null, ws, wsb, null)
    assert call(sinks=-1) == -1 and call(window=0) == -1 and call(window=-5) == -1
    assert call(B=-1) == -1 and call(Hq=3, Hkv=2) == -1 and call(ctx=0) == -1 and call(scale=0.0) == -1
    assert call(D=96) == -2 and call(N=2049) == -2 and call(stride=88) == -2 and call(qs=127) == -1
    assert call(B=0) == 0 and call(N=0) == 0 and call() == -1
    if not torch.cuda.is_available():  # made-up addresses: only where nothing could run
        p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4104)
        a = dict(q=p, pool=p, lens=p, table=p, out=p, ws=p, wsb=1 << 40)
        for name in ("q", "pool", "out"):
            assert call(**{**a, name: odd}) == -2
        assert call(**{**a, "wsb": 64}) == -4 and call(**{**a, "lens": null}) == -1


def test_binding_refuses_host_tensors():
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 8), dtype=torch.int32)
    with pytest.raises(ValueError):
        sd.spec_kv4_attention_window(q, torch.zeros((8, 80), dtype=torch.uint8), i, i[0, :1], 1, 0, 4)


# ------------------------------------------------------------------------ GPU

@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    return sd.lib()


SHAPES = [
    # B, N, Hq, Hkv, D, lens, page
    (1, 1, 1, 1, 64, [0], 1), (3, 1, 8, 8, 128, [15, 160, 17], 16), (4, 1, 32, 8, 128, [62, 63, 640, 65], 16),
    (2, 3, 15, 3, 64, [127, 400], 7), (1, 1, 17, 1, 128, [300], 4), (2, 5, 8, 2, 128, [0, 530], 16),
    (2, 8, 4, 1, 64, [500, 1], 16), (1, 16, 12, 4, 64, [777], 5), (2, 33, 1, 1, 128, [0, 461], 16),
    (2, 64, 8, 1, 64, [63, 529], 64), (1, 70, 5, 1, 128, [357], 16), (1, 150, 2, 1, 64, [300], 16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,Hq,Hkv,D,lens,page", SHAPES)
@pytest.mark.parametrize("sinks,window", [(0, 1), (0, 5), (4, 3), (4, 64), (1, 129), (130, 100), (7, 5000), (1000, 2)])
@pytest.mark.parametrize("tree", [True, False])
def test_matches_64_bits(gpu, B, N, Hq, Hkv, D, lens, page, sinks, window, tree):
    c = make_case(B + N * 3 + Hq * 7 + D, B, N, Hq, Hkv, D, lens, page, tree=tree)
    stats = sd.new_stats()
    out, lse = run(c, sinks, window, stats=stats)
    check(out, lse, expected(c, sinks, window))
    assert int(stats.sum()) == 0
    again, _ = run(c, sinks, window, lse=False)
    assert torch.equal(out, again)


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,Hq,Hkv,D", [(90, 34, 8, 8, 64), (60, 40, 16, 4, 128), (85, 20, 16, 8, 128)])
@pytest.mark.parametrize("sinks,window", [(0, 1), (4, 3), (7, 40), (130, 100), (3, 300)])
def test_large_batches(gpu, B, N, Hq, Hkv, D, sinks, window):
    """More row tiles than the few that go to the kernel of 16 rows: the tensor
    memory's, with one accumulator and with two.  Padded requests, positions from
    depths and at random, and nothing but NaN and no slots out of sight."""
    rng = np.random.default_rng(N + window)
    lens = rng.integers(0, 400, B)
    lens[:3] = [0, 1, window]
    c = make_case(N, B, N, Hq, Hkv, D, lens, page=5)
    nn = rng.integers(0, N + 1, B).astype(np.int32)
    nn[:2] = N
    pos = c["lens"][:, None] + depths(c["mask"])
    pos[B // 2:] = rng.integers(-5, 500, pos[B // 2:].shape)
    want = expected(c, sinks, window, positions=pos, num_nodes=nn)
    for b, n in enumerate(c["lens"]):
        gone = slice(sinks, max(sinks, n - window + 1))
        c["rows"][c["table"][b, gone]] = 0xff
        c["table"][b, gone][::3] = -1
    stats = sd.new_stats()
    out = torch.full(c["q"].shape, 3.0, dtype=torch.bfloat16, device="cuda")
    _, lse = run(c, sinks, window, positions=pos, num_nodes=torch.from_numpy(nn).cuda(), out=out, stats=stats)
    rows = np.arange(N)[None] < nn[:, None]
    check(out, lse, want, rows)
    assert (out.cpu()[torch.from_numpy(~rows)] == 3.0).all() and int(stats.sum()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 12, 70])
def test_window_that_reaches_everything(gpu, N):
    """A window beyond every length: the plain attention, bit for bit."""
    c = make_case(N, 3, N, 4, 2, 128, [0, 300, 77])
    window = 2**40  # beyond every position
    out, lse = run(c, 0, window)
    want_lse = torch.empty_like(lse)
    want = sd.spec_kv4_attention(c["q"].cuda(), torch.from_numpy(c["rows"]).cuda(), torch.from_numpy(c["table"]).cuda(),
                                 torch.from_numpy(c["lens"]).cuda(), 2, scale=c["scale"], lse=want_lse,
                                 tree_mask=torch.from_numpy(c["mask"]).cuda())
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out, lse = run(c, 2**31, 1)  # all sinks
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(1, 4), (5, 3), (20, 4)])
def test_positions_out_of_sight_are_not_touched(gpu, N, G):
    """Their slots may be freed (out of range here) or hold anything (NaN here)."""
    c = make_case(N, 2, N, G, 1, 64, [900, 333])
    sinks, window = 3, 50
    want = expected(c, sinks, window)
    table, rows = c["table"].copy(), c["rows"].copy()
    for b, n in enumerate(c["lens"]):
        gone = slice(sinks, n - window + 1)
        rows[table[b, gone]] = 0xff                       # NaN steps
        table[b, gone][::2] = -1
        table[b, gone][1::4] = 2**31 - 1
    c["table"], c["rows"] = table, rows
    stats = sd.new_stats()
    out, lse = run(c, sinks, window, stats=stats)
    check(out, lse, want)
    assert int(stats.sum()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [4, 20, 90])
def test_positions_that_are_no_positions(gpu, N):
    c = make_case(N, 2, N, 4, 1, 64, [200, 5])
    rng = np.random.default_rng(0)
    pos = rng.integers(-2**31, 2**31, (2, N)).astype(np.int32)
    pos[:, ::3] = c["lens"][:, None] + rng.integers(-3, N + 3, pos[:, ::3].shape)
    out, lse = run(c, 2, 7, positions=pos)
    check(out, lse, expected(c, 2, 7, positions=pos))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [6, 40])
def test_padded_batch_and_rows_behind(gpu, N):
    c = make_case(11, 4, N, 4, 2, 64, [100, 0, 700, 40])
    nn = np.array([N, 0, N // 2, 1], np.int32)
    out = torch.full(c["q"].shape, 3.0, dtype=torch.bfloat16, device="cuda")
    _, lse = run(c, 3, 33, num_nodes=torch.from_numpy(nn).cuda(), out=out)
    rows = np.arange(N)[None] < nn[:, None]
    check(out, lse, expected(c, 3, 33, num_nodes=nn), rows)
    assert (out.cpu()[torch.from_numpy(~rows)] == 3.0).all() and (lse.cpu()[torch.from_numpy(~rows)] == 77.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [2, 40])
def test_bad_requests_and_slots(gpu, N):
    c = make_case(12, 4, N, 4, 2, 64, [100, 100, 100, 100])
    c["lens"] = np.array([100, -1, 101, 60], np.int32)          # the second and third do not fit
    c["table"][0, [0, 99, 30]] = [-1, 10**9, -7]                # two in sight, one not
    stats = sd.new_stats()
    out, lse = run(c, 2, 10, stats=stats)
    check(out, lse, expected(c, 2, 10))
    assert stats.tolist()[sd.STATS["bad_request"]] == 2 + 2


@pytest.mark.gpu
@pytest.mark.parametrize("N", [4, 40])
def test_rows_that_see_nothing(gpu, N):
    """A mask without the node itself, outside the window's context."""
    c = make_case(13, 2, N, 4, 2, 128, [50, 3])
    c["mask"][:, N - 1] = 0
    pos = c["lens"][:, None] + np.minimum(np.arange(N), 9)[None] + np.zeros((2, 1), int)
    out, lse = run(c, 0, 2, positions=pos)
    check(out, lse, expected(c, 0, 2, positions=pos))
    assert (out[:, N - 1] == 0).all() and torch.isneginf(lse[:, N - 1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(1, 4), (3, 8), (9, 8), (64, 4)])
def test_long_window_cut_between_ctas(gpu, N, G):
    c = make_case(N, 1, N, G, 1, 128, [40011], spread=0.7)
    out, lse = run(c, 5, 20001)
    check(out, lse, expected(c, 5, 20001))


@pytest.mark.gpu
def test_strided_queries_captured_on_another_stream(gpu):
    c = make_case(14, 3, 6, 8, 2, 64, [70, 0, 300])
    wide = torch.randn((3, 6, 12, 64), device="cuda").to(torch.bfloat16)
    q = wide[:, :, 2:10]
    q.copy_(c["q"])
    args = {k: torch.from_numpy(c[k]).cuda() for k in ("rows", "table", "lens", "mask")}
    pos = torch.from_numpy(c["lens"][:, None] + depths(c["mask"])).cuda()
    out, lse = torch.empty(c["q"].shape, dtype=torch.bfloat16, device="cuda"), torch.empty((3, 6, 8), device="cuda")
    ws = torch.empty(sd.spec_kv4_attention_ws_size(3, 6, 8, 2, 64), dtype=torch.uint8, device="cuda")

    def call():
        sd.spec_kv4_attention_window(q, args["rows"], args["table"], args["lens"], 2, 4, 32, positions=pos,
                                     tree_mask=args["mask"], scale=c["scale"], out=out, lse=lse, ws=ws)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
    torch.cuda.synchronize()
    c["lens"] = np.array([9, 250, 64], np.int32)  # replayed with other lengths
    args["lens"].copy_(torch.from_numpy(c["lens"]))
    pos.copy_(torch.from_numpy(c["lens"][:, None] + depths(c["mask"])))
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph.replay()
    torch.cuda.synchronize()
    check(out, lse, expected(c, 4, 32))


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(1, 4), (5, 4), (12, 4), (34, 2), (70, 4)])
@pytest.mark.parametrize("window", [1, 5, 40])
def test_positions_count_from_the_root(gpu, N, G, window):
    """Positions of the text, which an eviction has left behind the cache's: the
    depths are the same, and so is every bit."""
    c = make_case(N + window, 3, N, 2 * G, 2, 64, [300, 2, 45])
    pos = c["lens"][:, None].astype(np.int64) + depths(c["mask"])
    out, lse = run(c, 3, window, positions=pos)
    check(out, lse, expected(c, 3, window, positions=pos))
    moved = pos + np.array([[100000], [-7], [2**31 - 1 - 45 - N]])
    again, again_lse = run(c, 3, window, positions=moved)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    check(again, again_lse, expected(c, 3, window, positions=moved))


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(9, 1), (9, 4), (40, 4)])
@pytest.mark.parametrize("window", [3, 30])
def test_a_mask_without_positions(gpu, N, G, window):
    """Each node is then one further on, whatever its mask shows."""
    c = make_case(N, 2, N, G, 1, 64, [100, 4])
    out, lse = run(c, 2, window, positions=None)
    check(out, lse, expected(c, 2, window, positions=None))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 4, 40])
def test_slots_beyond_32_bits(gpu, N):
    """Rows of 1 MB: the last slots lie more than 2^32 bytes behind the first."""
    c = make_case(25, 2, N, 4, 1, 64, [130, 3])
    slots, far = c["rows"].shape[0], 5000
    wide = torch.zeros((far, 1 << 20), dtype=torch.uint8, device="cuda")
    wide[far - slots:, :80] = torch.from_numpy(c["rows"]).cuda()
    out = sd.spec_kv4_attention_window(
        c["q"].cuda(), wide[:, :80], torch.from_numpy(c["table"] + far - slots).cuda(), torch.from_numpy(c["lens"]).cuda(), 1,
        2, 50, positions=torch.from_numpy(c["lens"][:, None] + depths(c["mask"])).cuda(), scale=c["scale"],
        tree_mask=torch.from_numpy(c["mask"]).cuda())
    check(out, None, expected(c, 2, 50))


def test_reference_counts_positions_from_the_root():
    c = make_case(1, 2, 9, 2, 1, 64, [20, 3])
    pos = c["lens"][:, None].astype(np.int64) + depths(c["mask"])
    want = expected(c, 1, 4, positions=pos)
    moved = expected(c, 1, 4, positions=pos + np.array([[1000], [-3]]))
    assert all(np.array_equal(want[n], moved[n]) for n in ("out", "lse", "count"))


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,Hq,Hkv,D,lens", [(1, 2048, 2, 1, 64, [300]), (2, 700, 4, 2, 128, [0, 2500]),
                                               (1, 1025, 1, 1, 128, [77])])
@pytest.mark.parametrize("sinks,window", [(4, 128), (0, 1024), (300, 1)])
@pytest.mark.parametrize("tree", [True, False])
def test_chunks_of_a_prompt(gpu, B, N, Hq, Hkv, D, lens, sinks, window, tree):
    """Up to the most nodes a call may have, as a chain and as a tree."""
    c = make_case(N + window, B, N, Hq, Hkv, D, lens, tree=tree)
    stats = sd.new_stats()
    out, lse = run(c, sinks, window, stats=stats)
    check(out, lse, expected(c, sinks, window))
    assert int(stats.sum()) == 0
