"""spec_kv4_weight_sums against weights in 64 bits over the same cache rows.

Bounds.  A score is a sum of at most D products step (q . c) and lo sum q, in
fp32 (the tensor cores' sums may cut instead of rounding, 2^-23 an addition):
at most (D + 16) additions and products, relative to the parts' magnitude
|scale| sum |q| (|lo| + |k - lo|).  q's elements 2^-24 of its row's largest may
round in fp16, by 2^-25 of the largest.  Factors, lse log2(e) and the
difference round by 2^-24 of the score's and lse's magnitude, four times at
most; the exponential by 2^-21.  A weight moves by its value times the sum of
these, and the sum of n weights and prev by (n + 1) 2^-24 of the total."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_draft_select_gb300 as sd
from oracle import target as ref
from speculative_decoding_draft_select_gb300.build import build

from test_kv4_attention import make_case


def add_rows(c, seed=0, accepted=None, path=None):
    """lse of the rows as a chain behind the context, prev, and the path."""
    rng = np.random.default_rng(seed)
    B, N, Hq, D = c["q"].shape
    c["prev"] = rng.exponential(1.0, c["table"].shape).astype(np.float32)
    c["accepted"] = None if accepted is None else np.asarray(accepted, np.int32)
    c["path"] = path
    c["lse"] = np.zeros((B, N, Hq), np.float32)
    for b in range(B):
        R = N if accepted is None else accepted[b] + 1
        row = np.arange(R) if path is None else path[b, :R]
        q = c["q"].float().numpy()[b:b + 1, row]
        r = ref.kv4_attention(q, c["rows"], c["table"][b:b + 1], c["lens"][b:b + 1], c["Hkv"], c["scale"])
        c["lse"][b, row] = r["lse"][0]
    return c


def on(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(c, prev="case", out=None, **kw):
    out = torch.full(c["table"].shape, 55.0, device="cuda") if out is None else out
    kw.setdefault("q", c["q"].cuda())
    return sd.spec_kv4_weight_sums(kw.pop("q"), on(c["lse"]), on(c["rows"]), on(c["table"]), on(c["lens"]), c["Hkv"],
                                   accept_path=on(c["path"]), accept_length=on(c["accepted"]),
                                   prev=on(c["prev"]) if isinstance(prev, str) else prev, out=out, scale=c["scale"], **kw)


def expected(c, prev=True):
    return ref.kv4_weight_sums(c["q"].float().numpy(), c["lse"], c["rows"], c["table"], c["lens"], c["Hkv"], c["scale"],
                               accept_path=c["path"], accept_length=c["accepted"], prev=c["prev"] if prev else None)


def check(got, r, D, left=55.0):
    got = got.cpu().numpy().astype(np.float64)
    move = (r["parts"] * (D + 16) * 2.0**-23 + r["far"] * 2.0**-25 + r["size"] * 4 * 2.0**-24 + r["w"] * 2.0**-21)
    bound = move * 1.01 + (r["count"] + 1) * 2.0**-24 * (np.abs(r["sums"]) + move) + 2.0**-120
    off = np.abs(got - r["sums"]) - bound
    t = r["touched"]
    assert (off[t] <= 0).all(), f"worst excess {off[t].max()}, bound there {bound[t][off[t].argmax()]}"
    assert (got[~t] == left).all()


# ------------------------------------------------------------------------ CPU

def test_reference_by_hand():
    """Two equal positions and a row that sees both, one head: half a weight each."""
    k = np.zeros((2, 1, 64), np.float32)
    rows = ref.kv4_rows(k, k)
    r = ref.kv4_weight_sums(np.ones((1, 1, 1, 64)), np.log([[[2.0]]]), rows, np.array([[0, 1, 0]], np.int32), [1], 1, 1.0,
                            prev=np.ones((1, 3)))
    assert np.allclose(r["sums"], [[1.5, 1.5, 1.0]]) and r["touched"].tolist() == [[True, True, False]]


def test_host_checks():
    build()
    lib, null = sd.lib(), None

    def call(B=1, N=1, Hq=2, Hkv=1, D=64, q=null, qs=128, lse=null, pool=null, slots=8, stride=80, lens=null, table=null,
             ctx=8, scale=1.0, prev=null, out=null, ws=null, wsb=0):
        return lib.spec_kv4_weight_sums(B, N, Hq, Hkv, D, q, qs, lse, null, null, pool, slots, stride, lens, table, ctx,
                                        scale, prev, out, null, ws, wsb, null)
    size = lib.spec_kv4_weight_sums_ws_size
    assert size(1, 1, 32, 1, 128) == 0 and size(1, 8, 32, 8, 64) == 0 and size(1, 33, 1, 1, 128) > 128 * 128 * 2
    assert size(3, 33, 8, 2, 64) == 6 * size(1, 33, 4, 1, 64) and size(1, 2049, 1, 1, 64) == 0 and size(0, 64, 1, 1, 64) == 0
    assert call(B=-1) == -1 and call(N=-1) == -1 and call(Hkv=0) == -1 and call(Hq=3, Hkv=2) == -1 and call(ctx=0) == -1
    assert call(slots=0) == -1 and call(scale=float("nan")) == -1 and call(scale=-1.0) == -1
    assert call(D=96) == -2 and call(N=2049) == -2 and call(B=65536) == -2 and call(Hq=4097) == -2 and call(scale=1e-9) == -2
    assert call(qs=127) == -1 and call(stride=64) == -1 and call(stride=88) == -2 and call(qs=132) == -2
    assert call(B=0) == 0 and call(N=0) == 0 and call() == -1
    if not torch.cuda.is_available():  # made-up addresses: only where nothing could run
        p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4104)
        a = dict(q=p, lse=p, pool=p, lens=p, table=p, out=p)
        for name in ("q", "pool"):
            assert call(**{**a, name: odd}) == -2
        for name in a:
            assert call(**{**a, name: null}) == -1
        assert call(**a, prev=ctypes.c_void_p(4100)) == -1        # sums and their new ones overlap in part
        many = dict(a, N=17, qs=128)
        assert call(**many) == -1 and call(**many, ws=odd) == -1 and call(**many, ws=p, wsb=64) == -4


def test_binding_refuses_host_tensors():
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 8), dtype=torch.int32)
    with pytest.raises(ValueError):
        sd.spec_kv4_weight_sums(q, torch.zeros((1, 1, 1)), torch.zeros((8, 80), dtype=torch.uint8), i, i[0, :1], 1)


# ------------------------------------------------------------------------ GPU

@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    return sd.lib()


SHAPES = [
    # B, N, Hq, Hkv, D, lens, page
    (1, 1, 1, 1, 64, [0], 1), (1, 1, 1, 1, 128, [1], 1), (3, 1, 8, 8, 128, [15, 31, 32], 16),
    (4, 1, 32, 8, 128, [62, 63, 640, 65], 16), (2, 3, 15, 3, 64, [127, 400], 7), (1, 1, 17, 1, 128, [300], 4),
    (2, 5, 8, 2, 128, [0, 530], 16), (2, 8, 4, 1, 64, [500, 1], 16), (1, 16, 12, 4, 64, [777], 5),
    (2, 33, 2, 1, 128, [0, 461], 16), (1, 64, 8, 2, 128, [190], 16), (1, 70, 5, 1, 64, [257], 16),
    (40, 2, 2, 2, 64, list(range(40)), 1), (1, 2, 20, 20, 64, [90], 16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,Hq,Hkv,D,lens,page", SHAPES)
@pytest.mark.parametrize("commit", [True, False])
def test_matches_64_bits(gpu, B, N, Hq, Hkv, D, lens, page, commit):
    c = make_case(B + N * 3 + Hq * 7 + D, B, N, Hq, Hkv, D, lens, page)
    rng = np.random.default_rng(N)
    accepted = path = None
    if commit:
        accepted = rng.integers(0, N, B)
        path = np.stack([np.concatenate(([0], 1 + rng.permutation(N - 1))) for _ in range(B)]).astype(np.int32)
        for b in range(B):
            path[b, :accepted[b] + 1].sort()
    add_rows(c, N, accepted, path)
    stats = sd.new_stats()
    got = run(c, stats=stats)
    check(got, expected(c), D)
    assert int(stats.sum()) == 0
    assert torch.equal(got, run(c))
    assert torch.equal(got, run(c, prev=on(c["prev"]), out=None)[:, :]) and got.dtype == torch.float32
    check(run(c, prev=None), expected(c, prev=False), D)
    # in place
    p = on(c["prev"])
    assert run(c, prev=p, out=p) is p
    t = torch.from_numpy(expected(c)["touched"]).cuda()
    assert torch.equal(p[t], got[t]) and torch.equal(p[~t], on(c["prev"])[~t])


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(1, 4), (2, 8), (40, 4)])
def test_long_context(gpu, N, G):
    c = add_rows(make_case(N, 1, N, 2 * G, 2, 128, [20011], spread=0.7))
    got = run(c)
    check(got, expected(c), 128)
    # every row's weights sum to one
    assert abs(float((got - on(c["prev"]))[0, :20011 + N].double().sum()) - N * 2 * G) < 1e-3 * N * G


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,G,Hkv,D", [(1, 9, 4, 1, 64), (2, 33, 1, 3, 128), (3, 17, 8, 2, 64), (1, 100, 3, 1, 128),
                                         (2, 64, 8, 1, 64)])
def test_many_rows(gpu, B, N, G, Hkv, D):
    """33 to 512 rows of a KV head, over contexts that end in every part of a tile."""
    c = add_rows(make_case(N, B, N, G * Hkv, Hkv, D, [1601, 130 - N, 0][:B], spread=1.0), accepted=[N - 1, N // 2, 0][:B])
    stats = sd.new_stats()
    got = run(c, stats=stats)
    check(got, expected(c), D)
    assert int(stats.sum()) == 0
    assert torch.equal(got, run(c))


@pytest.mark.gpu
def test_few_and_many_rows_in_one_batch(gpu):
    """Paths from one row to all of 40; bad entries and lengths among them."""
    B, N = 6, 40
    c = make_case(21, B, N, 4, 2, 64, [300, 0, 5, 700, 90, 40], spread=1.0)
    rng = np.random.default_rng(0)
    path = np.stack([np.concatenate(([0], 1 + rng.permutation(N - 1))) for _ in range(B)]).astype(np.int32)
    add_rows(c, 1, [39, 0, 15, 16, 2, 30], path)
    c["path"][0, 5], c["path"][3, 16], c["path"][4, 1] = -1, N, 2**31 - 1
    c["accepted"][5] = N
    stats = sd.new_stats()
    got = run(c, stats=stats)
    check(got, expected(c), 64)
    assert stats.tolist()[sd.STATS["bad_request"]] == 4


@pytest.mark.gpu
def test_many_rows_in_many_segments(gpu):
    """Enough tiles that CTAs work alone, over several segments and requests."""
    c = make_case(3, 12, 6, 8, 1, 64, [5003, 4000, 3333, 17, 0, 5100, 2900, 128, 4900, 4801, 5055, 61], spread=0.8)
    add_rows(c)
    got = run(c)
    check(got, expected(c), 64)
    assert torch.equal(got, run(c))


@pytest.mark.gpu
@pytest.mark.parametrize("N,G", [(1, 8), (16, 4)])
def test_ragged_batch(gpu, N, G):
    c = add_rows(make_case(N + G, 7, N, 2 * G, 2, 64, [0, 1, 2500, 64, 0, 700, 63], page=5))
    check(run(c), expected(c), 64)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [2, 20])
def test_bad_requests_slots_and_rows(gpu, N):
    c = add_rows(make_case(12, 5, N, 4, 2, 64, [100] * 5), path=np.tile(np.arange(N, dtype=np.int32), (5, 1)),
                 accepted=np.full(5, N - 1))
    c["lens"] = np.array([100, -1, 101, 60, 100], np.int32)     # the second and third do not fit
    c["accepted"] = np.array([N - 1, 0, N - 1, -2, N], np.int32)  # nor do the fourth's and fifth's rows
    c["table"][0, [0, 99, 30]] = [-1, 10**9, -7]
    c["path"][0, 1] = N
    stats = sd.new_stats()
    got = run(c, stats=stats)
    r = expected(c)
    check(got, r, 64)
    assert r["touched"].any(1).tolist() == [True, False, False, False, False]
    assert stats.tolist()[sd.STATS["bad_request"]] == 4 + 3 + 1


@pytest.mark.gpu
@pytest.mark.parametrize("N", [2, 12])
def test_rows_without_a_finite_lse_add_nothing(gpu, N):
    c = add_rows(make_case(13, 2, N, 4, 2, 128, [70, 3]))
    for i, bad in enumerate((float("-inf"), float("inf"), float("nan"))):
        c["lse"][i % 2, i % N, i] = bad
    c["q"][0, 0, 0] = float("nan")
    c["q"][1, N - 1, 1] = float("inf")
    c["lse"][0, 0, 0] = c["lse"][1, N - 1, 1] = float("nan")
    got = run(c)
    c["q"] = torch.where(torch.isfinite(c["q"].float()), c["q"], 0)
    check(got, expected(c), 128)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0**-126, 2.0**-60, 2.0**-13, 2.0**20, 2.0**30])
def test_rows_far_from_one(gpu, size):
    """K shrinks as q grows, so that the scores stay near one; q's smallest are
    subnormal in bf16, where the scale cannot bring the scores back."""
    c = make_case(14, 1, 2, 4, 2, 64, [90])
    k = np.random.default_rng(1).normal(0, 1, (c["rows"].shape[0], 2, 64)).astype(np.float32)
    shrink = 2.0**-10 if size > 1 else 1.0
    c["rows"] = ref.kv4_rows(k * np.float32(shrink), k)
    c["q"] = (c["q"].float() * size).to(torch.bfloat16)
    c["scale"] = float(np.clip(1.0 / (size * shrink) / 8, 2.0**-20, 2.0**20))
    add_rows(c)
    check(run(c), expected(c), 64)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [3, 8, 9, 17, 60])
@pytest.mark.parametrize("N", [6, 40])
def test_rows_of_different_sizes(gpu, N, spread):
    """Rows from 2^-spread of the largest on, some without a finite lse, some zero."""
    c = make_case(17, 2, N, 4, 2, 128, [200, 60])
    size = 2.0 ** -np.random.default_rng(spread).integers(0, spread + 1, (2, N, 4))
    size[0, 1] = 0
    c["q"] = (c["q"].float() * torch.from_numpy(size)[..., None].float()).to(torch.bfloat16)
    add_rows(c)
    c["lse"][1, N // 2, 1] = float("-inf")
    check(run(c), expected(c), 128)


@pytest.mark.gpu
def test_elements_far_below_their_row(gpu):
    c = make_case(15, 2, 3, 4, 2, 128, [90, 40])
    c["q"][..., ::2] *= 2.0**-22
    c["q"][..., 5::7] = 0
    c["rows"] = ref.kv4_rows(np.random.default_rng(3).normal(3, 1, (c["rows"].shape[0], 2, 128)).astype(np.float32),
                             np.zeros((c["rows"].shape[0], 2, 128), np.float32))
    add_rows(c)
    check(run(c), expected(c), 128)


@pytest.mark.gpu
def test_strided_captured_on_another_stream(gpu):
    c = add_rows(make_case(16, 3, 6, 8, 2, 64, [70, 0, 300]), accepted=[5, 2, 0])
    wide = torch.zeros((3, 6, 12, 64), device="cuda", dtype=torch.bfloat16)
    q = wide[:, :, 2:10]
    q.copy_(c["q"])
    x = {k: on(c[k]) for k in ("lse", "rows", "table", "lens", "accepted", "prev")}
    pool = torch.zeros((c["rows"].shape[0], 2 * c["rows"].shape[1]), dtype=torch.uint8, device="cuda")
    part = pool[:, c["rows"].shape[1]:]                         # the second of two layers that share slots
    part.copy_(x["rows"])
    sums = x["prev"].clone()

    def call():
        sd.spec_kv4_weight_sums(q, x["lse"], part, x["table"], x["lens"], 2, accept_length=x["accepted"], prev=sums,
                                scale=c["scale"])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
        graph.replay()
    torch.cuda.synchronize()
    once = expected(c)
    c["prev"] = np.where(once["touched"], once["sums"], c["prev"]).astype(np.float32)
    r = expected(c)                                             # the second time on top of the first
    for name in ("w", "parts", "far", "size", "count"):
        r[name] = r[name] * 2
    r["count"] += 2
    t = r["touched"]
    check(torch.where(torch.from_numpy(t).cuda(), sums, 55.0), r, 64)
    assert torch.equal(sums[torch.from_numpy(~t).cuda()], x["prev"][torch.from_numpy(~t).cuda()])


@pytest.mark.gpu
@pytest.mark.parametrize("D,N", [(64, 2), (64, 12), (128, 2), (128, 12)])
def test_rows_as_large_as_they_may_be(gpu, D, N):
    """scale log2(e) |q| up to 2^118 over positions whose K is zero: equal weights."""
    c = make_case(22, 2, N, 8, 2, D, [90, 0])
    zero = np.zeros((c["rows"].shape[0], 2, D), np.float32)
    c["rows"], c["scale"] = ref.kv4_rows(zero, zero), 2.0**-3
    c["q"] = torch.where(c["q"].float() < 0, -1.0, 1.0).mul(1.375 * 2.0**120).to(torch.bfloat16)  # 2^117.99
    add_rows(c)
    check(run(c), expected(c), D)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [2, 12, 40])
@pytest.mark.parametrize("spread", [20.0, 400.0])
def test_scores_far_from_zero(gpu, N, spread):
    """Scores and lse of hundreds and thousands, whose difference counts."""
    c = make_case(23, 2, N, 8, 2, 128, [300, 77], spread=spread)
    add_rows(c)
    check(run(c), expected(c), 128)


@pytest.mark.gpu
@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 1000, 1, 64), (1, 4096, 2, 64), (300, 8, 1, 64), (2, 512, 256, 64)])
def test_many_heads(gpu, N, Hq, Hkv, D):
    c = add_rows(make_case(N, 1, N, Hq, Hkv, D, [70]))
    check(run(c), expected(c), D)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [2, 20])
def test_the_same_node_twice(gpu, N):
    """A path may name a node again: another row, one position further on."""
    c = make_case(24, 2, N, 4, 2, 64, [50, 9])
    path = np.zeros((2, N), np.int32)
    path[1] = N - 1
    add_rows(c, 2, [N - 1, N - 1], path)
    check(run(c), expected(c), 64)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 40])
def test_slots_beyond_32_bits(gpu, N):
    """Rows of 1 MB: the last slots lie more than 2^32 bytes behind the first."""
    c = add_rows(make_case(25, 2, N, 4, 1, 64, [130, 3]))
    slots, far = c["rows"].shape[0], 5000
    wide = torch.zeros((far, 1 << 20), dtype=torch.uint8, device="cuda")
    wide[far - slots:, :80] = on(c["rows"])
    got = sd.spec_kv4_weight_sums(c["q"].cuda(), on(c["lse"]), wide[:, :80], on(c["table"] + far - slots), on(c["lens"]), 1,
                                  prev=on(c["prev"]), out=torch.full(c["table"].shape, 55.0, device="cuda"), scale=c["scale"])
    check(got, expected(c), 64)


def wide_groups(rng, slots, Hkv, D, span):
    """K whose groups of 32 channels reach from one value to another `span`
    further on: the cache's whole range, spans on both sides of fp16's largest
    over the groups, or every third group far wider than the others."""
    u = rng.random((slots, Hkv, D // 32, 32))
    u[..., 0], u[..., 1] = 0, 1
    width = {"all": np.full(u.shape[:3], 2 * 57344.0), "border": rng.uniform(65000, 66500, u.shape[:3]),
             "some": np.where(rng.random(u.shape[:3]) < 1 / 3, 2 * 57344.0, 3.0)}[span][..., None]
    least = np.where(width < 100, -1.5, -57344.0 + rng.random(width.shape) * (2 * 57344.0 - width))
    return (least + u * width).reshape(slots, Hkv, D).astype(np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G", [(4, 4), (12, 4), (33, 4)])
@pytest.mark.parametrize("span", ["all", "border", "some"])
def test_groups_wider_than_half_precision(gpu, D, N, G, span):
    """The cache holds K up to +-57344, so code times step may pass fp16's
    largest; q is small enough that scores stay near one."""
    c = make_case(18, 2, N, 2 * G, 2, D, [300, 45])
    rng = np.random.default_rng(D + N)
    slots = c["rows"].shape[0]
    c["rows"] = ref.kv4_rows(wide_groups(rng, slots, 2, D, span), rng.normal(0, 1, (slots, 2, D)).astype(np.float32))
    c["q"] = (c["q"].float() * 2.0**-15).to(torch.bfloat16)
    add_rows(c)
    got = run(c)
    check(got, expected(c), D)
    assert torch.equal(got, run(c))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,spread", [(4, 0), (12, 0), (33, 0), (33, 20)])
def test_few_wide_groups(gpu, D, N, spread):
    """Tiles with a wide group among tiles without, over several heads, segments and
    requests; rows of one size and of many."""
    c = make_case(19, 3, N, 8, 2, D, [9001, 0, 700])
    rng = np.random.default_rng(D + N)
    slots = c["rows"].shape[0]
    k = rng.normal(0, 1, (slots, 2, D)).astype(np.float32)
    at = rng.random(slots) < 0.003
    k[at] = wide_groups(rng, int(at.sum()), 2, D, "all") * (rng.random((int(at.sum()), 2, D // 32)) < 0.5).repeat(32, 2)
    c["rows"] = ref.kv4_rows(k, k)
    size = 2.0 ** -rng.integers(0, spread + 1, (3, N, 8)) * 2.0**-15
    c["q"] = (c["q"].float() * torch.from_numpy(size)[..., None].float()).to(torch.bfloat16)
    add_rows(c)
    got = run(c)
    check(got, expected(c), D)
    assert torch.equal(got, run(c))
