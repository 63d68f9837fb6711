"""spec_evict_slots against its plain statement: whole numbers and copies, so
every output has to be equal."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_draft_select_gb300 as sd
from oracle import target as ref
from speculative_decoding_draft_select_gb300.build import build

from test_kv4_attention import slot_table

BAD = sd.STATS["bad_request"]


def make(seed, lens, ctx, page, width=48, spread=3.0):
    rng = np.random.default_rng(seed)
    B = len(lens)
    table, slots = slot_table(rng, B, ctx, page)
    sums = np.exp(rng.normal(0, spread, table.shape)).astype(np.float32)
    sums[rng.random(table.shape) < 0.1] = 0
    return {"lens": np.asarray(lens, np.int32), "table": table, "sums": sums,
            "rows": rng.integers(0, 256, (slots, width)).astype(np.uint8)}


def on(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run_and_check(c, page, budget, limit, sinks, recent, pool=True, apart=False, stats=None):
    x = {k: on(v) for k, v in c.items()}
    pool = x["rows"] if pool and page > 1 else None
    out_sums = torch.full(c["sums"].shape, 55.0, device="cuda") if apart else x["sums"]
    got = sd.spec_evict_slots(x["sums"], x["lens"], x["table"], page, budget, limit=limit, sinks=sinks, recent=recent,
                              kv_pool=pool, sums_out=out_sums if apart else None, stats=stats)
    r = ref.evict(c["sums"], c["lens"], c["table"], page, budget, limit, sinks, recent,
                  rows=c["rows"] if pool is not None else None)
    np.testing.assert_array_equal(got["kept"].cpu().numpy(), r["kept"])
    np.testing.assert_array_equal(got["new_kv_len"].cpu().numpy(), r["new_kv_len"])
    n = int(got["num_freed"])
    assert n == len(r["freed"]) and got["freed"][:n].tolist() == r["freed"]
    np.testing.assert_array_equal(x["table"].cpu().numpy(), r["table"])
    want = torch.from_numpy(r["sums"])
    if apart:
        inside = np.arange(c["sums"].shape[1])[None] < np.where(r["new_kv_len"] >= 0, c["lens"], 0)[:, None]
        want = torch.where(torch.from_numpy(inside), want, torch.tensor(55.0))
        assert torch.equal(x["sums"].cpu().view(torch.int32), torch.from_numpy(c["sums"]).view(torch.int32))
    assert torch.equal(out_sums.cpu().view(torch.int32), want.view(torch.int32))
    if pool is not None:
        np.testing.assert_array_equal(pool.cpu().numpy(), r["pool"])
    elif page > 1:
        np.testing.assert_array_equal(x["rows"].cpu().numpy(), c["rows"])
    return got


# ------------------------------------------------------------------------ CPU

def test_reference_by_hand():
    """Five positions to three: the first, the last and the larger of the rest."""
    sums = np.array([[0.0, 2.0, 1.0, 2.0, 0.5, 9.0]], np.float32)
    table = np.array([[10, 11, 12, 13, 14, 15]], np.int32)
    r = ref.evict(sums, [5], table, 1, 3, 3, 1, 1)
    assert r["kept"].tolist() == [[0, 1, 4]] and r["freed"] == [12, 13] and r["new_kv_len"].tolist() == [3]
    assert r["table"].tolist() == [[10, 11, 14, 13, 14, 15]] and r["sums"].tolist() == [[0, 2, 0.5, 0, 0, 9]]
    # pages of two: slots 2 p and 2 p + 1 in pages 3, 0, 2
    table = np.array([[6, 7, 0, 1, 4, 5]], np.int32)
    rows = np.arange(8, dtype=np.uint8)[:, None].repeat(4, 1)
    r = ref.evict(sums, [5], table, 2, 3, 4, 1, 1, rows=rows)
    assert r["freed"] == [2] and (r["table"] == table).all()
    assert r["pool"][:, 0].tolist() == [4, 1, 2, 3, 4, 5, 6, 7]     # place 2 (slot 0) takes position 4's
    r = ref.evict(sums, [5], table, 2, 3, 5, 1, 1)
    assert (r["kept"] == -1).all() and r["new_kv_len"].tolist() == [5] and r["freed"] == []


def test_host_checks():
    build()
    lib, null = sd.lib(), None

    def call(B=1, page=1, budget=4, limit=4, sinks=1, recent=1, lens=null, sums=null, out=null, table=null, ctx=8,
             kept=null, freed=null, cap=64, num=null, new=null, pool=null, slots=8, bps=16, ws=null, wsb=0):
        return lib.spec_evict_slots(B, page, budget, limit, sinks, recent, lens, sums, out, table, ctx, kept, freed, cap,
                                    num, new, pool, slots, bps, null, ws, wsb, null)
    assert call(B=-1) == -1 and call(page=0) == -1 and call(budget=0) == -1 and call(limit=3) == -1 and call(ctx=0) == -1
    assert call(sinks=-1) == -1 and call(recent=-1) == -1 and call(sinks=2, recent=3) == -1
    assert call(sinks=2**31 - 1, recent=2**31 - 1) == -1
    assert call(B=65536) == -2 and call(ctx=2**30) == -2 and call(budget=2**30, limit=2**30) == -2 and call() == -1
    cap = lib.spec_evict_freed_capacity
    assert cap(3, 10, 1, 4) == 18 and cap(3, 10, 4, 4) == 6 and cap(3, 10, 4, 5) == 3 and cap(3, 10, 1, 11) == 0
    assert cap(-1, 10, 1, 4) == -1 and cap(1, 0, 1, 4) == -1 and cap(1, 10, 0, 4) == -1 and cap(1, 10, 1, 0) == -1
    assert lib.spec_evict_ws_size(0, 1, 4) == 0 and lib.spec_evict_ws_size(1, 1, 0) == 0
    assert lib.spec_evict_ws_size(3, 1, 5) >= 2 * 60 and lib.spec_evict_ws_size(3, 16, 5) >= 2 * 60
    if not torch.cuda.is_available():  # made-up addresses: only where nothing could run
        p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4104)
        a = dict(lens=p, sums=p, out=p, table=p, kept=p, freed=p, num=p, new=p, ws=p, wsb=1 << 40)
        for name in ("lens", "sums", "out", "table", "kept", "freed", "num", "new", "ws"):
            assert call(**{**a, name: null}) == -1
        assert call(**{**a, "cap": 3}) == -1 and call(**{**a, "ws": odd}) == -1 and call(**{**a, "wsb": 64}) == -4
        assert call(**a, pool=odd) == -2 and call(**a, pool=p, bps=24) == -2 and call(**a, pool=p, slots=0) == -1
        assert call(**{**a, "out": ctypes.c_void_p(4100)}) == -1      # sums and their new ones overlap in part


def test_lengths_apart_from_the_results():
    """Lengths are read until the last launch ends: no result may lie over them."""
    build()
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing could run")
    at = lambda a: ctypes.c_void_p(1 << 20 | a)  # noqa: E731

    def call(B=4, page=16, lens=at(0), kept=at(0x1000), freed=at(0x2000), num=at(0x3000), new=at(0x4000), cap=64):
        return sd.lib().spec_evict_slots(B, page, 4, 4, 1, 1, lens, at(0x10000), at(0x20000), at(0x30000), 8, kept, freed,
                                         cap, num, new, at(0x40000), 8, 16, None, at(0x50000), 1 << 20, None)
    refused = -1
    for page in (1, 16):
        assert call(page=page) != refused
        assert call(page=page, new=at(0)) == refused                    # the lengths themselves
    assert call(new=at(12)) == refused and call(lens=at(0x400c)) == refused
    assert call(new=at(16)) != refused and call(lens=at(0x3ff0)) != refused  # neighbours
    assert call(kept=at(0)) == refused and call(lens=at(0x103c)) == refused and call(lens=at(0x1040)) != refused
    assert call(freed=at(8)) == refused and call(lens=at(0x20fc)) == refused and call(lens=at(0x2100)) != refused
    assert call(num=at(12)) == refused and call(num=at(16)) != refused


def test_binding_refuses_host_tensors():
    i = torch.zeros((1, 8), dtype=torch.int32)
    with pytest.raises(ValueError):
        sd.spec_evict_slots(torch.zeros((1, 8)), i[0, :1], i, 1, 4)


# ------------------------------------------------------------------------ GPU

@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    return sd.lib()


SETS = [
    # lens, ctx, budget, limit, sinks, recent
    ([5], 5, 3, 3, 1, 1), ([1, 0, 2], 4, 1, 1, 0, 0), ([7, 9, 8, 0, 1], 9, 8, 8, 0, 0), ([9], 12, 4, 4, 4, 0),
    ([9], 12, 4, 4, 0, 4), ([9, 30], 33, 4, 4, 2, 2), ([100, 63, 64, 65, 300], 300, 64, 64, 4, 16),
    ([100, 63, 64, 65, 300], 320, 33, 70, 3, 7), ([1500, 700], 1501, 1024, 1024, 4, 128), ([4096, 513, 0], 4096, 777, 900, 3, 129),
    ([5000, 8192], 8200, 4097, 4100, 0, 1), ([16000, 9], 16384, 100, 100, 4, 50), ([33000], 33000, 8191, 8191, 4, 1024),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,ctx,budget,limit,sinks,recent", SETS)
@pytest.mark.parametrize("page", [1, 5, 16])
def test_matches_the_statement(gpu, lens, ctx, budget, limit, sinks, recent, page):
    c = make(ctx + budget, lens, ctx, page)
    stats = sd.new_stats()
    run_and_check(c, page, budget, limit, sinks, recent, stats=stats)
    run_and_check(c, page, budget, limit, sinks, recent, apart=True, stats=stats)
    assert int(stats.sum()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 4])
@pytest.mark.parametrize("ctx", [600, 20000])
def test_ties_signs_and_what_is_no_number(gpu, page, ctx):
    c = make(1, [ctx, ctx - 7, 300, ctx], ctx, page)
    rng = np.random.default_rng(2)
    c["sums"][0] = 1.0                                        # all equal
    c["sums"][1] = rng.choice(np.array([0.0, -0.0, 1.0], np.float32), c["sums"].shape[1])
    c["sums"][2] = rng.choice(np.array([np.nan, np.inf, -np.inf, -1.0, 3.0, 1e-42], np.float32), c["sums"].shape[1])
    c["sums"][3, ::2] = np.nan
    run_and_check(c, page, 200, 250, 4, 30)
    run_and_check(c, page, 299, 299, 0, 0)


@pytest.mark.gpu
def test_one_key_apart(gpu):
    """Sums that differ in their last bits alone: the last counting pass decides."""
    c = make(3, [3000, 2999], 3000, 1)
    rng = np.random.default_rng(4)
    c["sums"][:] = (np.float32(1.0).view(np.int32) + rng.integers(0, 4000, c["sums"].shape)).astype(np.int32).view(np.float32)
    run_and_check(c, 1, 1500, 1500, 0, 0)


@pytest.mark.gpu
def test_keys_beyond_shared_memory(gpu):
    """A longer request than the cluster's shared memory holds keys of."""
    c = make(5, [150001, 3], 150001, 1)
    run_and_check(c, 1, 60000, 60000, 4, 1000)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [20, 160, 310])
def test_large_batches_in_a_wide_table(gpu, B):
    """Fewer CTAs a request, so that the longest one's keys do not all fit."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 300, B)
    lens[B // 2], lens[-1] = 40000, 9000
    run_and_check(make(B, lens, 40000, 1), 1, 120, 150, 4, 10)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [16, 112, 128, 144, 4096])
def test_payload_widths(gpu, width):
    c = make(6, [700, 90, 1200], 1201, 16, width=width)
    run_and_check(c, 16, 300, 300, 4, 20)


@pytest.mark.gpu
def test_without_a_pool_the_payload_stays(gpu):
    c = make(7, [700, 90], 701, 16)
    run_and_check(c, 16, 300, 300, 4, 20, pool=False)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 4])
def test_bad_requests_and_slots(gpu, page):
    c = make(8, [100, -1, 101, 60], 100, page)
    c["lens"][2] = c["table"].shape[1] + 1
    stats = sd.new_stats()
    c["table"][3, [50, 59, 2]] = [10**9, -5, -1]               # page > 1: two sources at the end, one place
    run_and_check(c, page, 20, 20, 2, 18, stats=stats)
    assert int(stats[BAD]) == 2 + (3 if page > 1 else 0)


@pytest.mark.gpu
def test_pages_whose_slots_are_none(gpu):
    """A freed page is named by its first slot: none of a negative one, and never page 0."""
    c = make(14, [64, 64], 64, 16, width=16)
    c["table"][0, 48], c["table"][1, 32] = -1, -17
    got = run_and_check(c, 16, 20, 20, 0, 0)
    freed = got["freed"][:int(got["num_freed"])].tolist()
    assert freed[1] == -1 and freed[2] < 0


@pytest.mark.gpu
def test_limits_beyond_32_bits(gpu):
    c = make(15, [40, 64], 64, 1)
    x = {k: on(v) for k, v in c.items()}
    got = sd.spec_evict_slots(x["sums"], x["lens"], x["table"], 1, 20, limit=2**40)
    assert got["new_kv_len"].tolist() == [40, 64] and int(got["num_freed"]) == 0
    with pytest.raises(ValueError):
        sd.spec_evict_slots(x["sums"], x["lens"], x["table"], 1, 2**40)


@pytest.mark.gpu
def test_nothing_to_do(gpu):
    c = make(9, [3, 4], 8, 1)
    got = run_and_check(c, 1, 5, 6, 1, 1)
    assert int(got["num_freed"]) == 0
    empty = sd.spec_evict_slots(torch.zeros((0, 8), device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                                torch.zeros((0, 8), dtype=torch.int32, device="cuda"), 1, 5)
    assert int(empty["num_freed"]) == 0


@pytest.mark.gpu
def test_many_requests(gpu):
    rng = np.random.default_rng(10)
    c = make(10, rng.integers(0, 90, 700), 90, 1)
    run_and_check(c, 1, 30, 40, 2, 5)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 16])
def test_captured_on_another_stream_and_again(gpu, page):
    """Two cuts of the same tensors: new sums and lengths between them."""
    c = make(11, [500, 30, 9000], 9000, page)
    x = {k: on(v) for k, v in c.items()}
    B, budget = 3, 200
    cap = sd.spec_evict_freed_capacity(B, c["table"].shape[1], page, budget)
    out = {"kept": torch.empty((B, budget), dtype=torch.int32, device="cuda"),
           "freed": torch.empty((cap,), dtype=torch.int32, device="cuda"),
           "num_freed": torch.empty((1,), dtype=torch.int32, device="cuda"),
           "new_kv_len": torch.empty((B,), dtype=torch.int32, device="cuda")}
    ws = torch.empty(sd.spec_evict_ws_size(B, page, budget), dtype=torch.uint8, device="cuda")

    def call():
        sd.spec_evict_slots(x["sums"], x["lens"], x["table"], page, budget, limit=250, sinks=3, recent=20,
                            kv_pool=x["rows"] if page > 1 else None, out=out, ws=ws)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
    torch.cuda.synchronize()
    for k, v in make(12, [500, 600, 251], 9000, page).items():
        c[k] = v
        x[k].copy_(on(v))
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph.replay()
    torch.cuda.synchronize()
    r = ref.evict(c["sums"], c["lens"], c["table"], page, budget, 250, 3, 20, rows=c["rows"] if page > 1 else None)
    np.testing.assert_array_equal(out["kept"].cpu().numpy(), r["kept"])
    assert out["freed"][:int(out["num_freed"])].tolist() == r["freed"]
    np.testing.assert_array_equal(x["table"].cpu().numpy(), r["table"])
    np.testing.assert_array_equal(x["sums"].cpu().numpy(), r["sums"])
    if page > 1:
        np.testing.assert_array_equal(x["rows"].cpu().numpy(), r["pool"])


@pytest.mark.gpu
def test_payload_beyond_32_bits(gpu):
    """Rows of 1 MB: the last slots lie more than 2^32 bytes behind the first."""
    c = make(16, [90, 31, 70], 96, 16, width=48)
    far, slots, width = 5000, c["rows"].shape[0], 1 << 20
    table = on(c["table"] + (far - slots) // 16 * 16)
    first = (far - slots) // 16 * 16
    pool = torch.zeros((far, width), dtype=torch.uint8, device="cuda")
    pool[first:first + slots, width - 48:] = on(c["rows"])
    got = sd.spec_evict_slots(on(c["sums"]), on(c["lens"]), table, 16, 40, sinks=3, recent=9, kv_pool=pool)
    r = ref.evict(c["sums"], c["lens"], c["table"], 16, 40, 40, 3, 9, rows=c["rows"])
    np.testing.assert_array_equal(got["kept"].cpu().numpy(), r["kept"])
    np.testing.assert_array_equal(pool[first:first + slots, width - 48:].cpu().numpy(), r["pool"])
    assert int(pool[:, :width - 48].sum(dtype=torch.int64)) == 0 and int(pool[:first].sum(dtype=torch.int64)) == 0
    assert got["freed"][:int(got["num_freed"])].tolist() == [p + first // 16 for p in r["freed"]]


@pytest.mark.gpu
def test_pages_larger_than_a_request(gpu):
    run_and_check(make(17, [60, 33, 50], 60, 64, width=32), 64, 40, 45, 2, 5)


@pytest.mark.gpu
def test_most_requests(gpu):
    """65535 requests, the most of a call: a few are cut."""
    rng = np.random.default_rng(18)
    lens = rng.integers(0, 9, 65535)
    lens[::1000] = 12
    run_and_check(make(18, lens, 12, 1), 1, 8, 9, 1, 2)
