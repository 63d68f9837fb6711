"""The bounded cache's operators together, as steps use them: attention with and
without a window, verification, compaction, the accepted path's weights added to
the positions' sums, eviction, and the next step over what was kept; eager,
captured, and under the bounds-checking build."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import speculative_decoding_draft_select_gb300 as sd
from oracle import target as ref
from speculative_decoding_draft_select_gb300 import pipeline as pl
from speculative_decoding_draft_select_gb300.build import build

from test_kv4_attention import check
from test_weight_sums import check as check_sums

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
B, TOPK, STEPS, N, V, HQ, HKV, D = 4, 3, 3, 12, 700, 8, 2, 64
CTX, BUDGET, LIMIT, SINKS, RECENT, WINDOW = 192, 96, 120, 4, 16, 40


def test_numbers_of_more_than_32_bits():
    """ctypes cuts them to their lowest bits: -2^40 would be 0."""
    assert sd._i32(-5, "sinks") == -5 and sd._i32(2**31 - 1, "sinks") == 2**31 - 1
    assert sd._i32(2**40, "window", clamp=True) == 2**31 - 1 and sd._i32(7, "window", clamp=True) == 7
    for x in (2**31, 2**40, -2**31 - 1, -2**40):
        with pytest.raises(ValueError):
            sd._i32(x, "sinks")
        if x < 0:
            with pytest.raises(ValueError):
                sd._i32(x, "window", clamp=True)


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    return sd.lib()


def inputs(seed, page):
    rng = np.random.default_rng(seed)
    lens = np.array([0, 115, 150, 119], np.int32)
    pages = CTX // page
    perm = rng.permutation(B * pages).reshape(B, pages)
    pos = np.arange(CTX)
    table = np.ascontiguousarray(perm[:, pos // page] * page + pos % page, np.int32)
    f = lambda *s: torch.from_numpy(rng.normal(0, 1, s).astype(np.float32))  # noqa: E731
    kv = lambda n: f(B, n, HKV, D).to(torch.bfloat16)  # noqa: E731
    target = f(B, N, V) * 2
    target[:, :, 5] += 30 * (torch.arange(N) % 2 == 0)        # a token that the drafts below name too
    draft = f(B + (STEPS - 1) * B * TOPK, V)
    draft[:, 5] += 12
    return {
        "lens": torch.from_numpy(lens), "table": torch.from_numpy(table),
        "pool": torch.zeros((B * pages * page, sd.spec_kv4_slot_bytes(HKV, D)), dtype=torch.uint8),
        "ctx_k": kv(150), "ctx_v": kv(150), "k": kv(N), "v": kv(N), "q": f(B, N, HQ, D).to(torch.bfloat16),
        "draft": draft.to(torch.bfloat16), "root": torch.from_numpy(rng.integers(0, V, B).astype(np.int32)),
        "target": target.to(torch.bfloat16), "sums": torch.from_numpy(rng.exponential(1.0, (B, CTX)).astype(np.float32)),
    }


def fill(x):
    sd.spec_kv4_append(x["ctx_k"], x["ctx_v"], x["pool"], x["table"], torch.zeros_like(x["lens"]), num_nodes=x["lens"])


def outputs():
    o = {n: torch.zeros((B, N, HQ, D), dtype=torch.bfloat16, device="cuda") for n in ("full", "near")}
    o["lse"] = torch.zeros((B, N, HQ), device="cuda")
    return o


def step(buf, x, o, page):
    pl.run_draft(buf, x["draft"], 1.0, x["root"], x["lens"])
    pl.run_kv4_append(buf, x["k"], x["v"], x["lens"], x["table"], x["pool"])
    pl.run_attention(buf, x["q"], x["lens"], x["table"], x["pool"], HKV, out=o["full"], lse=o["lse"])
    pl.run_attention(buf, x["q"], x["lens"], x["table"], x["pool"], HKV, out=o["near"], window=WINDOW, sinks=SINKS)
    pl.run_verify(buf, x["target"], "greedy")
    pl.run_compact(buf, x["lens"], x["table"], page, kv_pool=x["pool"])
    pl.run_weight_sums(buf, x["q"], o["lse"], x["lens"], x["table"], x["pool"], HKV, x["sums"])
    return pl.run_evict(buf, x["sums"], buf.compact_out["new_kv_len"], x["table"], page, BUDGET, limit=LIMIT, sinks=SINKS,
                        recent=RECENT, kv_pool=x["pool"] if page > 1 else None)


def verify_step(buf, x, o, out, start, page):
    """Every stage against the plain statements; x: after the step, start: before."""
    tree = {k: v.cpu().numpy() for k, v in buf.tree.items()}
    lens, table = start["lens"].numpy(), start["table"].numpy().copy()
    new = ref.kv4_rows(start["k"].float().numpy().reshape(-1, HKV, D),
                       start["v"].float().numpy().reshape(-1, HKV, D)).reshape(B, N, -1)
    pool = start["pool"].numpy().copy()
    for b in range(B):
        pool[table[b, lens[b]:lens[b] + N]] = new[b]
    q = start["q"].float().numpy()
    same = dict(tree_mask=tree["tree_mask"])
    check(o["full"], o["lse"], ref.kv4_attention(q, pool, table, lens, HKV, D ** -0.5, **same))
    check(o["near"], None, ref.kv4_attention(q, pool, table, lens, HKV, D ** -0.5, window=WINDOW, sinks=SINKS,
                                             positions=tree["positions"], **same))
    path, acc = (buf.verify_out[n].cpu().numpy() for n in ("accept_path", "accept_length"))
    length = buf.compact_out["new_kv_len"].cpu().numpy()
    assert (length == lens + acc + 1).all()
    for b in range(B):                                          # what compaction leaves
        if page == 1:
            table[b, lens[b]:length[b]] = table[b, lens[b] + path[b, :acc[b] + 1]]
        else:
            for i in range(acc[b] + 1):
                pool[table[b, lens[b] + i]] = new[b, path[b, i]]
    r = ref.kv4_weight_sums(q, o["lse"].cpu().numpy(), pool, table, lens, HKV, D ** -0.5, accept_path=path,
                            accept_length=acc, prev=start["sums"].numpy())
    # the sums themselves have been cut: they are read where nothing was
    sums, kept = x["sums"].cpu(), out["kept"].cpu().numpy()
    before = torch.from_numpy(r["sums"].astype(np.float32))
    cut = length > LIMIT
    whole = {k: v[~cut] for k, v in r.items()}
    check_sums(torch.where(torch.from_numpy(whole["touched"]), sums[torch.from_numpy(~cut)], 55.0), whole, D)
    assert cut.any() and not cut.all()
    for b in range(B):
        if not cut[b]:
            assert (kept[b] == -1).all() and int(out["new_kv_len"][b]) == length[b]
            continue
        at = kept[b]
        assert int(out["new_kv_len"][b]) == BUDGET and (np.diff(at) > 0).all()
        assert at[:SINKS].tolist() == list(range(SINKS))
        assert at[-RECENT:].tolist() == list(range(length[b] - RECENT, length[b]))
        # the kept of the middle are no smaller than the others, as far as the sums are known
        rest = np.setdiff1d(np.arange(SINKS, length[b] - RECENT), at)
        middle = at[SINKS:-RECENT]
        assert before[b, middle].min() >= before[b, rest].max() * (1 - 1e-4)
        assert torch.allclose(sums[b, :BUDGET], before[b, at], rtol=1e-4) and (sums[b, BUDGET:length[b]] == 0).all()
        rows = pool[table[b, at]]
        after = x["table"].cpu().numpy()[b, :BUDGET]
        np.testing.assert_array_equal(x["pool"].cpu().numpy()[after], rows)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 16])
def test_steps_together(gpu, page):
    x = {k: v.cuda() for k, v in inputs(page, page).items()}
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=page)
    fill(x)
    o = outputs()
    for _ in range(2):
        start = {k: v.cpu().clone() for k, v in x.items()}
        out = step(buf, x, o, page)
        torch.cuda.synchronize()
        verify_step(buf, x, o, out, start, page)
        # the next step goes on behind what was kept (longer again, so that some are cut)
        x["lens"].copy_(out["new_kv_len"])
        grow = torch.where(x["lens"] == BUDGET, 25, 0).to(torch.int32)
        sd.spec_kv4_append(x["ctx_k"], x["ctx_v"], x["pool"], x["table"], x["lens"], num_nodes=grow)
        x["lens"] += grow
        if page == 1:  # slots behind the budget are the caller's to hand out again: fresh ones here
            x["table"].copy_(torch.arange(B * CTX, device="cuda", dtype=torch.int32).view(B, CTX))
            x["pool"].zero_()
            sd.spec_kv4_append(x["ctx_k"], x["ctx_v"], x["pool"], x["table"], torch.zeros_like(x["lens"]),
                               num_nodes=x["lens"])
    assert int(buf.stats[sd.STATS["bad_request"]]) == 0 and int(buf.stats[sd.STATS["wait_timeout"]]) == 0


@pytest.mark.gpu
def test_captured_step(gpu):
    page = 16
    x = {k: v.cuda() for k, v in inputs(5, page).items()}
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=page)
    fill(x)
    o, kept = outputs(), {}
    graph = pl.capture_step(lambda: kept.update(step(buf, x, o, page)))
    fresh = inputs(6, page)
    for k, v in fresh.items():
        x[k].copy_(v)
    fill(x)
    start = {k: v.cpu().clone() for k, v in x.items()}
    graph.replay()
    torch.cuda.synchronize()
    verify_step(buf, x, o, kept, start, page)


@pytest.mark.gpu
def test_two_captured_calls_do_not_share_a_workspace(gpu):
    """Sums of many rows and of few by one buf: each size keeps its own."""
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=16)
    x = {k: v.cuda() for k, v in inputs(7, 16).items()}
    fill(x)
    sd.spec_kv4_append(x["k"], x["v"], x["pool"], x["table"], x["lens"])
    buf.verify_out["accept_length"].fill_(N - 1)
    buf.verify_out["accept_path"].copy_(torch.arange(N, device="cuda").expand(B, N))
    lse = torch.zeros((B, N, HQ), device="cuda")
    got, graphs = [], []
    for heads in (HQ, HKV):                                     # 48 and 12 rows a KV head
        q, z = x["q"][:, :, :heads].contiguous(), lse[:, :, :heads].contiguous()
        sums = torch.zeros((B, CTX), device="cuda")
        graphs.append(pl.capture_step(lambda: pl.run_weight_sums(buf, q, z, x["lens"], x["table"], x["pool"], HKV, sums)))
        got.append((q, z, sums))
    held = {n: w.data_ptr() for n, w in buf.sums_ws.items()}
    assert len(held) == 1
    for q, z, sums in got:
        sums.zero_()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert {n: w.data_ptr() for n, w in buf.sums_ws.items()} == held
    for q, z, sums in got:
        r = ref.kv4_weight_sums(q.float().cpu().numpy(), z.cpu().numpy(), x["pool"].cpu().numpy(), x["table"].cpu().numpy(),
                                x["lens"].cpu().numpy(), HKV, D ** -0.5, prev=np.zeros((B, CTX)))
        check_sums(torch.where(torch.from_numpy(r["touched"]).cuda(), sums, 55.0), r, D)


@pytest.mark.gpu
def test_text_longer_than_the_cache(gpu):
    """After an eviction the drafts stand behind the text, the cache is shorter:
    the windows are those of the cache."""
    x = {k: v.cuda() for k, v in inputs(8, 16).items()}
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=16)
    fill(x)
    sd.spec_kv4_append(x["k"], x["v"], x["pool"], x["table"], x["lens"])
    got, positions = [], []
    for text in (x["lens"], x["lens"] + torch.tensor([0, 7, 4000, 2**30], dtype=torch.int32, device="cuda")):
        pl.run_draft(buf, x["draft"], 1.0, x["root"], text)
        positions.append(buf.tree["positions"] - text[:, None])
        got += [pl.run_attention(buf, x["q"], x["lens"], x["table"], x["pool"], HKV, window=w, sinks=SINKS)
                for w in (2, WINDOW)]
    assert torch.equal(positions[0], positions[1]) and int(positions[0].max()) < N - 1
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])


@pytest.mark.gpu
def test_cut_again(gpu):
    """The lengths of one cut go into the next as a copy; the held tensor itself,
    which the next cut writes, is refused before anything is launched."""
    x = {k: v.cuda() for k, v in inputs(9, 16).items()}
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=16)
    cut = dict(sinks=SINKS, recent=RECENT, kv_pool=x["pool"])
    first = pl.run_evict(buf, x["sums"], x["lens"], x["table"], 16, BUDGET, **cut)
    assert first["new_kv_len"].tolist() == [0, BUDGET, BUDGET, BUDGET]
    before = x["sums"].clone()
    with pytest.raises(sd.SpecError):
        pl.run_evict(buf, x["sums"], first["new_kv_len"], x["table"], 16, BUDGET, **cut)
    assert torch.equal(before, x["sums"]) and first["new_kv_len"].tolist() == [0, BUDGET, BUDGET, BUDGET]
    grown = first["new_kv_len"] + 1
    again = pl.run_evict(buf, x["sums"], grown, x["table"], 16, BUDGET, **cut)
    assert again is first and again["new_kv_len"].tolist() == [1, BUDGET, BUDGET, BUDGET]


def sums_case(buf, seed, heads):
    """run_weight_sums's inputs of whole chains of nodes, and what it has to give."""
    x = {k: v.cuda() for k, v in inputs(seed, 16).items()}
    fill(x)
    sd.spec_kv4_append(x["k"], x["v"], x["pool"], x["table"], x["lens"])
    buf.verify_out["accept_length"].fill_(N - 1)
    buf.verify_out["accept_path"].copy_(torch.arange(N, device="cuda").expand(B, N))
    rng = np.random.default_rng(seed)
    x["q"] = torch.from_numpy(rng.normal(0, 1, (B, N, heads, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    x["lse"] = torch.from_numpy(rng.normal(4, 1, (B, N, heads)).astype(np.float32)).cuda()
    x["sums"] = torch.zeros((B, CTX), device="cuda")
    r = ref.kv4_weight_sums(x["q"].float().cpu().numpy(), x["lse"].cpu().numpy(), x["pool"].cpu().numpy(),
                            x["table"].cpu().numpy(), x["lens"].cpu().numpy(), HKV, D ** -0.5)
    return x, r


def check_case(x, r):
    check_sums(torch.where(torch.from_numpy(r["touched"]).cuda(), x["sums"], 55.0), r, D)


@pytest.mark.gpu
def test_workspaces_of_two_sizes(gpu):
    """Captured calls of 48 and of 144 rows a KV head: each keeps its own, and the
    first's is still its own when the second has been captured."""
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=16)
    cases = [sums_case(buf, 11, 4 * HKV), sums_case(buf, 12, 12 * HKV)]
    graphs, held = [], []
    for x, _ in cases:
        graphs.append(pl.capture_step(lambda: pl.run_weight_sums(buf, x["q"], x["lse"], x["lens"], x["table"], x["pool"],
                                                                 HKV, x["sums"])))
        held.append({n: w.data_ptr() for n, w in buf.sums_ws.items()})
    assert len(held[0]) == 1 and len(set(held[1].values())) == 2 and held[0].items() <= held[1].items()
    for order in ((0, 1), (1, 0)):
        for x, _ in cases:
            x["sums"].zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for x, r in cases:
            check_case(x, r)
    assert {n: w.data_ptr() for n, w in buf.sums_ws.items()} == held[1]


@pytest.mark.gpu
def test_layers_side_by_side(gpu):
    """Two layers' sums and cuts on two streams, each with tensors of its own."""
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=16)
    streams, layers = [torch.cuda.Stream() for _ in range(2)], []
    for seed in (13, 14):
        x, r = sums_case(buf, seed, 4 * HKV)
        ws = torch.empty(sd.spec_kv4_weight_sums_ws_size(B, N, 4 * HKV, HKV, D), dtype=torch.uint8, device="cuda")
        c = {k: v.cuda() for k, v in inputs(seed, 16).items()}
        new = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        out = {"kept": new(B, BUDGET), "freed": new(sd.spec_evict_freed_capacity(B, CTX, 16, BUDGET)), "num_freed": new(1),
               "new_kv_len": new(B)}
        cut_ws = torch.empty(sd.spec_evict_ws_size(B, 16, BUDGET), dtype=torch.uint8, device="cuda")
        layers.append((x, r, ws, c, out, cut_ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, (x, r, ws, c, out, cut_ws) in zip(streams, layers):
            with torch.cuda.stream(stream):
                x["sums"].zero_()
                pl.run_weight_sums(buf, x["q"], x["lse"], x["lens"], x["table"], x["pool"], HKV, x["sums"], ws=ws)
                got = pl.run_evict(buf, c["sums"].clone(), c["lens"], c["table"], 16, BUDGET, sinks=SINKS, recent=RECENT,
                                   out=out, ws=cut_ws)
                assert got is out
    torch.cuda.synchronize()
    assert not buf.sums_ws and not buf.evict_out
    for x, r, ws, c, out, cut_ws in layers:
        check_case(x, r)
        w = ref.evict(c["sums"].cpu().numpy(), c["lens"].cpu().numpy(), c["table"].cpu().numpy(), 16, BUDGET, BUDGET, SINKS,
                      RECENT)
        np.testing.assert_array_equal(out["kept"].cpu().numpy(), w["kept"])
        assert out["freed"][:int(out["num_freed"])].tolist() == w["freed"]
        np.testing.assert_array_equal(out["new_kv_len"].cpu().numpy(), w["new_kv_len"])


@pytest.mark.gpu
def test_refusals_of_numbers_beyond_32_bits(gpu):
    x = {k: v.cuda() for k, v in inputs(10, 16).items()}
    start = {k: x[k].clone() for k in ("sums", "table")}
    for sinks, window in ((-2**40, 5), (0, -2**40 + 5), (2, -2**32 + 1)):
        with pytest.raises(ValueError):
            sd.spec_kv4_attention_window(x["q"], x["pool"], x["table"], x["lens"], HKV, sinks, window)
    for name in ("page_size", "budget", "limit", "sinks", "recent"):
        a = {**dict(page_size=1, budget=BUDGET, limit=LIMIT, sinks=SINKS, recent=RECENT), name: -2**32 + 1}
        with pytest.raises(ValueError):
            sd.spec_evict_slots(x["sums"], x["lens"], x["table"], **a)
    assert all(torch.equal(x[k], v) for k, v in start.items())


@pytest.mark.gpu
@pytest.mark.timeout(1200)
def test_under_the_bounds_checking_build():
    """The new calls' tests against libspecdec_debug.so: no index that depends
    on the inputs leaves its buffer (conftest checks each test's count)."""
    if os.environ.get("SPECDEC_DEBUG") == "1":
        pytest.skip("already inside the debug run")
    build(debug=True)
    cmd = [sys.executable, "-m", "pytest", "tests/test_kv4_window.py", "tests/test_weight_sums.py", "tests/test_evict.py",
           "tests/test_bounded_cache.py", "-m", "gpu", "-q", "-p", "no:cacheprovider"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, SPECDEC_DEBUG="1"), capture_output=True, text=True, timeout=1100)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " error" not in r.stdout, tail
