"""The target pass's operators together, as a step uses them: draft tree, K and
V of its nodes into the 4-bit cache, attention under the tree mask, adjusted
logits, verify, compaction of the same cache, and the next step's attention
over what was kept; eager, captured, and under the bounds-checking build."""
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

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
B, TOPK, STEPS, N, V, HQ, HKV, D = 3, 3, 3, 12, 700, 8, 2, 64


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    return sd.lib()


def inputs(seed, page):
    rng = np.random.default_rng(seed)
    lens = np.array([0, 37, 150], np.int32)
    max_ctx = 176
    pages = max_ctx // page
    perm = rng.permutation(B * pages).reshape(B, pages)
    pos = np.arange(max_ctx)
    table = np.ascontiguousarray(perm[:, pos // page] * page + pos % page, np.int32)
    rows = B + (STEPS - 1) * B * TOPK
    f = lambda *s: torch.from_numpy(rng.normal(0, 1, s).astype(np.float32))  # noqa: E731
    kv = lambda n: f(B, n, HKV, D).to(torch.bfloat16)  # noqa: E731
    return {
        "lens": torch.from_numpy(lens), "table": torch.from_numpy(table),
        "pool": torch.zeros((B * pages * page, sd.spec_kv4_slot_bytes(HKV, D)), dtype=torch.uint8),
        "ctx_k": kv(150), "ctx_v": kv(150), "k": kv(N), "v": kv(N), "q": f(B, N, HQ, D).to(torch.bfloat16),
        "draft": f(rows, V).to(torch.bfloat16), "root": torch.from_numpy(rng.integers(0, V, B).astype(np.int32)),
        "target": (f(B, N, V) * 2).to(torch.bfloat16),
        "history": torch.from_numpy(rng.integers(0, V, (B, 20)).astype(np.int32)),
        "rep": torch.tensor([1.3, 1.0, 0.9]), "freq": torch.tensor([0.2, 0.0, 0.4]),
        "allowed": torch.from_numpy(rng.integers(-2**31, 2**31, (2, (V + 31) // 32)).astype(np.int32)),
        "allowed_row": torch.from_numpy(rng.integers(-1, 2, (B, N)).astype(np.int32)),
    }


def step(buf, x, page, out, adjusted):
    pl.run_draft(buf, x["draft"], 1.0, x["root"], x["lens"])
    pl.run_kv4_append(buf, x["k"], x["v"], x["lens"], x["table"], x["pool"])
    pl.run_attention(buf, x["q"], x["lens"], x["table"], x["pool"], HKV, out=out)
    pl.run_adjust(buf, x["target"], out=adjusted, history=x["history"], rep_penalty=x["rep"], freq_penalty=x["freq"],
                  allowed=x["allowed"], allowed_row=x["allowed_row"])
    pl.run_verify(buf, adjusted, "greedy")
    pl.run_compact(buf, x["lens"], x["table"], page, kv_pool=x["pool"])


def verify_step(buf, x, start, page, out, adjusted):
    """Every stage against the plain statements; x: after the step, start: before."""
    tree = {k: v.cpu().numpy() for k, v in buf.tree.items()}
    lens, table = start["lens"].numpy(), start["table"].numpy()
    n_rows = ref.kv4_rows(start["k"].float().numpy().reshape(-1, HKV, D),
                          start["v"].float().numpy().reshape(-1, HKV, D)).reshape(B, N, -1)
    pool = start["pool"].numpy().copy()
    for b in range(B):
        pool[table[b, lens[b]:lens[b] + N]] = n_rows[b]
    r = ref.kv4_attention(start["q"].float().numpy(), pool, table, lens, HKV, D ** -0.5, tree_mask=tree["tree_mask"])
    check(out, None, r)
    want = ref.adjust_logits(start["target"].float().numpy(), history=start["history"].numpy(), rep=start["rep"].numpy(),
                             freq=start["freq"].numpy(), draft=tree["draft_token"], tree_mask=tree["tree_mask"],
                             allowed=start["allowed"].numpy(), allowed_row=start["allowed_row"].numpy())
    assert torch.equal(adjusted.cpu(), torch.from_numpy(want).to(torch.bfloat16))
    # the greedy walk over the adjusted rows, and what it leaves of the cache
    path, acc = buf.verify_out["accept_path"].cpu().numpy(), buf.verify_out["accept_length"].cpu().numpy()
    rounded = torch.from_numpy(want).to(torch.bfloat16).float().numpy()
    new_len = buf.compact_out["new_kv_len"].cpu().numpy()
    for b in range(B):
        at, kept = 0, [0]
        while True:
            t = int(np.argmax(rounded[b, at]))
            child = [m for m in range(N) if tree["parent"][b, m] == at and tree["draft_token"][b, m] == t]
            if not child:
                break
            at = child[0]
            kept.append(at)
        assert path[b, :len(kept)].tolist() == kept and acc[b] == len(kept) - 1
        assert new_len[b] == lens[b] + len(kept)
        slots = x["table"].cpu().numpy()[b, lens[b]:new_len[b]]
        np.testing.assert_array_equal(x["pool"].cpu().numpy()[slots], n_rows[b, kept])


def fill(x):
    sd.spec_kv4_append(x["ctx_k"], x["ctx_v"], x["pool"], x["table"], torch.zeros_like(x["lens"]), num_nodes=x["lens"])


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 16])
def test_steps_together(gpu, page):
    x = {k: v.cuda() for k, v in inputs(page, page).items()}
    # a drafted child is the target's choice in some rows, so that paths are kept
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=page)
    fill(x)
    out, adjusted = torch.empty_like(x["q"]), torch.empty_like(x["target"])
    tree = pl.run_draft(buf, x["draft"], 1.0, x["root"], x["lens"])
    first = tree["retrieve_next_token"].long().clamp(min=0)
    tok = tree["draft_token"].long().gather(1, first)
    x["target"].scatter_add_(2, tok[..., None], torch.full_like(tok[..., None], 30, dtype=torch.bfloat16))
    for turn in range(2):
        start = {k: v.cpu().clone() for k, v in x.items()}
        step(buf, x, page, out, adjusted)
        torch.cuda.synchronize()
        verify_step(buf, x, start, page, out, adjusted)
        # the next step begins where this one's accepted path ends
        x["lens"].copy_(buf.compact_out["new_kv_len"])
        if turn == 0:
            assert int(buf.verify_out["accept_length"].max()) >= 1
    assert int(buf.stats[sd.STATS["bad_request"]]) == 0 and int(buf.stats[sd.STATS["wait_timeout"]]) == 0


@pytest.mark.gpu
def test_captured_step(gpu):
    page = 16
    x = {k: v.cuda() for k, v in inputs(5, page).items()}
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=page)
    fill(x)
    out, adjusted = torch.empty_like(x["q"]), torch.empty_like(x["target"])
    graph = pl.capture_step(lambda: step(buf, x, page, out, adjusted))
    fresh = inputs(6, page)
    for k, v in fresh.items():
        x[k].copy_(v)
    fill(x)
    start = {k: v.cpu().clone() for k, v in x.items()}
    graph.replay()
    torch.cuda.synchronize()
    verify_step(buf, x, start, page, out, adjusted)


@pytest.mark.gpu
def test_captured_steps_of_two_head_layouts(gpu):
    """One buf serves layers of different heads: the larger workspace does not
    replace the one that a captured call holds."""
    page = 16
    x = {k: v.cuda() for k, v in inputs(8, page).items()}
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=page)
    pl.run_draft(buf, x["draft"], 1.0, x["root"], x["lens"])
    fill(x)
    pl.run_kv4_append(buf, x["k"], x["v"], x["lens"], x["table"], x["pool"])
    narrow = x["q"][:, :, :HKV].contiguous()  # one query head a KV head
    few, many = torch.empty_like(narrow), torch.empty_like(x["q"])
    graph = pl.capture_step(lambda: pl.run_attention(buf, narrow, x["lens"], x["table"], x["pool"], HKV, out=few))
    held = {n: w.data_ptr() for n, w in buf.attention_ws.items()}
    pl.run_attention(buf, x["q"], x["lens"], x["table"], x["pool"], HKV, out=many)
    assert len(held) == 1 and len(buf.attention_ws) == 2
    assert all(buf.attention_ws[n].data_ptr() == at for n, at in held.items())
    few.zero_()
    graph.replay()
    torch.cuda.synchronize()
    mask = buf.tree["tree_mask"].cpu().numpy()
    for q, out in ((narrow, few), (x["q"], many)):
        check(out, None, ref.kv4_attention(q.float().cpu().numpy(), x["pool"].cpu().numpy(), x["table"].cpu().numpy(),
                                           x["lens"].cpu().numpy(), HKV, D ** -0.5, tree_mask=mask))


@pytest.mark.gpu
@pytest.mark.timeout(1200)
def test_under_the_bounds_checking_build():
    """The new calls' tests against libspecdec_debug.so: no index that depends
    on the inputs leaves its buffer (conftest checks each test's count)."""
    if os.environ.get("SPECDEC_DEBUG") == "1":
        pytest.skip("already inside the debug run")
    build(debug=True)
    cmd = [sys.executable, "-m", "pytest", "tests/test_adjust_logits.py", "tests/test_kv4_cache.py",
           "tests/test_kv4_attention.py", "tests/test_target_step.py", "-m", "gpu", "-k", "not gigabytes", "-q", "-p",
           "no:cacheprovider"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, SPECDEC_DEBUG="1"), capture_output=True, text=True, timeout=1100)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " error" not in r.stdout, tail


@pytest.mark.gpu
def test_two_layers_on_two_streams(gpu):
    """Two layers of one layout at once, each with a workspace of its own; the buffers' is not touched."""
    page = 16
    x = {k: v.cuda() for k, v in inputs(9, page).items()}
    buf = pl.StepBuffers("tree", B, TOPK, STEPS, N, V, "cuda", want_q=False, page_size=page)
    pl.run_draft(buf, x["draft"], 1.0, x["root"], x["lens"])
    fill(x)
    pl.run_kv4_append(buf, x["k"], x["v"], x["lens"], x["table"], x["pool"])
    q2 = -x["q"]
    size = sd.spec_kv4_attention_ws_size(B, N, HQ, HKV, D)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.empty_like(x["q"]) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(side):
            pl.run_attention(buf, q2, x["lens"], x["table"], x["pool"], HKV, out=out[1], ws=ws[1])
        pl.run_attention(buf, x["q"], x["lens"], x["table"], x["pool"], HKV, out=out[0], ws=ws[0])
    torch.cuda.synchronize()
    assert not buf.attention_ws
    mask = buf.tree["tree_mask"].cpu().numpy()
    for q, o in ((x["q"], out[0]), (q2, out[1])):
        check(o, None, ref.kv4_attention(q.float().cpu().numpy(), x["pool"].cpu().numpy(), x["table"].cpu().numpy(),
                                         x["lens"].cpu().numpy(), HKV, D ** -0.5, tree_mask=mask))
