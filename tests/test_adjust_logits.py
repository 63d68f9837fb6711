"""spec_adjust_logits: penalties, biases and grammar masks on the logits of a
tree's nodes, bit for bit against a plain statement in the same precision."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_draft_select_gb300 as sd
from oracle import target as ref
from speculative_decoding_draft_select_gb300.build import build


def random_mask(rng, B, N):
    mask = np.zeros((B, N, N), np.uint8)
    mask[:, 0, 0] = 1
    for b in range(B):
        for n in range(1, N):
            mask[b, n] = mask[b, rng.integers(0, n)]
            mask[b, n, n] = 1
    return mask


def make_case(seed, B, N, V, dtype, H=40, M=6, few=7, edges=True):
    """Inputs whose tokens crowd on `few` ids, so that histories, paths,
    biases and masks meet on the same tokens."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 3, (B, N, V)).astype(np.float32)
    if edges:
        flat = x.reshape(-1)
        for value in (np.nan, np.inf, -np.inf, 0.0, -0.0, np.finfo(np.float32).min):
            flat[rng.integers(0, flat.size, max(1, flat.size // 50))] = value
    hot = rng.integers(0, V, few)
    ids = lambda *s: np.where(rng.random(s) < 0.8, rng.choice(hot, s), rng.integers(-3, V + 3, s)).astype(np.int32)  # noqa: E731
    words = (V + 31) // 32
    c = {
        "x": torch.from_numpy(x).to(dtype),
        "history": ids(B, H), "history_lens": rng.integers(0, H + 1, B).astype(np.int32),
        "prompt_lens": rng.integers(0, H + 1, B).astype(np.int32),
        "rep": rng.uniform(0.7, 1.6, B).astype(np.float32), "freq": rng.uniform(-0.3, 0.6, B).astype(np.float32),
        "pres": rng.uniform(-0.3, 0.6, B).astype(np.float32), "draft": ids(B, N), "tree_mask": random_mask(rng, B, N),
        "bias_ids": ids(B, M), "bias_vals": rng.normal(0, 3, (B, M)).astype(np.float32),
        "allowed": rng.integers(-2**31, 2**31, (B * N + 2, words)).astype(np.int32),
        "allowed_row": rng.integers(-1, B * N + 2, (B, N)).astype(np.int32),
    }
    c["allowed"][0] = 0  # a row that allows nothing
    return c


NAMES = {"history": "history", "history_lens": "history_lens", "prompt_lens": "prompt_lens", "rep": "rep_penalty",
         "freq": "freq_penalty", "pres": "pres_penalty", "draft": "draft_token", "tree_mask": "tree_mask",
         "bias_ids": "bias_ids", "bias_vals": "bias_vals", "allowed": "allowed", "allowed_row": "allowed_row",
         "num_nodes": "num_nodes"}


def on_gpu(c, keep=None):
    return {NAMES[k]: torch.from_numpy(v).cuda() for k, v in c.items() if k != "x" and (keep is None or k in keep)}


def expected(c, keep=None):
    args = {k: v for k, v in c.items() if k != "x" and (keep is None or k in keep)}
    return torch.from_numpy(ref.adjust_logits(c["x"].float().numpy(), **args)).to(c["x"].dtype)


def same(got, want):
    got, want = got.cpu(), want
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.float(), nan=7.0), torch.nan_to_num(want.float(), nan=7.0))


# ------------------------------------------------------------------------ CPU

def test_reference_by_hand():
    x = np.array([[[2.0, -2.0, 1.0, 0.5], [2.0, -2.0, 1.0, 0.5]]], np.float32)
    out = ref.adjust_logits(x, history=np.array([[0, 1, 1]], np.int32), prompt_lens=np.array([1]), rep=np.array([2.0]),
                            freq=np.array([0.25]), pres=np.array([0.5]), draft=np.array([[1, 2]], np.int32),
                            bias_ids=np.array([[3, 3]], np.int32), bias_vals=np.array([[1.0, 2.0]], np.float32),
                            allowed=np.array([[15], [7]], np.int32))
    # row 0: token 0 in the prompt, token 1 twice in the answer; row 1 also token 2 once, token 3 masked
    np.testing.assert_array_equal(out[0, 0], [1.0, -4.0 - 0.5 - 0.5, 1.0, 3.5])
    np.testing.assert_array_equal(out[0, 1], [1.0, -5.0, 0.5 - 0.25 - 0.5, -np.inf])


def test_host_checks():
    build()
    lib, null = sd.lib(), None

    def call(B=1, N=2, V=8, dtype=1, logits=null, out=null, H=0, M=0, allowed=null, rows=0):
        return lib.spec_adjust_logits(B, N, V, dtype, logits, out, null, null, H, null, null, null, null, null, null,
                                      null, null, null, M, allowed, rows, null, null, null)
    assert call(B=-1) == -1 and call(N=0) == -1 and call(V=0) == -1 and call(H=-1) == -1 and call(M=-1) == -1
    assert call(dtype=5) == -2 and call(V=(1 << 22) + 1) == -2 and call(N=2049) == -2 and call(B=65536) == -2
    assert call(H=(1 << 28) + 1) == -2
    assert call(B=0) == 0
    assert call() == -1          # no logits
    assert call(M=3) == -1       # biases announced, none given
    if not torch.cuda.is_available():  # made-up addresses: only where nothing could run
        p, q = ctypes.c_void_p(4096), ctypes.c_void_p(4098)
        assert call(logits=p, out=q) == -1                      # overlapping, not in place
        assert call(logits=ctypes.c_void_p(4097), out=p) == -1  # not element aligned
        assert call(logits=p, out=p, allowed=p, rows=1) == -1   # two rows of nodes, one mask row


def test_binding_refuses():
    x = torch.zeros((1, 2, 8))
    with pytest.raises(ValueError):
        sd.spec_adjust_logits(x)


# ------------------------------------------------------------------------ GPU

@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    return sd.lib()


SHAPES = [(1, 1, 1), (1, 1, 31), (2, 1, 33), (3, 2, 4096), (2, 3, 4097), (4, 9, 1000), (1, 2, 50257), (5, 17, 515),
          (1, 64, 8200), (700, 1, 40)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,V", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matches_reference(gpu, B, N, V, dtype):
    c = make_case(B * 31 + N * 7 + V, B, N, V, dtype)
    x = c["x"].cuda()
    args = on_gpu(c)
    out = sd.spec_adjust_logits(x, out=torch.empty_like(x), **args)
    want = expected(c)
    same(out, want)
    same(x, c["x"])  # the input is left as it was
    assert sd.spec_adjust_logits(x, **args) is x  # in place
    same(x, want)


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [(), ("history",), ("history", "rep"), ("history", "freq", "pres", "history_lens"),
                                  ("draft", "rep", "freq"), ("draft", "tree_mask", "pres"), ("bias_ids", "bias_vals"),
                                  ("allowed", "allowed_row"), ("allowed",)])
def test_parts_alone(gpu, keep):
    c = make_case(5, 3, 6, 777, torch.bfloat16)
    x = c["x"].cuda()
    out = sd.spec_adjust_logits(x, out=torch.empty_like(x), **on_gpu(c, keep))
    same(out, expected(c, keep))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift_in,shift_out", [(0, 1), (1, 1), (3, 0), (5, 7)])
def test_alignments(gpu, dtype, shift_in, shift_out):
    B, N, V = 2, 5, 1003
    c = make_case(9, B, N, V, dtype)
    wide = [torch.full((B * N * V + 16,), 3.0, dtype=dtype, device="cuda") for _ in range(2)]
    x = wide[0][shift_in:shift_in + B * N * V].view(B, N, V)
    y = wide[1][shift_out:shift_out + B * N * V].view(B, N, V)
    x.copy_(c["x"])
    sd.spec_adjust_logits(x, out=y, **on_gpu(c))
    same(y, expected(c))
    assert (wide[1][:shift_out] == 3).all() and (wide[1][shift_out + B * N * V:] == 3).all()


@pytest.mark.gpu
def test_padded_batch_and_bad_requests(gpu):
    B, N, V = 5, 4, 600
    c = make_case(11, B, N, V, torch.bfloat16)
    c["num_nodes"] = np.array([4, 0, 2, -3, 9], np.int32)
    c["history_lens"][:] = [3, 0, 1000, -5, 40]  # two outside [0, H]
    c["rep"][:] = [1.2, 0.0, -1.0, np.nan, 1.0]  # of requests 0, 2, 4 (the others have no nodes), one is bad
    c["allowed_row"][:] = [[0, 1, 2, 10**6], [10**6] * 4, [3, -7, 0, 0], [0] * 4, [1, 1, 1, 1]]
    stats = sd.new_stats()
    x = c["x"].cuda()
    out = torch.full_like(x, 5.0)
    sd.spec_adjust_logits(x, out=out, stats=stats, **on_gpu(c))
    want = expected(c)
    for b, n in enumerate([4, 0, 2, 0, 4]):
        same(out[b, :n], want[b, :n])
        assert (out[b, n:] == 5).all()  # left as they were
    assert int(stats[sd.STATS["bad_request"]]) == 3  # request 2's length and penalty, one mask row


@pytest.mark.gpu
def test_long_chain_on_one_token(gpu):
    """Every node carries one of three tokens: the longest lists, in place."""
    B, N, V = 1, 300, 64
    c = make_case(13, B, N, V, torch.float32, few=3, edges=False)
    c["draft"][:] = np.arange(N) % 3
    del c["tree_mask"]
    x = c["x"].cuda()
    sd.spec_adjust_logits(x, **on_gpu(c))
    same(x, expected(c))


@pytest.mark.gpu
def test_most_nodes(gpu):
    B, N, V = 1, 2048, 70
    c = make_case(14, B, N, V, torch.bfloat16, few=30)
    c["tree_mask"] = (np.random.default_rng(3).random((B, N, N)) < 0.01).astype(np.uint8)
    c["allowed_row"][:] = -1
    x = c["x"].cuda()
    sd.spec_adjust_logits(x, **on_gpu(c))
    same(x, expected(c))


@pytest.mark.gpu
def test_captured_and_other_stream(gpu):
    c = make_case(15, 3, 8, 5000, torch.bfloat16)
    x, args = c["x"].cuda(), on_gpu(c)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sd.spec_adjust_logits(x, out=out, **args)
    side.synchronize()
    same(out, expected(c))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sd.spec_adjust_logits(x, out=out, **args)
    other = make_case(16, 3, 8, 5000, torch.bfloat16)
    x.copy_(other["x"])
    for k, v in on_gpu(other).items():
        args[k].copy_(v)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    same(out, expected(other))


@pytest.mark.gpu
def test_binding_checks(gpu):
    x = torch.zeros((2, 3, 64), device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for bad in ({"history": i(3, 4)}, {"draft_token": i(2, 2)}, {"bias_ids": i(2, 4)}, {"allowed": i(6, 3)},
                {"allowed": i(5, 2)}, {"rep_penalty": i(2)}, {"out": torch.zeros((2, 3, 65), device="cuda")},
                {"out": torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda")},
                {"allowed": i(6, 2), "allowed_row": i(3, 2)}, {"history": torch.zeros((2, 4), dtype=torch.int32)}):
        with pytest.raises((ValueError, sd.SpecError)):
            sd.spec_adjust_logits(x, **bad)
    with pytest.raises(ValueError):
        sd.spec_adjust_logits(x.half())
    with pytest.raises(ValueError):
        sd.spec_adjust_logits(x.transpose(0, 1))


def test_empty_batch():
    build()
    p = ctypes.c_void_p(4096)  # not read: there is nothing to do
    for M, rows in ((3, 0), (0, 0), (3, 2)):
        assert sd.lib().spec_adjust_logits(0, 2, 8, 1, None, None, None, None, 0, None, None, None, None, None, None, None,
                                           None, None, M, p, rows, None, None, None) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("twice", [False, True])
def test_bias_of_every_token(gpu, twice):
    B, N, V = 2, 3, 9001
    c = make_case(21, B, N, V, torch.float32)
    rng = np.random.default_rng(22)
    ids = np.stack([rng.permutation(V) for _ in range(B)]).astype(np.int32)
    if twice:  # in one chunk of the vocabulary and far apart, and side by side
        ids[0, -1], ids[1, 7] = ids[0, 0], ids[1, 6]
    c["bias_ids"], c["bias_vals"] = ids, rng.normal(0, 3, ids.shape).astype(np.float32)
    x = c["x"].cuda()
    same(sd.spec_adjust_logits(x, **on_gpu(c)), expected(c))


@pytest.mark.gpu
def test_empty_shapes_through_the_binding(gpu):
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros((0, 3, 64), device="cuda")
    assert sd.spec_adjust_logits(x, history=i(0, 4), bias_ids=i(0, 2), bias_vals=i(0, 2).float(), draft_token=i(0, 3),
                                 allowed=i(1, 2)).shape == (0, 3, 64)
    with pytest.raises(sd.SpecError):
        sd.spec_adjust_logits(torch.zeros((2, 3, 0), device="cuda"), allowed=i(2, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("B,V,N,biases", [(1000, 64, 511, True), (1000, 64, 512, True), (1000, 64, 513, True),
                                          (1000, 64, 1536, False), (500, 64, 1792, True), (1000, 64, 2048, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shared_memory_around_the_default_limit(gpu, B, V, N, biases, dtype):
    """Node counts at which a block's shared memory, the fixed part included, passes 48 KB; most rows are not live."""
    rng = np.random.default_rng(N)
    live = 3
    x = torch.zeros((B, N, V), dtype=dtype, device="cuda")
    c = make_case(N, B, live, V, dtype, edges=False)
    x[:, :live] = c["x"].cuda()
    keep = ("history", "history_lens", "rep", "freq", "draft") + (("bias_ids", "bias_vals") if biases else ())
    args = on_gpu(c, keep)
    args["draft_token"] = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    args["draft_token"][:, :live] = torch.from_numpy(c["draft"]).cuda()
    nodes = torch.full((B,), live, dtype=torch.int32, device="cuda")
    sd.spec_adjust_logits(x, num_nodes=nodes, **args)
    some = rng.integers(0, B, 40)
    want = expected({k: (v if k != "x" else v)[some] for k, v in c.items() if k == "x" or k in keep}, keep)
    same(x[torch.from_numpy(some).cuda(), :live], want)
    assert not bool(x[:, live:].any())


@pytest.mark.gpu
def test_two_threads_of_different_sizes(gpu):
    """Launches that need much and little shared memory beyond the default, from two threads at once."""
    import threading

    B, V, failed = 1000, 64, []

    def work(N):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                x = torch.ones((B, N, V), device="cuda")
                draft = torch.zeros((B, N), dtype=torch.int32, device="cuda")
                ids = torch.full((B, 1), 5, dtype=torch.int32, device="cuda")
                vals, one = torch.ones((B, 1), device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
                for _ in range(300):
                    sd.spec_adjust_logits(x, draft_token=draft, bias_ids=ids, bias_vals=vals, num_nodes=one)
                torch.cuda.current_stream().synchronize()
                assert bool((x[:, 0, 5] == 301).all()) and bool((x[:, 1:] == 1).all())
        except Exception as e:  # noqa: BLE001
            failed.append((N, e))

    threads = [threading.Thread(target=work, args=(N,)) for N in (513, 1400)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
