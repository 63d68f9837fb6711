"""The 4-bit KV cache: append and gather, bit for bit against a plain
statement of the format, and moved by the slot compaction as opaque rows."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_draft_select_gb300 as sd
from oracle import target as ref
from speculative_decoding_draft_select_gb300.build import build


def slot_table(rng, B, max_ctx, page):
    """req_to_token [B, max_ctx] over shuffled pages, and the slot count."""
    pages = -(-max_ctx // page)
    perm = rng.permutation(B * pages).reshape(B, pages)
    pos = np.arange(max_ctx)
    return np.ascontiguousarray(perm[:, pos // page] * page + pos % page, np.int32), B * pages * page


def values(rng, shape, dtype, edges=True):
    x = rng.normal(0, 2, shape).astype(np.float32)
    flat = x.reshape(-1, 32)
    flat[::5] += 7.0                      # groups far from zero
    if edges and flat.shape[0] > 8:
        flat[1] = 0.25                    # no spread: step 0
        flat[2] *= 1e-7                   # a step below fp16's smallest
        flat[3, 5], flat[3, 6] = 1e38, -1e38
        flat[4, 0], flat[4, 1], flat[4, 2] = np.nan, np.inf, -np.inf
        flat[6] = np.nan
        flat[7] = 57344.0 * np.linspace(-1, 1, 32)
    return torch.from_numpy(x).to(dtype)


# ------------------------------------------------------------------------ CPU

def test_format_by_hand():
    """One group 0, 1, .., 15, 0, ..: lo 0, step 1, the codes themselves."""
    x = (np.arange(64) % 16).astype(np.float32).reshape(1, 1, 64)
    row = ref.kv4_rows(x, x - 3)
    assert row.shape == (1, 80)
    # channels 0, 2, 4, 6 in the low half of the first word, 1, 3, 5, 7 in its high half
    assert row[0, :4].tolist() == [0x20, 0x64, 0x31, 0x75]
    assert np.array_equal(row[0, :32], row[0, 32:64])
    meta = row[0, 64:80].view(np.float16)
    assert meta.tolist() == [1.0, 0.0, 1.0, 0.0, 1.0, -3.0, 1.0, -3.0]
    k, v = ref.kv4_values(row, 1, 64)
    assert np.array_equal(k, x) and np.array_equal(v, x - 3)


def test_codes_are_finite_at_the_limit():
    rng = np.random.default_rng(0)
    x = values(rng, (9, 1, 64), torch.float32).numpy()
    k, v = ref.kv4_values(ref.kv4_rows(x, x), 1, 64)
    assert np.isfinite(k.astype(np.float16)).all()


def test_quantisation_error_bound():
    """Off by half a step, plus fp16's roundings of lo and of 15 steps."""
    rng = np.random.default_rng(1)
    x = rng.normal(1, 2, (50, 2, 128)).astype(np.float32)
    k, _ = ref.kv4_values(ref.kv4_rows(x, x), 2, 128)
    g = x.reshape(50, 2, 4, 32)
    spread = (g.max(-1) - g.min(-1))[..., None]
    bound = spread / 30 * (1 + 1e-3) + np.abs(g.min(-1))[..., None] * 2.0**-11 + spread * 2.0**-11 + 1e-6
    assert (np.abs(k.reshape(g.shape) - g) <= bound).all()


def test_host_checks():
    build()
    lib, null = sd.lib(), None
    assert sd.spec_kv4_slot_bytes(8, 128) == 8 * 160 and sd.spec_kv4_slot_bytes(1, 64) == 80
    for H, D in ((0, 128), (257, 128), (8, 96), (8, 0)):
        with pytest.raises(sd.SpecError):
            sd.spec_kv4_slot_bytes(H, D)

    def app(B=1, N=1, H=1, D=64, dtype=1, k=null, ks=64, v=null, vs=64, ctx=8, pool=null, slots=8, stride=80):
        return lib.spec_kv4_append(B, N, H, D, dtype, k, ks, v, vs, null, k, k, ctx, pool, slots, stride, null, null)

    def gat(B=1, N=1, H=1, D=64, dtype=1, ctx=8, slots=8, stride=80):
        return lib.spec_kv4_gather(B, N, H, D, dtype, null, slots, stride, null, null, null, ctx, null, null, null, null)
    for f in (app, gat):
        assert f(B=-1) == -1 and f(N=-1) == -1 and f(H=0) == -1 and f(ctx=0) == -1 and f(slots=0) == -1
        assert f(stride=64) == -1 and f(stride=88) == -2 and f(D=80) == -2 and f(dtype=9) == -2 and f(H=300, stride=10**6) == -2
        assert f(B=0) == 0 and f(N=0) == 0 and f(N=2**31 - 1, B=4) == -2 and f() == -1
    assert app(ks=63) == -1 and app(vs=0) == -1
    if not torch.cuda.is_available():  # made-up addresses: only where nothing could run
        p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4104)
        assert app(k=odd, v=p, pool=p) == -2 and app(k=p, v=odd, pool=p) == -2 and app(k=p, v=p, pool=odd) == -2
        assert app(k=p, v=p, pool=p, ks=68) == -2
        assert lib.spec_kv4_gather(1, 1, 1, 64, 1, p, 8, 80, null, p, p, 8, odd, p, null, null) == -2


def test_binding_refuses_host_tensors():
    t = torch.zeros((1, 1, 1, 64))
    i = torch.zeros((1, 8), dtype=torch.int32)
    pool = torch.zeros((8, 80), dtype=torch.uint8)
    with pytest.raises(ValueError):
        sd.spec_kv4_append(t, t, pool, i, i[0, :1])
    with pytest.raises(ValueError):
        sd.spec_kv4_gather(pool, i, i[0, :1], 1, 1, 64)


# ------------------------------------------------------------------------ GPU

@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    return sd.lib()


def f32(t):
    return t.float().cpu().numpy()


SHAPES = [(1, 1, 1, 64, 1), (3, 1, 8, 128, 16), (2, 5, 3, 64, 5), (4, 17, 2, 128, 1), (1, 333, 1, 128, 16),
          (2, 2, 256, 64, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,H,D,page", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_and_gather(gpu, B, N, H, D, page, dtype):
    rng = np.random.default_rng(B * 100 + N + D)
    lens = rng.integers(0, 20, B).astype(np.int32)
    table, slots = slot_table(rng, B, 24 + N, page)
    k, v = values(rng, (B, N, H, D), dtype), values(rng, (B, N, H, D), dtype)
    before = torch.from_numpy(rng.integers(0, 256, (slots, sd.spec_kv4_slot_bytes(H, D))).astype(np.uint8))
    pool, tab, ln = before.cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda()
    stats = sd.new_stats()
    sd.spec_kv4_append(k.cuda(), v.cuda(), pool, tab, ln, stats=stats)
    want = before.numpy().copy()
    at = np.stack([table[b, lens[b]:lens[b] + N] for b in range(B)])
    want[at.reshape(-1)] = ref.kv4_rows(f32(k).reshape(-1, H, D), f32(v).reshape(-1, H, D))
    np.testing.assert_array_equal(pool.cpu().numpy(), want)  # other slots untouched
    gk, gv = sd.spec_kv4_gather(pool, tab, ln, N, H, D, dtype=dtype, stats=stats)
    wk, wv = ref.kv4_values(want[at.reshape(-1)], H, D)
    for got, w in ((gk, wk), (gv, wv)):
        # the values are sums of two fp16 numbers, rounded once (fp64 -> fp32
        # -> bf16 would round twice; code * step + lo has at most 11 + 4 + 15
        # bits only when lo and step are far apart, so fp32 may round)
        w32 = torch.from_numpy(w.astype(np.float32)).reshape(B, N, H, D).to(dtype)
        assert torch.equal(got.cpu(), w32)
    assert int(stats.sum()) == 0


@pytest.mark.gpu
def test_strided_parts_of_a_fused_projection_and_a_layer_of_a_wider_slot(gpu):
    rng = np.random.default_rng(7)
    B, N, H, D, layers, layer = 3, 4, 2, 64, 3, 1
    row = sd.spec_kv4_slot_bytes(H, D)
    lens = np.array([0, 3, 9], np.int32)
    table, slots = slot_table(rng, B, 16, 4)
    qkv = values(rng, (B, N, 6 + 2 * H, D), torch.bfloat16, edges=False).cuda()
    k, v = qkv[:, :, 6:6 + H], qkv[:, :, 6 + H:]
    wide = torch.from_numpy(rng.integers(0, 256, (slots, layers * row)).astype(np.uint8))
    pool, tab, ln = wide.cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda()
    part = pool[:, layer * row:(layer + 1) * row]
    sd.spec_kv4_append(k, v, part, tab, ln)
    want = wide.numpy().copy()
    at = np.concatenate([table[b, lens[b]:lens[b] + N] for b in range(B)])
    want[at, layer * row:(layer + 1) * row] = ref.kv4_rows(f32(k).reshape(-1, H, D), f32(v).reshape(-1, H, D))
    np.testing.assert_array_equal(pool.cpu().numpy(), want)
    gk, _ = sd.spec_kv4_gather(part, tab, ln, N, H, D, dtype=torch.float32)
    wk, _ = ref.kv4_values(want[at, layer * row:(layer + 1) * row], H, D)
    assert torch.equal(gk.cpu(), torch.from_numpy(wk.astype(np.float32)).reshape(B, N, H, D))
    with pytest.raises(ValueError):
        sd.spec_kv4_append(k.transpose(1, 2), v.transpose(1, 2), part, tab, ln)


@pytest.mark.gpu
def test_padded_batch_and_positions_out_of_range(gpu):
    rng = np.random.default_rng(8)
    B, N, H, D = 6, 3, 1, 64
    table, slots = slot_table(rng, B, 10, 1)
    table[4, 5], table[4, 6] = -1, slots  # request 4's first two tokens have no slot
    lens = np.array([0, 8, -1, 2, 5, 1], np.int32)       # 1: the last of its tokens is past the table
    nodes = np.array([3, 3, 2, 0, 3, -4], np.int32)
    k = values(rng, (B, N, H, D), torch.bfloat16, edges=False)
    before = rng.integers(0, 256, (slots, 80)).astype(np.uint8)
    pool = torch.from_numpy(before).cuda()
    tab, ln, nn = (torch.from_numpy(t).cuda() for t in (table, lens, nodes))
    stats = sd.new_stats()
    sd.spec_kv4_append(k.cuda(), k.cuda(), pool, tab, ln, num_nodes=nn, stats=stats)
    rows = ref.kv4_rows(f32(k).reshape(-1, H, D), f32(k).reshape(-1, H, D)).reshape(B, N, -1)
    want = before.copy()
    kept = [(0, 0), (0, 1), (0, 2), (1, 0), (1, 1), (4, 2)]
    for b, n in kept:
        want[table[b, lens[b] + n]] = rows[b, n]
    np.testing.assert_array_equal(pool.cpu().numpy(), want)
    assert int(stats[sd.STATS["bad_request"]]) == 1 + 2 + 2  # 1's last, 2's two, 4's two
    out = torch.full((B, N, H, D), 9.0, device="cuda")
    gk, gv = sd.spec_kv4_gather(pool, tab, ln, N, H, D, dtype=torch.float32, num_nodes=nn, k=out, v=out.clone(), stats=stats)
    assert int(stats[sd.STATS["bad_request"]]) == 10
    for b in range(B):
        for n in range(N):
            if n >= max(nodes[b], 0):
                assert (gk[b, n] == 9).all() and (gv[b, n] == 9).all()  # left as they were
            elif (b, n) in kept:
                w = ref.kv4_values(rows[b, n][None], H, D)[0][0].astype(np.float32)
                assert np.array_equal(gk[b, n].cpu().numpy(), w)
            else:
                assert (gk[b, n] == 0).all()


@pytest.mark.gpu
def test_slots_past_two_gigabytes(gpu):
    """Byte offsets of slots near the end of a pool of more than 4 GB."""
    H, D = 256, 128
    row = sd.spec_kv4_slot_bytes(H, D)
    slots = (5 << 30) // row
    pool = torch.zeros((slots, row), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[slots - 1, slots // 2]], dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(9)
    k = values(rng, (1, 2, H, D), torch.bfloat16)
    sd.spec_kv4_append(k.cuda(), k.cuda(), pool, table, lens)
    want = ref.kv4_rows(f32(k)[0], f32(k)[0])
    np.testing.assert_array_equal(pool[slots - 1].cpu().numpy(), want[0])
    np.testing.assert_array_equal(pool[slots // 2].cpu().numpy(), want[1])
    gk, _ = sd.spec_kv4_gather(pool, table, lens, 2, H, D, dtype=torch.float32)
    np.testing.assert_array_equal(gk.cpu().numpy().reshape(2, H, D), ref.kv4_values(want, H, D)[0].astype(np.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 4])
def test_compaction_moves_the_rows(gpu, page):
    """Nodes appended, the accepted path kept by spec_compact_slots, and the
    kept positions read back: the accepted nodes' rows, in path order."""
    rng = np.random.default_rng(page)
    B, N, H, D = 2, 7, 2, 64
    lens = np.array([5, 2], np.int32)
    table, slots = slot_table(rng, B, 16, page)
    k = values(rng, (B, N, H, D), torch.bfloat16, edges=False)
    pool = torch.zeros((slots, sd.spec_kv4_slot_bytes(H, D)), dtype=torch.uint8, device="cuda")
    tab, ln = torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda()
    sd.spec_kv4_append(k.cuda(), k.cuda(), pool, tab, ln)
    path = np.full((B, N), -1, np.int32)
    path[0, :4], path[1, :2] = [0, 2, 3, 6], [0, 5]
    acc = np.array([3, 1], np.int32)
    out = sd.spec_compact_slots(ln, torch.from_numpy(path).cuda(), torch.from_numpy(acc).cuda(), tab, page, kv_pool=pool)
    assert out["new_kv_len"].tolist() == [9, 4]
    gk, _ = sd.spec_kv4_gather(pool, tab, ln, N, H, D, dtype=torch.float32,
                               num_nodes=torch.from_numpy(acc + 1).cuda())
    rows = ref.kv4_rows(f32(k).reshape(-1, H, D), f32(k).reshape(-1, H, D)).reshape(B, N, -1)
    for b in range(B):
        for i in range(acc[b] + 1):
            w = ref.kv4_values(rows[b, path[b, i]][None], H, D)[0][0].astype(np.float32)
            assert np.array_equal(gk[b, i].cpu().numpy(), w), (b, i)


@pytest.mark.gpu
def test_captured(gpu):
    rng = np.random.default_rng(10)
    B, N, H, D = 2, 3, 2, 128
    table, slots = slot_table(rng, B, 64, 4)
    pool = torch.zeros((slots, sd.spec_kv4_slot_bytes(H, D)), dtype=torch.uint8, device="cuda")
    tab, ln = torch.from_numpy(table).cuda(), torch.zeros(B, dtype=torch.int32, device="cuda")
    k = values(rng, (B, N, H, D), torch.bfloat16, edges=False).cuda()
    gk = torch.empty((B, N, H, D), dtype=torch.float32, device="cuda")
    gv = torch.empty_like(gk)

    def step():
        sd.spec_kv4_append(k, k, pool, tab, ln)
        sd.spec_kv4_gather(pool, tab, ln, N, H, D, dtype=torch.float32, k=gk, v=gv)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for at in (7, 30):  # the captured step follows the lengths and the inputs
        ln.fill_(at)
        k.copy_(values(rng, (B, N, H, D), torch.bfloat16, edges=False))
        g.replay()
        torch.cuda.synchronize()
        rows = ref.kv4_rows(f32(k).reshape(-1, H, D), f32(k).reshape(-1, H, D))
        slot = np.concatenate([table[b, at:at + N] for b in range(B)])
        np.testing.assert_array_equal(pool.cpu().numpy()[slot], rows)
        np.testing.assert_array_equal(gk.cpu().numpy().reshape(-1, H, D), ref.kv4_values(rows, H, D)[0].astype(np.float32))
