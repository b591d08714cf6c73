"""The paged 4-bit cache on the GPU against the oracle: rows written and read
back bit for bit, attention over it within derived bounds, eviction exact."""
import numpy as np
import pytest
import torch

from oracle import text_oracle as T
from tests import text_util as U
from tests.gpu_util import guarded_copy, to_np
from vision_language_model_b200 import vlm

pytestmark = pytest.mark.gpu
PAGE, K_SG, V_SG = U.PAGE, U.K_SG, U.V_SG


def _ok(status):
    assert vlm.status_sync(status) == vlm.OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,kv_heads,lens,new", [
    (128, 8, [0], [1]),
    (128, 2, [63, 64, 0, 130], [1, 1, 1, 1]),
    (64, 3, [0, 5, 64, 1], [67, 0, 130, 3]),
    (128, 1, [61], [9]),
    (64, 5, [0, 0], [1, 64]),
])
def test_append_and_read_are_exact(dtype, dim, kv_heads, lens, new):
    ends = [a + b for a, b in zip(lens, new)]
    pages, table, _ = U.random_pool(1, ends, kv_heads, dim)
    n = sum(new)
    gain = torch.tensor([0.01, 1.0, 4.0, 30.0])[torch.arange(n * kv_heads * dim) // 16 % 4].reshape(n, kv_heads, dim)
    k = (U.rand16(2, (n, kv_heads, dim), torch.float32) * gain).to(dtype)
    v = (U.rand16(3, (n, kv_heads, dim), torch.float32) * gain.flip(0)).to(dtype)
    k[0, 0, :16] = 0  # a block of zeros
    k[0, 0, 16:32] = torch.finfo(dtype).max if dtype == torch.float16 else 3e4  # and one that saturates
    ref = pages.copy()
    at = 0
    for s, m in enumerate(new):
        T.write(ref, table, s, lens[s], k[at:at + m].float().numpy(), v[at:at + m].float().numpy(), K_SG, V_SG)
        at += m
    gp, gt, gl = guarded_copy(torch.from_numpy(pages)), U.cuda_int(table), U.cuda_int(lens)
    # rows that come as column blocks of one buffer
    kv = guarded_copy(torch.cat([k, v], 1))
    cu = U.cuda_int(np.concatenate([[0], np.cumsum(new)]))
    status = vlm.new_status()
    vlm.kv4_append(gp, gt, gl, kv[:, :kv_heads], kv[:, kv_heads:], K_SG, V_SG, cu_new=cu, status=status)
    _ok(status)
    got = gp.cpu().numpy()
    # a value of -0 may keep its sign: codes compared as values, scales as bytes, everything else untouched
    sign_only = (got ^ ref) & np.where(np.arange(got.shape[2]) < PAGE * dim, 0x88, 0).astype(np.uint8)
    assert np.array_equal(got ^ sign_only, ref)
    for nib in (0, 4):
        assert np.all((((got ^ ref) >> nib) & 8 == 0) | (((got >> nib) & 7) == 0) | (np.arange(got.shape[2]) >= PAGE * dim))
    rk, rv = vlm.kv4_read(gp, gt, K_SG, V_SG, cu, n, start=gl, dtype=dtype, status=status)
    _ok(status)
    at = 0
    for s, m in enumerate(new):
        for h in range(kv_heads):
            ek, ev = T.read(ref, table, s, h, ends[s], dim)
            for g, e, sg in ((rk, ek, K_SG), (rv, ev, V_SG)):
                want = torch.from_numpy(e[lens[s]:].astype(np.float32) * np.float32(sg)).to(dtype)
                assert torch.equal(g[at:at + m, h].cpu(), want)
        at += m


def test_append_one_row_each_without_offsets():
    lens = [0, 63, 64, 200]
    pages, table, _ = U.random_pool(4, [n + 1 for n in lens], 4, 128)
    k, v = U.rand16(5, (4, 4, 128), torch.bfloat16), U.rand16(6, (4, 4, 128), torch.bfloat16)
    gp, gt, gl = (guarded_copy(torch.from_numpy(pages)) for _ in range(2)), U.cuda_int(table), U.cuda_int(lens)
    a, b = gp
    vlm.kv4_append(a, gt, gl, k.cuda(), v.cuda(), K_SG, V_SG)
    vlm.kv4_append(b, gt, gl, k.cuda(), v.cuda(), K_SG, V_SG, cu_new=U.cuda_int([0, 1, 2, 3, 4]))
    assert torch.equal(a, b)
    ka, va = vlm.kv4_read(a, gt, K_SG, V_SG, None, 4, start=gl)
    kb, vb = vlm.kv4_read(a, gt, K_SG, V_SG, U.cuda_int([0, 1, 2, 3, 4]), 4, start=gl)
    assert torch.equal(ka, kb) and torch.equal(va, vb)


def test_append_infinities_saturate_and_nan_is_bounded():
    pages, table, _ = U.random_pool(7, [2], 1, 64)
    k = U.rand16(8, (2, 1, 64), torch.bfloat16)
    k[0, 0, 3], k[0, 0, 20], k[1, 0, 40] = float("inf"), float("-inf"), float("nan")
    gp, gt = guarded_copy(torch.from_numpy(pages)), U.cuda_int(table)
    cu = U.cuda_int([0, 2])
    vlm.kv4_append(gp, gt, None, k.cuda(), k.cuda(), K_SG, V_SG, cu_new=cu)
    rk, rv = vlm.kv4_read(gp, gt, K_SG, V_SG, cu, 2)
    assert torch.isfinite(rk).all() and torch.isfinite(rv).all()
    assert float(rk[0, 0, 3]) == pytest.approx(448 * 6 * K_SG, rel=2 ** -8)
    assert float(rk[0, 0, 20]) == pytest.approx(-448 * 6 * K_SG, rel=2 ** -8)


def _attend(lens, heads, kv_heads, dim, q_len, dtype, seed=11, weights=False, gain=1.0):
    """By clusters where the batch is small, and by runs of pages, which a table of more than 128 pages asks for."""
    _attend_width(lens, heads, kv_heads, dim, q_len, dtype, seed, weights, gain, None)
    _attend_width(lens, heads, kv_heads, dim, q_len, dtype, seed, weights, gain, max(130, -(-max(lens) // PAGE)))


def _attend_width(lens, heads, kv_heads, dim, q_len, dtype, seed, weights, gain, width):
    pages, table, _ = U.random_pool(seed, lens, kv_heads, dim, width=width)
    q = U.rand16(seed + 1, (len(lens) * q_len, heads, dim), dtype, gain)
    scale = dim ** -0.5
    o, a, w = T.cache_attention(pages, table, lens, q.float().numpy(), q_len, K_SG, V_SG, scale)
    gp, gt, gl = guarded_copy(torch.from_numpy(pages)), U.cuda_int(table), U.cuda_int(lens)
    gw = None
    if weights:
        before = torch.rand((len(lens), kv_heads, table.shape[1] * PAGE), generator=torch.Generator().manual_seed(seed))
        gw = guarded_copy(before)
    status = vlm.new_status()
    got = vlm.kv4_attention(gp, gt, gl, guarded_copy(q), K_SG, V_SG, weights=gw, status=status)
    _ok(status)
    k = np.full((1, dim), 6.0 * 120.0)
    ds = U.logit_error(q.float().numpy(), k, scale, float(np.float32(K_SG)))
    tol = U.cache_tolerance(dtype, o, a, ds, max(lens + [1]), 6 * 120 * V_SG)
    U.assert_close(got, o, tol, "output")
    if weights:
        rows = heads // kv_heads * q_len
        e = 2 * (2.0 ** -21 + np.expm1(2 * ds))
        U.assert_close(gw, before.double().numpy() + w, e * w + (rows + 4) * 2.0 ** -24 * (w + 1) + 1e-30, "weights")
        for s, n in enumerate(lens):
            assert torch.equal(gw[s, :, n:].cpu(), before[s, :, n:])
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,heads,kv_heads,dim,q_len", [
    ([1], 4, 1, 128, 1),
    ([0], 8, 2, 64, 1),
    ([15, 16, 17, 63, 64, 65, 0, 128, 129, 255], 8, 2, 128, 1),
    ([700, 3, 0, 1999], 32, 8, 128, 1),
    ([2, 1, 0, 64, 66, 300], 12, 2, 64, 4),
    ([513], 5, 5, 64, 8),
    ([260, 31], 28, 4, 128, 5),
    ([130, 64], 40, 1, 128, 3),
    ([4000], 2, 1, 128, 1),
    ([8192, 1], 16, 1, 64, 1),   # as many pages as a small batch may have
    ([100] * 9, 8, 4, 64, 1),
    ([100] * 10, 8, 4, 64, 1),
    ([100] * 55, 2, 1, 64, 1),   # as many units as clusters take on a GPU of 148 SMs
    ([100] * 56, 2, 1, 64, 1),   # and one more
    ([1] * 300 + [2000], 4, 2, 64, 1),   # runs of many units' starts
    ([20000, 40, 0, 1], 8, 8, 64, 1),    # runs that end where a unit starts, before its first page
])
def test_attention_over_the_cache(lens, heads, kv_heads, dim, q_len, dtype):
    _attend(lens, heads, kv_heads, dim, q_len, dtype, weights=False)


@pytest.mark.parametrize("lens,heads,kv_heads,dim,q_len,dtype", [
    ([1], 4, 1, 128, 1, torch.bfloat16),
    ([70, 0, 2, 640], 32, 8, 128, 1, torch.bfloat16),
    ([2, 1, 0, 64, 66, 300], 16, 4, 64, 4, torch.float16),
    ([1500], 20, 2, 128, 5, torch.float16),
])
def test_attention_sums_each_places_weight(lens, heads, kv_heads, dim, q_len, dtype):
    _attend(lens, heads, kv_heads, dim, q_len, dtype, weights=True)


@pytest.mark.parametrize("lens,heads,kv_heads,dim,q_len,dtype", [
    ([8192, 4100, 1], 16, 1, 128, 1, torch.bfloat16),   # four pages per warp, a ring of two
    ([2049, 0, 5, 6000], 16, 4, 128, 4, torch.float16),  # two tiles of rows side by side
    ([8192, 2047], 4, 1, 64, 3, torch.float16),
    ([3000, 700], 40, 1, 128, 3, torch.bfloat16),       # several row tiles: weights in a launch of their own
    ([2100] + [65] * 26, 8, 4, 64, 1, torch.bfloat16),  # 108 units: two waves of clusters
    ([2100] + [65] * 27, 8, 4, 64, 1, torch.bfloat16),  # 112: by runs
])
def test_weights_from_the_cluster_that_attends(lens, heads, kv_heads, dim, q_len, dtype):
    _attend(lens, heads, kv_heads, dim, q_len, dtype, weights=True)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gain", [2.0 ** -60, 6.0, 2.0 ** 40])
def test_attention_over_the_cache_at_extreme_queries(gain, dim):
    # 2^-60: every weight equal; 6: a few places have all the weight; 2^40: one has, whatever the ties
    lens, heads = [333], 4
    if gain < 2 ** 30:
        _attend(lens, heads, 2, dim, 1, torch.bfloat16, gain=gain)
        return
    pages, table, _ = U.random_pool(3, lens, 2, dim)
    q = U.rand16(4, (1, heads, dim), torch.bfloat16, gain)
    o, _, _ = T.cache_attention(pages, table, lens, q.float().numpy(), 1, K_SG, V_SG, dim ** -0.5)
    got = vlm.kv4_attention(guarded_copy(torch.from_numpy(pages)), U.cuda_int(table), U.cuda_int(lens), q.cuda(), K_SG,
                            V_SG)
    U.assert_close(got, o, 2.0 ** -8 * np.abs(o) + 1e-30)


@pytest.mark.parametrize("dim,kv_heads,lens,budget,sinks,recent", [
    (128, 2, [1], 1, 0, 0),
    (128, 2, [300, 64, 65, 0, 1], 64, 4, 16),
    (64, 3, [500, 129], 100, 0, 0),
    (64, 1, [200], 37, 20, 17),     # nothing to choose
    (128, 4, [5000], 1000, 1, 300),
    (128, 1, [4097, 8193], 4096, 0, 1),
])
@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
def test_eviction_is_exact(dim, kv_heads, lens, budget, sinks, recent, kind):
    n, out_pages = len(lens), -(-budget // PAGE) + 1
    pages, table, left = U.random_pool(21, lens, kv_heads, dim, spare=n * out_pages)
    rng = np.random.default_rng(5)
    w = rng.random((n, kv_heads, table.shape[1] * PAGE)).astype(np.float32)
    if kind == "ties":
        w = (w * 3).astype(np.int32).astype(np.float32)
    if kind == "odd":
        w = ((w - 0.5) * 8).round().astype(np.float32)
        w[..., ::7], w[..., 3::11], w[..., 5::13] = -0.0, np.inf, np.nan
        w[..., 6::17] = -np.inf
    to = left[:n * out_pages].reshape(n, out_pages)
    gp = guarded_copy(torch.from_numpy(pages))
    status = vlm.new_status()
    new, kept, gw = vlm.kv4_evict(gp, U.cuda_int(table), U.cuda_int(lens), guarded_copy(torch.from_numpy(w)),
                                  U.cuda_int(to), budget, sinks=sinks, recent=recent, status=status)
    _ok(status)
    assert new.cpu().tolist() == [min(x, budget) for x in lens]
    ref = pages.copy()
    want_w = np.zeros((n, kv_heads, out_pages * PAGE), np.float32)
    want_kept = np.full((n, kv_heads, budget), -1, np.int32)
    for s, m in enumerate(lens):
        for h in range(kv_heads):
            ids = T.keep(w[s, h], m, budget, sinks, recent)
            want_kept[s, h, :len(ids)] = ids
            want_w[s, h, :len(ids)] = w[s, h, ids]
            for at, j in enumerate(ids):
                src, dst = pages[table[s, j // PAGE], h], ref[to[s, at // PAGE], h]
                for off, _, width in T._parts(dim):
                    a, b = off + (at % PAGE) * width, off + (j % PAGE) * width
                    dst[a:a + width] = src[b:b + width]
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(gw.cpu().numpy().view(np.int32), want_w.view(np.int32))
    assert np.array_equal(gp.cpu().numpy(), ref)


@pytest.mark.parametrize("wrong", ["source", "twice", "outside", "source_entry"])
def test_eviction_writes_no_page_unless_its_pages_are_fresh(wrong):
    lens, budget = [300, 200], 128
    pages, table, left = U.random_pool(22, lens, 2, 128, spare=4)
    to = left[:4].reshape(2, 2).copy()
    if wrong == "source":
        to[1, 1] = table[0, 4]
    elif wrong == "twice":
        to[1, 1] = to[0, 0]
    elif wrong == "outside":
        to[0, 1] = pages.shape[0]
    else:
        table[1, 0] = -1
    gp = guarded_copy(torch.from_numpy(pages))
    w = torch.rand((2, 2, table.shape[1] * PAGE)).cuda()
    status = vlm.new_status()
    vlm.kv4_evict(gp, U.cuda_int(table), U.cuda_int(lens), w, U.cuda_int(to), budget, status=status)
    assert vlm.status_sync(status) == vlm.ERR_BAD_PAGE
    assert np.array_equal(gp.cpu().numpy(), pages)


def test_shared_source_pages_are_no_clash():
    pages, table, left = U.random_pool(23, [256, 256], 1, 64, spare=4)
    table[1, :2] = table[0, :2]
    to = left[:4].reshape(2, 2)
    status = vlm.new_status()
    w = torch.rand((2, 1, 256)).cuda()
    vlm.kv4_evict(guarded_copy(torch.from_numpy(pages)), U.cuda_int(table), U.cuda_int([256, 256]), w, U.cuda_int(to),
                  128, status=status)
    _ok(status)


def test_pages_and_lengths_outside_the_cache_are_reported_and_touch_nothing():
    lens = [100, 70]
    pages, table, _ = U.random_pool(24, lens, 2, 64)
    q = U.rand16(1, (2, 4, 64), torch.bfloat16).cuda()
    gp = guarded_copy(torch.from_numpy(pages))
    bad = table.copy()
    bad[0, 1] = pages.shape[0] + 5
    good = vlm.kv4_attention(gp, U.cuda_int(table), U.cuda_int(lens), q, K_SG, V_SG)
    for t, n in ((bad, lens), (table, [100, 129]), (table, [-1, 70])):
        status = vlm.new_status()
        got = vlm.kv4_attention(gp, U.cuda_int(t), U.cuda_int(n), q, K_SG, V_SG, status=status)
        assert vlm.status_sync(status) == vlm.ERR_BAD_PAGE
        other = 0 if n[1] == 129 else 1
        assert torch.equal(got[other], good[other])
    k = U.rand16(2, (3, 2, 64), torch.bfloat16).cuda()
    for t, n, cu in ((bad, [64, 64], [0, 1, 3]), (table, [127, 64], [0, 2, 3]), (table, [0, -2], [0, 1, 3]),
                     (table, [0, 0], [0, 1, 2])):
        before = gp.clone()
        status = vlm.new_status()
        vlm.kv4_append(gp, U.cuda_int(t), U.cuda_int(n), k, k, K_SG, V_SG, cu_new=U.cuda_int(cu), status=status)
        assert vlm.status_sync(status) == vlm.ERR_BAD_PAGE
        gp.copy_(before)
        status = vlm.new_status()
        vlm.kv4_read(gp, U.cuda_int(t), K_SG, V_SG, U.cuda_int(cu), 3, start=U.cuda_int(n), status=status)
        assert vlm.status_sync(status) == vlm.ERR_BAD_PAGE
    assert torch.equal(gp.cpu(), torch.from_numpy(pages))


@pytest.mark.parametrize("n_pages", [300, 262144, 262145])
def test_eviction_checks_pages_of_small_and_large_pools(n_pages):
    # the check's bit sets lie in shared memory up to 262,144 pages, in the workspace above
    lens, budget = [200, 130], 64
    pages = torch.zeros((n_pages, 1, T.page_bytes(64)), dtype=torch.uint8, device="cuda")
    table = np.array([[0, n_pages - 1, 5, 7], [3, 4, 6, -1]], np.int32)
    pages[torch.from_numpy(table.reshape(-1)[:7]).long().cuda()] = torch.randint(
        0, 100, (7, 1, T.page_bytes(64)), dtype=torch.uint8, device="cuda")
    w = torch.rand((2, 1, 256)).cuda()
    for to, rc in (([[n_pages - 2], [8]], vlm.OK), ([[8], [n_pages - 1]], vlm.ERR_BAD_PAGE),
                   ([[n_pages - 2], [n_pages - 2]], vlm.ERR_BAD_PAGE), ([[n_pages], [8]], vlm.ERR_BAD_PAGE)):
        pool = pages.clone()
        status = vlm.new_status()
        new, kept, _ = vlm.kv4_evict(pool, U.cuda_int(table), U.cuda_int(lens), w, U.cuda_int(to), budget, recent=10,
                                     status=status)
        assert vlm.status_sync(status) == rc
        if rc != vlm.OK:
            assert torch.equal(pool, pages)
            continue
        for s in range(2):
            ids = T.keep(w[s, 0].cpu().numpy(), lens[s], budget, 0, 10)
            assert np.array_equal(kept[s, 0].cpu().numpy(), ids)
            src = np.stack([pages[table[s, j // 64], 0, (j % 64) * 32:(j % 64 + 1) * 32].cpu().numpy() for j in ids])
            assert np.array_equal(pool[to[s][0], 0, :2048].cpu().numpy().reshape(64, 32), src)


def test_eviction_of_a_long_context():
    # more places than a thread keeps in registers, and every 16-bit half of the counts in use
    n, budget = 70_001, 33_000
    pages, table, left = U.random_pool(31, [n], 1, 64, spare=-(-budget // PAGE))
    rng = np.random.default_rng(6)
    w = np.float32(rng.random((1, 1, table.shape[1] * PAGE)) ** 8)
    w[w < 1e-4] = 0
    status = vlm.new_status()
    new, kept, gw = vlm.kv4_evict(guarded_copy(torch.from_numpy(pages)), U.cuda_int(table), U.cuda_int([n]),
                                  guarded_copy(torch.from_numpy(w)), U.cuda_int(left[None, :-(-budget // PAGE)]), budget,
                                  sinks=3, recent=500, status=status)
    _ok(status)
    ids = T.keep(w[0, 0], n, budget, 3, 500)
    assert np.array_equal(kept[0, 0].cpu().numpy(), ids)
    assert np.array_equal(gw[0, 0, :budget].cpu().numpy(), w[0, 0, ids])
