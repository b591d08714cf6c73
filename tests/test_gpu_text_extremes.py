"""The text side's attention where numbers get extreme: large logits, many small weights, infinities."""
import numpy as np
import pytest
import torch

from oracle import text_oracle as T
from tests import text_util as U
from tests.gpu_util import guarded_copy
from vision_language_model_b200 import vlm

pytestmark = pytest.mark.gpu
PAGE, K_SG, V_SG = U.PAGE, U.K_SG, U.V_SG


def _steep(seed, lens, kv_heads, dim, width):
    """A pool whose keys differ in column 1 alone as far as the queries of _steep_q go: their products are
    24 and a little, sums of two terms with 20 bits between them, so fp32 holds every one exactly."""
    pages, table, _ = U.random_pool(seed, lens, kv_heads, dim, width=width)
    (at, n, w), scales = T._parts(dim)[0], T._parts(dim)[2]
    rows = pages[..., at:at + n].reshape(*pages.shape[:2], PAGE, w)
    rows[..., 0] = (rows[..., 0] & 0xF0) | 7  # column 0: 6
    pages[..., at:at + n] = rows.reshape(*pages.shape[:2], n)
    pages[..., scales[0]:scales[0] + scales[1]:scales[2]] = 0x48  # times 4
    return pages, table


@pytest.mark.parametrize("size", [4096.0, 2.0 ** 20, 2.0 ** 26])
@pytest.mark.parametrize("lens,heads,kv_heads,dim,q_len,dtype", [
    ([700, 65], 4, 2, 128, 1, torch.bfloat16),
    ([700, 65], 16, 2, 64, 2, torch.float16),
    ([400], 40, 1, 64, 1, torch.bfloat16),     # several row tiles: the weights in a launch of their own
    ([1300, 0, 3], 8, 4, 128, 3, torch.float16),
])
@pytest.mark.parametrize("width", [128, 140])  # by clusters, and by runs that a join puts together
def test_weights_and_outputs_of_large_logits(lens, heads, kv_heads, dim, q_len, dtype, size, width):
    # logits of `size` in log2 units that differ by 4096 -> 0.005, 2^20 -> 1.3, 2^26 -> 85 per step of a code
    pages, table = _steep(41, lens, kv_heads, dim, width)
    q = torch.zeros((len(lens) * q_len, heads, dim), dtype=dtype)
    q[..., 0], q[..., 1] = 4.0, 4.0 * 2.0 ** -16
    scale = float(np.float32(size * np.log(2.0) / (4.0 * 24.0 * K_SG)))
    o, a, w = T.cache_attention(pages, table, lens, q.float().numpy(), q_len, K_SG, V_SG, scale)
    status = vlm.new_status()
    gw = guarded_copy(torch.zeros((len(lens), kv_heads, width * PAGE)))
    got = vlm.kv4_attention(guarded_copy(torch.from_numpy(pages)), U.cuda_int(table), U.cuda_int(lens), guarded_copy(q),
                            K_SG, V_SG, scale=scale, weights=gw, status=status)
    assert vlm.status_sync(status) == vlm.OK
    # A difference of two products is exact; its factor takes four roundings (and the product one), so a weight of
    # 2^-60 or more is off by 60 * 5 * 2^-24 ln 2, by 2^-21 of the exponential, and as much again where a run's
    # sums are joined; its sum by 2^-24 per term.
    e = 2 * (60 * 5 * 2.0 ** -24 * np.log(2.0) + 2.0 ** -21) + (max(lens) + 8) * 2.0 ** -24
    rows = heads // kv_heads * q_len
    U.assert_close(gw, w, (2 * e + rows * 2.0 ** -24) * w + rows * 2.0 ** -60, "weights")
    u = U.half_step(dtype)
    U.assert_close(got, o, u * np.abs(o) + (2.0 ** -11 + 2 * e) * a * (1 + u) + 2.0 ** -32 * max(lens) * 720 * V_SG +
                   float(torch.finfo(dtype).smallest_normal) * u, "output")


@pytest.mark.parametrize("gap", [20.6, 25.5])
@pytest.mark.parametrize("dim,dtype", [(64, torch.bfloat16), (128, torch.float16)])
def test_many_small_weights_beside_a_large_one(dim, dtype, gap):
    # 131,072 places, the first with 2^gap times the others' weight and a value of 0, so the others are the whole
    # output. So many sequences (sharing two pages) that most are one warp's: it keeps the first place's maximum.
    S, kv_heads, n = 250, 8, 131072
    pages = np.random.default_rng(7).integers(0, 256, (2, kv_heads, T.page_bytes(dim)), dtype=np.uint8)
    pages[..., PAGE * dim:] = 0x48
    (ka, kn, kw), (va, vn, vw) = T._parts(dim)[:2]
    pages[..., ka:ka + kn] = 0
    pages[..., va:va + vn] &= 0x77  # values >= 0: nothing cancels
    pages[0, :, ka], pages[0, :, va:va + vw] = 7, 0
    table = np.ones((S, n // PAGE), np.int32)
    table[:, 0] = 0
    q = torch.zeros((S, kv_heads, dim), dtype=dtype)
    q[..., 0] = 1.0
    scale = float(np.float32(gap * np.log(2.0) / (24.0 * K_SG)))
    o, a, _ = T.cache_attention(pages, table[:1], [n], q[:1].float().numpy(), 1, K_SG, V_SG, scale)
    status = vlm.new_status()
    got = vlm.kv4_attention(guarded_copy(torch.from_numpy(pages)), U.cuda_int(table), U.cuda_int([n] * S), q.cuda(), K_SG,
                            V_SG, scale=scale, status=status)
    assert vlm.status_sync(status) == vlm.OK
    # P rounded to fp16 (half a step; weights under 2^-21 of the largest by 2^-32 of it), exponentials of exact
    # logits (the factor's and the product's roundings, the unit's 2^-21), fp32 sums of a lane's share of the places
    u = U.half_step(dtype)
    e = 2.0 ** -11 + 2 * (gap * 5 * 2.0 ** -24 + 2.0 ** -21) + 2 * (n // 4) * 2.0 ** -24
    tol = u * np.abs(o) + e * a * (1 + u) + 2.0 ** -32 * n * 24 * V_SG + float(torch.finfo(dtype).smallest_normal) * u
    U.assert_close(got, np.broadcast_to(o, got.shape), np.broadcast_to(tol, got.shape))


@pytest.mark.parametrize("gap", [20.6, 25.5])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_many_small_weights_beside_a_large_one_in_a_prompt(dtype, dim, gap):
    # 131,072 keys, the first with 2^gap times the others' weight and a value of 0: the others are the whole output
    n, m = 131072, 3
    q, k = torch.zeros((m, 2, dim), dtype=dtype), torch.zeros((n, 1, dim), dtype=dtype)
    q[..., 0], k[0, 0, 0] = 1.0, 8.0
    v = U.rand16(51, (n, 1, dim), dtype).abs()
    v[0] = 0
    scale = float(np.float32(gap * np.log(2.0) / 8.0))
    o, a = T.prompt_attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), [m], [n], scale)
    got = vlm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), [m], [n], scale=scale)
    # P rounded (half a step; fp16's weights under 2^-21 of the largest by 2^-32 of it), exponentials of exact logits
    # (scale log2 e, the maximum's and the difference's products rounded: 2^-24 of them each; the unit 2^-21), fp32
    # sums of 1,024 tiles of 64 keys in O and in the row's sum, the tensor core's truncated to 2^-23
    u = U.half_step(dtype)
    e = u + 2 * (gap * 4 * 2.0 ** -24 + 2.0 ** -21) + (1024 + 64) * 2.0 ** -24 + 1024 * 8 * 2.0 ** -23
    floor = 2.0 ** -32 * n * float(v.max()) if dtype == torch.float16 else 0.0
    U.assert_close(got, o, u * np.abs(o) + e * a * (1 + u) + floor + float(torch.finfo(dtype).smallest_normal) * u)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_row_whose_logits_are_all_minus_infinity_is_nan(dim, dtype):
    # the softmax of nothing but -inf is 0 / 0; only a query that sees no key at all gives 0
    heads, kv_heads, q_lens, kv_lens = 4, 2, [200, 9], [200, 5]
    q = U.rand16(61, (sum(q_lens), heads, dim), dtype)
    k, v = (U.rand16(s, (sum(kv_lens), kv_heads, dim), dtype) for s in (62, 63))
    q[..., 0] = q[..., 0].abs() + 0.5
    k[:50, :, 0] = float("-inf")
    scale = dim ** -0.5
    got = vlm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), q_lens, kv_lens)
    o, a = T.prompt_attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), q_lens, kv_lens, scale)
    assert np.isnan(o[:50]).all() and torch.isnan(got[:50].float()).all()
    ds = U.logit_error(q.float().numpy(), np.where(np.isfinite(k.float().numpy()), k.float().numpy(), 0.0), scale)
    U.assert_close(got[50:], o[50:], U.prompt_tolerance(dtype, o[50:], a[50:], ds))
    assert not got[200:204].any()


@pytest.mark.parametrize("width", [128, 140])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_cache_row_whose_logits_are_all_minus_infinity_is_nan(dim, width):
    lens, heads, kv_heads = [70, 0, 300], 4, 2
    pages, table, _ = U.random_pool(64, lens, kv_heads, dim, width=width)
    at, n, w = T._parts(dim)[0]
    pages[..., at:at + n:w] |= 0x0F  # column 0 of every key: -6
    q = U.rand16(65, (len(lens) * 2, heads, dim), torch.bfloat16)
    q[:, 1, 0] = float("inf")
    gw = torch.zeros((len(lens), kv_heads, width * PAGE), device="cuda")
    got = vlm.kv4_attention(guarded_copy(torch.from_numpy(pages)), U.cuda_int(table), U.cuda_int(lens), guarded_copy(q),
                            K_SG, V_SG, weights=gw).float().cpu()
    o, _, want = T.cache_attention(pages, table, lens, q.float().numpy(), 2, K_SG, V_SG, dim ** -0.5)
    assert np.array_equal(np.isnan(o), torch.isnan(got).numpy())
    assert torch.isnan(got[:2, 1]).all() and torch.isnan(got[4:, 1]).all() and not got[2:4].any()
    assert np.array_equal(np.isnan(want), torch.isnan(gw).cpu().numpy())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
def test_infinite_values_reach_the_rows_that_see_them(dim, dtype):
    heads, kv_heads, lens = 4, 2, [150, 90, 333]
    n = sum(lens)
    q, k, v = (U.rand16(s, (n, h, dim), dtype) for s, h in ((1, heads), (2, kv_heads), (3, kv_heads)))
    at = 0
    for m in lens:
        for j, col, bad in ((100, 60, float("inf")), (130, 14, float("-inf")), (101, 3, float("nan"))):
            if j < m:
                v[at + j, :, col] = bad
        at += m
    got = vlm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), lens).float().cpu()
    at = 0
    for m in lens:
        x = got[at:at + m]
        assert (x[100:, :, 60] == float("inf")).all() and torch.isfinite(x[:100]).all()
        assert (x[130:, :, 14] == float("-inf")).all() and torch.isfinite(x[:130, :, 14]).all()
        assert torch.isnan(x[101:, :, 3]).all() and torch.isfinite(x[:101, :, 3]).all()
        at += m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim", [
    ([300], [300], 8, 2, 128), ([300], [300], 8, 2, 64), ([70, 1, 129], [500, 130, 129], 6, 2, 64), ([257], [300], 3, 3, 128),
])
def test_a_prompt_with_exact_logits_is_off_by_its_roundings_alone(q_lens, kv_lens, heads, kv_heads, dim, dtype):
    # one column per query is not 0, so a logit is one product of two 16-bit values, exact in fp32
    T_ = sum(q_lens)
    g = torch.Generator().manual_seed(91)
    hot = torch.nn.functional.one_hot(torch.randint(0, dim, (T_, heads), generator=g), dim)
    q = (U.rand16(92, (T_, heads, dim), torch.float32) * 6.0 * hot).to(dtype)
    k, v = (U.rand16(s, (sum(kv_lens), kv_heads, dim), dtype) for s in (93, 94))
    scale = 0.5
    o, a = T.prompt_attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), q_lens, kv_lens, scale)
    got = vlm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), q_lens, kv_lens, scale=scale)
    # logits up to L in log2 units: the scale, the maximum's and the exponent's products round them by 2^-24 each; the
    # unit 2^-21; both in the weights and in their sum. The tensor core truncates each of the n terms of a sum to 2^-23.
    L = scale * 1.4427 * float(q.float().abs().max() * k.float().abs().max())
    n, u = max(kv_lens), U.half_step(dtype)
    e = u + 2 * (5 * L * 2.0 ** -24 + 2.0 ** -21) + n * (2.0 ** -23 + 2.0 ** -24)
    floor = 2.0 ** -32 * n * float(v.float().abs().max()) if dtype == torch.float16 else 0.0
    U.assert_close(got, o, u * np.abs(o) + e * a * (1 + u) + floor + float(torch.finfo(dtype).smallest_normal) * u)


@pytest.mark.parametrize("dim", [64, 128])
def test_scales_up_to_the_largest_fp32_value(dim):
    # the key whose product is largest has all the weight, however large the logits get
    heads, kv_heads, n = 4, 2, 150
    q, k, v = (U.rand16(s, (n, h, dim), torch.bfloat16) for s, h in ((95, heads), (96, kv_heads), (97, kv_heads)))
    o, _ = T.prompt_attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), [n], [n], 3e38)
    got = vlm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), [n], scale=3e38)
    U.assert_close(got, o, 2.0 ** -8 * np.abs(o) + 1e-30)
    lens = [150, 65]
    pages, table, _ = U.random_pool(98, lens, kv_heads, dim)
    cq = U.rand16(99, (2, heads, dim), torch.bfloat16, 2.0 ** 120)
    for k_sg, scale in ((K_SG, 3e38), (3e38, 1.0)):
        o, _, w = T.cache_attention(pages, table, lens, cq.float().numpy(), 1, k_sg, V_SG, scale)
        gw = torch.zeros((2, kv_heads, table.shape[1] * PAGE), device="cuda")
        got = vlm.kv4_attention(guarded_copy(torch.from_numpy(pages)), U.cuda_int(table), U.cuda_int(lens), cq.cuda(), k_sg,
                                V_SG, scale=scale, weights=gw)
        U.assert_close(got, o, 2.0 ** -8 * np.abs(o) + 1e-30)
        assert np.array_equal(gw.cpu().numpy(), w.astype(np.float32))
