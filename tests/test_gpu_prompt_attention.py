"""Causal prompt attention on the GPU against the fp64 oracle, element by
element within a bound derived from its roundings."""
import numpy as np
import pytest
import torch

from oracle import text_oracle as T
from tests import text_util as U
from tests.gpu_util import guarded, guarded_copy, to_np
from vision_language_model_b200 import vlm

pytestmark = pytest.mark.gpu


def _run(q_lens, kv_lens, heads, kv_heads, dim, dtype, gain=1.0, seed=1, scale=None):
    q = U.rand16(seed, (sum(q_lens), heads, dim), dtype, gain)
    k = U.rand16(seed + 1, (sum(kv_lens), kv_heads, dim), dtype)
    v = U.rand16(seed + 2, (sum(kv_lens), kv_heads, dim), dtype)
    status = vlm.new_status()
    got = vlm.prompt_attention(guarded_copy(q), guarded_copy(k), guarded_copy(v), q_lens, kv_lens, scale=scale,
                               status=status)
    assert vlm.status_sync(status) == vlm.OK
    s = dim ** -0.5 if scale is None else scale
    o, a = T.prompt_attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), q_lens, kv_lens, s)
    ds = U.logit_error(q.float().numpy(), k.float().numpy(), s)
    U.assert_close(got, o, U.prompt_tolerance(dtype, o, a, ds))
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads", [
    ([1], [1], 1, 1),
    ([37], [37], 4, 1),
    ([128], [128], 1, 1),
    ([129, 1, 255], [129, 1, 255], 2, 1),
    ([300], [300], 8, 2),
    ([5, 64, 1, 200], [133, 64, 700, 201], 6, 2),
    ([33], [1000], 5, 5),
    ([40], [40], 16, 1),
    ([1, 2, 3, 0, 4], [1, 0, 3, 5, 2], 4, 2),   # an empty sequence, no keys, fewer keys than queries
    ([700], [350], 2, 1),
    ([9], [300], 56, 1),
    ([3], [129], 128, 1),
])
def test_prompt_attention(q_lens, kv_lens, heads, kv_heads, dim, dtype):
    _run(q_lens, kv_lens, heads, kv_heads, dim, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_attention_of_an_image_prompt(dtype):
    _run([1100], [1100], 8, 2, 128, dtype, gain=4.0, seed=5)


def test_prompt_attention_scale_and_many_sequences():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 9, 600)]  # more than one launch's table
    _run(lens, lens, 4, 2, 64, torch.bfloat16, scale=0.3)


@pytest.mark.parametrize("lens,heads,kv_heads,dim", [
    ([900] * 3 + [64] * 10, 32, 8, 64),          # 440 work items: the host chooses each one's CTA
    ([900] * 3 + [64] * 19, 32, 8, 64),          # 512
    ([900] * 3 + [64] * 20, 32, 8, 64),          # 520: dealt out in turn
    ([2500] + [1] * 150, 8, 2, 128),             # few large ones among many small ones
    ([1500, 3, 0, 701, 702], 16, 4, 128),
    ([10] * 18 + [5000], 8, 8, 64),              # the largest share is one item's
])
def test_prompt_attention_does_not_depend_on_the_order_of_work(lens, heads, kv_heads, dim):
    q = U.rand16(21, (sum(lens), heads, dim), torch.bfloat16).cuda()
    k, v = (U.rand16(s, (sum(lens), kv_heads, dim), torch.bfloat16).cuda() for s in (22, 23))
    out = torch.full_like(q, 7.0)
    status = vlm.new_status()
    vlm.prompt_attention(q, k, v, lens, out=out, status=status)
    assert vlm.status_sync(status) == vlm.OK
    at = 0
    for n in lens:
        rows = slice(at, at + n)
        if n:
            assert torch.equal(out[rows], vlm.prompt_attention(q[rows], k[rows], v[rows], [n]))
        at += n


def test_prompt_attention_of_column_blocks_into_a_strided_output():
    heads, kv_heads, dim, lens = 8, 2, 128, [77, 200]
    T_ = sum(lens)
    qkv = U.rand16(7, (T_, heads + 2 * kv_heads, dim), torch.bfloat16).cuda()
    q, k, v = qkv.split([heads, kv_heads, kv_heads], 1)
    buf = torch.full((T_ + 3, heads + 1, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:T_, :heads]
    vlm.prompt_attention(q, k, v, lens, out=out)
    ref = vlm.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), lens)
    assert torch.equal(out, ref)
    assert (buf[T_:] == 7).all() and (buf[:, heads:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
def test_what_a_row_does_not_see_does_not_reach_it(dim, dtype):
    heads, kv_heads, lens = 4, 2, [150, 90, 333]
    n = sum(lens)
    q, k, v = (U.rand16(s, (n, h, dim), dtype).cuda() for s, h in ((1, heads), (2, kv_heads), (3, kv_heads)))
    clean = vlm.prompt_attention(q, k, v, lens)
    # from place 100 of every sequence on: infinities and NaN in keys and values
    k2, v2 = k.clone(), v.clone()
    at = 0
    for m in lens:
        for j, bad in ((100, float("inf")), (101, float("nan")), (130, float("-inf")), (300, float("nan"))):
            if j < m:
                v2[at + j, :, (7 * j) % dim] = bad
                k2[at + j, :, 3] = bad
        at += m
    got = vlm.prompt_attention(q, k2, v2, lens)
    only_v = vlm.prompt_attention(q, k, v2, lens)
    at = 0
    for m in lens:
        top = min(100, m)
        assert torch.equal(got[at:at + top], clean[at:at + top])
        assert torch.equal(only_v[at:at + top], clean[at:at + top])
        if m > 100:
            col = 700 % dim
            assert (only_v[at + 100:at + m, :, col] == float("inf")).all() or m > 101
            assert not torch.isfinite(only_v[at + 101:at + m, :, 707 % dim].float()).any()
            assert torch.isfinite(only_v[at + 100, :, :].float()).sum() == heads * (dim - 1)
            other = [c for c in range(dim) if c not in {(7 * j) % dim for j in (100, 101, 130, 300)}]
            assert torch.equal(only_v[at:at + m][:, :, other], clean[at:at + m][:, :, other])
        at += m


def test_a_nan_logit_makes_its_row_nan():
    for bad in (float("nan"), float("inf")):
        q, k, v = (U.rand16(s, (300, h, 64), torch.bfloat16).cuda() for s, h in ((1, 2), (2, 1), (3, 1)))
        q[:, :, 0] = q[:, :, 0].abs() + 0.5
        k[77, :, 0] = bad
        got = vlm.prompt_attention(q, k, v, [300])
        assert torch.isfinite(got[:77].float()).all()
        assert torch.isnan(got[77:].float()).all()


def test_sequences_are_independent_and_results_repeat():
    heads, kv_heads, dim, lens = 8, 2, 128, [200, 1, 515, 77]
    n = sum(lens)
    q, k, v = (U.rand16(s, (n, h, dim), torch.bfloat16).cuda() for s, h in ((1, heads), (2, kv_heads), (3, kv_heads)))
    both = vlm.prompt_attention(q, k, v, lens)
    assert torch.equal(both, vlm.prompt_attention(q, k, v, lens))
    at = 0
    for m in lens:
        alone = vlm.prompt_attention(q[at:at + m], k[at:at + m], v[at:at + m], [m])
        assert torch.equal(both[at:at + m], alone)
        at += m


def test_more_work_items_than_one_launch_takes():
    # 128 heads on one key head: 2 tokens per item; only the last 64 queries see a key
    q_len, kv_len, heads, dim = 160_000, 64, 128, 64
    k, v = U.rand16(1, (kv_len, 1, dim), torch.bfloat16), U.rand16(2, (kv_len, 1, dim), torch.bfloat16)
    q = torch.randn((q_len, heads, dim), generator=torch.Generator("cuda").manual_seed(3), device="cuda",
                    dtype=torch.bfloat16)
    out = torch.full_like(q, 7.0)
    status = vlm.new_status()
    before = vlm.launch_count()
    vlm.prompt_attention(q, k.cuda(), v.cuda(), [q_len], [kv_len], out=out, status=status)
    assert vlm.launch_count() - before > 1
    assert vlm.status_sync(status) == vlm.OK
    assert not out[:q_len - kv_len].any()
    ql = q[q_len - kv_len:].float().cpu().numpy()
    o, a = T.prompt_attention(ql, k.float().numpy(), v.float().numpy(), [kv_len], [kv_len], dim ** -0.5)
    ds = U.logit_error(ql, k.float().numpy(), dim ** -0.5)
    U.assert_close(out[q_len - kv_len:], o, U.prompt_tolerance(torch.bfloat16, o, a, ds))


@pytest.mark.parametrize("dtype,gain", [(torch.bfloat16, 1e7), (torch.float16, 1e4)])
def test_logits_of_any_size(dtype, gain):
    # the largest logit of a row, up to 10^15, has all the weight
    heads, dim, n = 4, 128, 200
    q, k = U.rand16(1, (n, heads, dim), dtype, gain), U.rand16(2, (n, 2, dim), dtype, gain)
    v = U.rand16(3, (n, 2, dim), dtype)
    o, _ = T.prompt_attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), [n], [n], dim ** -0.5)
    got = vlm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), [n])
    U.assert_close(got, o, U.half_step(dtype) * np.abs(o) + 1e-6)


def test_a_sequence_does_not_depend_on_its_neighbours_values():
    # the row tiles of a short sequence are filled up with the next one's queries: those may be anything
    heads, kv_heads, dim = 4, 2, 128
    lens = [200, 130]
    q, k, v = (U.rand16(s, (330, h, dim), torch.bfloat16).cuda() for s, h in ((1, heads), (2, kv_heads), (3, kv_heads)))
    ref = vlm.prompt_attention(q, k, v, lens)
    for bad in (3e38, float("inf"), float("nan"), 1e30):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        q2[200:], k2[200:], v2[200:] = bad, bad, bad
        got = vlm.prompt_attention(q2, k2, v2, lens)
        assert torch.equal(got[:200], ref[:200])
