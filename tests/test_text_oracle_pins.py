"""The text oracle pinned: attention against torch in fp64, the 4-bit pages
against torch's own E4M3 and the format's definition, the choice of places
against brute force."""
import itertools

import numpy as np
import pytest
import torch

from oracle import text_oracle as T
from oracle import vlm_oracle as O


@pytest.mark.parametrize("m,n", [(1, 1), (5, 5), (3, 9), (7, 4)])
def test_attention_against_torch(m, n):
    rng = np.random.default_rng(m * 10 + n)
    q, k, v = rng.normal(size=(m, 16)), rng.normal(size=(n, 16)), rng.normal(size=(n, 16))
    o, p, a = T.attend(q, k, v, 0.3, n - m)
    s = torch.from_numpy(q) @ torch.from_numpy(k).T * 0.3
    mask = torch.ones(m, n, dtype=torch.bool).tril(n - m)
    ref = torch.softmax(s.masked_fill(~mask, -torch.inf), -1).nan_to_num(0.0)
    np.testing.assert_allclose(p, ref.numpy(), rtol=0, atol=1e-14)
    np.testing.assert_allclose(o, (ref @ torch.from_numpy(v)).numpy(), rtol=0, atol=1e-13)
    np.testing.assert_allclose(a, (ref @ torch.from_numpy(v).abs()).numpy(), rtol=0, atol=1e-13)


def test_what_is_not_seen_does_not_count():
    rng = np.random.default_rng(1)
    q, k, v = (rng.normal(size=(6, 8)) for _ in range(3))
    o, _, _ = T.attend(q, k, v, 1.0, 0)
    k[4], v[4, 2], v[5] = np.nan, np.inf, np.nan
    o2, _, _ = T.attend(q, k, v, 1.0, 0)
    np.testing.assert_array_equal(o[:4], o2[:4])
    assert np.isnan(o2[4:]).all()


def test_grouped_heads_and_packing():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(7, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    o, _ = T.prompt_attention(q, k, v, [3, 4], [5, 4], 0.5)
    for h in range(4):
        np.testing.assert_array_equal(o[:3, h], T.attend(q[:3, h], k[:5, h // 2], v[:5, h // 2], 0.5, 2)[0])
        np.testing.assert_array_equal(o[3:, h], T.attend(q[3:, h], k[5:, h // 2], v[5:, h // 2], 0.5, 0)[0])


def test_e4m3_codes_against_torch():
    codes = np.arange(127, dtype=np.uint8)
    vals = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(T.e4m3_values(codes), vals)
    np.testing.assert_array_equal(T.e4m3_bytes(vals), codes)
    assert np.isnan(T.e4m3_values([127, 255])).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_pages_hold_what_the_recipe_says(dim):
    rng = np.random.default_rng(3)
    pages = rng.integers(0, 256, (4, 3, T.page_bytes(dim)), dtype=np.uint8)
    before = pages.copy()
    table = np.array([[2, 0]], np.int32)
    k, v = rng.normal(size=(70, 3, dim)), rng.normal(size=(70, 3, dim)) * 3
    T.write(pages, table, 0, 10, k, v, 0.01, 0.02)
    for h in range(3):
        gk, gv = T.read(pages, table, 0, h, 80, dim)
        for got, x, sg in ((gk, k, 0.01), (gv, v, 0.02)):
            q, sb = O.quantize_nvfp4(np.float32(x[:, h]), np.float32(sg))
            np.testing.assert_array_equal(got[10:], q * np.repeat(sb, 16, axis=1))
    np.testing.assert_array_equal(pages[[1, 3]], before[[1, 3]])  # other pages and rows as they were
    for off, _, w in T._parts(dim):
        np.testing.assert_array_equal(pages[2][:, off:off + 10 * w], before[2][:, off:off + 10 * w])
        np.testing.assert_array_equal(pages[0][:, off + 16 * w:off + 64 * w], before[0][:, off + 16 * w:off + 64 * w])


def test_weights_are_column_sums():
    rng = np.random.default_rng(4)
    pages = rng.integers(0, 256, (3, 1, T.page_bytes(64)), dtype=np.uint8)
    pages[..., 64 * 64:] = pages[..., 64 * 64:] % 40 + 0x48
    q = rng.normal(size=(2, 4, 64))
    o, a, w = T.cache_attention(pages, np.array([[1, 2]]), [100], q, 2, 0.01, 0.01, 0.125)
    assert w.shape == (1, 1, 128) and np.isclose(w.sum(), 8) and not w[0, 0, 100:].any()
    _, p, _ = T.attend(q[:, 0], T.read(pages, np.array([[1, 2]]), 0, 0, 100, 64)[0] * np.float64(np.float32(0.01)),
                       np.zeros((100, 64)), 0.125, 98)
    assert p[0, 99] == 0 and p[1, 99] > 0


def test_places_kept_by_brute_force():
    for w in itertools.product([0.0, 1.0, np.nan], repeat=5):
        w = np.array(w, np.float32)
        for budget, sinks, recent in [(2, 0, 0), (3, 1, 1), (4, 0, 2), (2, 1, 1)]:
            kept = T.keep(w, 5, budget, sinks, recent)
            mid = list(range(sinks, 5 - recent))
            mid.sort(key=lambda j: (np.isnan(w[j]), 0 if np.isnan(w[j]) else -w[j], j))
            want = sorted([*range(sinks), *mid[:budget - sinks - recent], *range(5 - recent, 5)])
            assert kept.tolist() == want
    assert T.keep(np.zeros(9), 4, 4, 0, 0).tolist() == [0, 1, 2, 3]
    assert T.keep(np.array([-0.0, 0.0, -0.0]), 3, 2, 0, 0).tolist() == [0, 1]
