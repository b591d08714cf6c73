"""Work items of the prompt attention that follow one another on a CTA: long ones, ones whose second row
tile has no token, ones without a key."""
import pytest
import torch

from tests import text_util as U
from vision_language_model_b200 import vlm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads", [
    # two live row tiles, then items of one key tile with an idle row tile, then items without a key
    ([250] * 30 + [100] * 40 + [60] * 20, [250] * 30 + [100] * 40 + [0] * 20, 8, 8),
    ([250] * 12 + [100] * 20 + [60] * 20, [250] * 12 + [100] * 20 + [0] * 20, 8, 8),  # few: the host chooses the CTAs
    ([63, 64, 40, 1] * 40, [63, 10, 0, 1] * 40, 32, 8),
    ([600] * 8 + [5] * 90, [600] * 8 + [0] * 90, 16, 8),
])
@pytest.mark.parametrize("dim", [64, 128])
def test_short_items_behind_long_ones_keep_their_rows_sums(q_lens, kv_lens, heads, kv_heads, dim):
    q = U.rand16(71, (sum(q_lens), heads, dim), torch.bfloat16).cuda()
    k, v = (U.rand16(s, (sum(kv_lens), kv_heads, dim), torch.bfloat16).cuda() for s in (72, 73))
    status = vlm.new_status()
    runs = [vlm.prompt_attention(q, k, v, q_lens, kv_lens, status=status) for _ in range(20)]
    assert vlm.status_sync(status) == vlm.OK
    for r in runs[1:]:
        assert torch.equal(r, runs[0])
    q0 = k0 = 0
    for m, n in zip(q_lens, kv_lens):
        rows, keys = slice(q0, q0 + m), slice(k0, k0 + n)
        assert torch.equal(runs[0][rows], vlm.prompt_attention(q[rows], k[keys], v[keys], [m], [n]))
        q0, k0 = q0 + m, k0 + n


@pytest.mark.parametrize("q_len,kv_len,heads,kv_heads", [
    (256, 256, 2, 2),    # 128 tokens per row tile: the first keys' tile is the first row tile's last, and whole to the second
    (128, 168, 8, 2),    # 32 tokens per row tile
    (168, 199, 6, 2),    # 42
])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_value_replaced_for_one_row_tile_is_replaced_for_both(q_len, kv_len, heads, kv_heads, dim, dtype):
    # The weights of key 5 round to 0: where its infinite value is replaced and noted the rows get infinity, where the
    # product reads it NaN. Both row tiles of an item have to do the same, whichever comes first.
    q = U.rand16(81, (q_len, heads, dim), dtype)
    k, v = (U.rand16(s, (kv_len, kv_heads, dim), dtype) for s in (82, 83))
    q[..., 0], k[..., 0], k[5, :, 0], v[5, :, 7] = 8.0, 0.0, -1000.0, float("inf")
    args = [x.cuda() for x in (q, k, v)]
    runs = [vlm.prompt_attention(*args, [q_len], [kv_len]) for _ in range(20)]
    for r in runs[1:]:
        assert torch.equal(r.view(torch.int16), runs[0].view(torch.int16))
    sees = max(0, 5 - (kv_len - q_len))  # the first query that sees key 5
    got = runs[0].float().cpu()
    assert torch.isfinite(got[:sees]).all()
    assert (got[sees:, :, 7] == float("inf")).all()
    assert torch.isfinite(got[:, :, [c for c in range(dim) if c != 7]]).all()
