"""Inputs and error bounds shared by the tests of the text side's attention."""
import numpy as np
import torch

from oracle import text_oracle as T
from tests.gpu_util import guarded_copy, to_np

PAGE = T.PAGE
K_SG, V_SG = 16.0 / 2688.0, 8.0 / 2688.0


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def rand16(seed, shape, dtype, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(dtype)


def random_pool(seed, lens, kv_heads, dim, spare=0, width=None):
    """(pages, table, spare page ids) on the host: random codes and scales 4 .. 120, pages in shuffled
    order, bytes behind a sequence's end anything at all (NaN scales among them), table entries behind
    its last page outside the pool."""
    rng = np.random.default_rng(seed)
    need = [-(-n // PAGE) for n in lens]
    width = max([1] + need) if width is None else width
    n_pages = sum(need) + spare + 2
    pages = rng.integers(0, 256, (n_pages, kv_heads, T.page_bytes(dim)), dtype=np.uint8)
    pages[..., PAGE * dim:] = pages[..., PAGE * dim:] % 40 + 0x48
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), width), -7, np.int32)
    at = 0
    for s, (n, m) in enumerate(zip(lens, need)):
        table[s, :m] = order[at:at + m]
        at += m
        if n % PAGE:
            last = pages[table[s, m - 1]]
            for p in (2, 3):
                off, _, w = T._parts(dim)[p]
                last[:, off + (n % PAGE) * w:off + PAGE * w] = 0x7F
    return pages, table, order[at:]


def cuda_int(v):
    return guarded_copy(torch.as_tensor(np.asarray(v, np.int32)).reshape(np.asarray(v).shape))


def logit_error(q, k, scale, mul=1.0):
    """Bound of an fp32 logit's error: products and sums of d terms, the tensor
    cores truncating each to 2^-23 of its size, q off by 2^-25 of its largest
    value, and the factors (scale, log2 e) rounded a few times."""
    q, k = np.abs(np.asarray(q, np.float64)), np.abs(np.asarray(k, np.float64)) * mul
    big = float((q.sum(-1)[..., None] * 0 + q.max(-1, keepdims=True)).max()) if q.size else 0.0
    norms = np.sqrt((q ** 2).sum(-1)).max() * np.sqrt((k ** 2).sum(-1)).max() if q.size and k.size else 0.0
    d = q.shape[-1]
    return scale * ((d + 8) * 2.0 ** -23 * norms + 2.0 ** -25 * big * (k.sum(-1).max() if k.size else 0.0))


def assert_close(got, ref, tol, what=""):
    g = to_np(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside the bound, worst {np.nanmax(np.abs(g - ref) - tol):.3e} over, first {np.argwhere(bad)[0]}"


def prompt_tolerance(dtype, o, a, ds):
    """P rounded (half a step of a), its exponentials (7.5e-5 of the polynomial, 2^-22 of the other) and
    logits, in the sum and in what it is divided by; the output rounded."""
    u = half_step(dtype)
    tiny = float(torch.finfo(dtype).smallest_normal) * u + 1e-30
    p_floor = 2.0 ** -24 if dtype == torch.float16 else 0.0  # weights below fp16's subnormal step
    return u * np.abs(o) + (u + 2 * (1e-4 + np.expm1(2 * ds))) * a * (1 + u) + tiny + p_floor


def cache_tolerance(dtype, o, a, ds, n, vmax):
    """P rounded to fp16 (half a step 2^-11; weights under 2^-14 by 2^-25), exponentials 2^-21."""
    u = half_step(dtype)
    return u * np.abs(o) + (2.0 ** -11 + 2 * (2.0 ** -21 + np.expm1(2 * ds))) * a * (1 + u) + 2.0 ** -25 * n * vmax + \
        float(torch.finfo(dtype).smallest_normal) * u
