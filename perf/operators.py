"""The text side's attention operators, measured: cases, inputs, plain forms, the library's calls and exact values.

Four operators that take the prompt (text rows and scattered image rows) through the language model's attention:
  prompt  causal attention of packed prompts with grouped heads (vlm.prompt_attention);
  append  keys and values of new tokens quantised into a paged 4-bit cache, and read back (vlm.kv4_append, vlm.kv4_read);
  cache   attention of a few new tokens over that cache, optionally summing every key's weight (vlm.kv4_attention);
  evict   the keys with the largest summed weights kept in fresh pages, the others dropped (vlm.kv4_evict, vlm.kv4_read).

The cache: pages of 64 tokens, uint8 [n_pages, kv_heads, page bytes]; a page of one head holds the E2M1 codes of its keys
[64, dim / 2] (the even column in the low nibble), those of its values, and the E4M3 scales [64, dim / 16] of its keys and of
its values. A value stands for code * scale * the tensor's fp32 global scale.
"""
import math

import torch

own = False

PAGE = 64
K_SG, V_SG = 16.0 / 2688.0, 8.0 / 2688.0  # static global scales: |k| to 16 and |v| to 8 before a scale saturates
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
HEADS = [(32, 8), (32, 8), (16, 4), (8, 8), (16, 1), (12, 2), (28, 4), (5, 5), (40, 8)]


# ----------------------------------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------------------------------

def _text(v):
    return ",".join(str(int(x)) for x in v)


def _ints(t):
    return [int(x) for x in t.split(",")]


def listed():
    d = dict(heads=32, kv_heads=8, dim=128)  # the text decoder beside the encoder: 32 query and 8 key heads of 128
    return [
        # a short question without an image: the call's latency
        dict(name="prompt_short", op="prompt", dtype="bf16", **d, q_lens="37", kv_lens="37"),
        # one 1540 x 1540 image (3,025 merged tokens) with its question, an odd length
        dict(name="prompt_image", op="prompt", dtype="bf16", **d, q_lens="3241", kv_lens="3241"),
        # requests that arrive together, one token to some thousand, smaller heads, the other type
        dict(name="prompt_ragged", op="prompt", dtype="f16", heads=16, kv_heads=4, dim=64,
             q_lens="1,1790,33,640,129,1,977,256,2303", kv_lens="1,1790,161,640,129,900,977,256,2303"),
        # the encode + scatter workload's own batch: 4 sequences of 4,096 tokens
        dict(name="prompt_batch", op="prompt", dtype="bf16", **d, q_lens="4096,4096,4096,4096",
             kv_lens="4096,4096,4096,4096"),
        # one decoding step of 64 sequences: a row each, into pages that are part full
        dict(name="append_step", op="append", dtype="bf16", **d, lens=_text(211 * i + 5 for i in range(64)),
             new=_text([1] * 64)),
        # the prompts of the encode + scatter batch into an empty cache, and one that goes on
        dict(name="append_prompts", op="append", dtype="bf16", **d, lens="0,0,0,0,1001", new="4096,4096,4096,4096,333"),
        # one user's next token after an image and a question: latency
        dict(name="cache_one", op="cache", dtype="bf16", **d, lens="3242", q_len=1, weights=False),
        # a serving batch of ragged lengths, one of them not yet begun
        dict(name="cache_batch", op="cache", dtype="bf16", **d,
             lens=_text([0] + [(i * 7919) % 16000 + 1 for i in range(1, 32)]), q_len=1, weights=False),
        # the longest contexts of the configuration, 131,072 tokens, beside a short one
        dict(name="cache_long", op="cache", dtype="bf16", **d, lens="131072,131071,77,98304", q_len=1, weights=False),
        # four drafted tokens to verify, every key's weight summed for a later eviction, smaller heads
        dict(name="cache_verify", op="cache", dtype="f16", heads=16, kv_heads=4, dim=64,
             lens=_text((i * 1237) % 6000 + 2 for i in range(24)), q_len=4, weights=True),
        # one image's keys thinned to a third once the question has been read
        dict(name="evict_image", op="evict", dtype="bf16", kv_heads=8, dim=128, lens="3242", budget=1024, sinks=4,
             recent=128),
        # a batch of long contexts cut to a quarter, one that fits as it is
        dict(name="evict_batch", op="evict", dtype="bf16", kv_heads=8, dim=128,
             lens="16384,16001,9000,16383,4097,500,12345,16384", budget=4096, sinks=16, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "append", "cache", "evict"])
    heads, kv_heads = rng.choice(HEADS)
    dim, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "f16"])
    base = dict(op=op, dtype=dtype, kv_heads=kv_heads, dim=dim)
    if op == "prompt":
        n, top = _log(rng, 1, 12), _log(rng, 16, 4096)
        q = [_log(rng, 1, top) for _ in range(n)]
        kv = [x + (_log(rng, 1, 2048) if rng.random() < 0.3 else 0) for x in q]
        while n * max(q) * max(kv) * heads > 32 << 26:  # the largest listed case's scores
            q, kv = [(x + 1) // 2 for x in q], [max((x + 1) // 2, (y + 1) // 2) for x, y in zip(q, kv)]
        return dict(base, heads=heads, q_lens=_text(q), kv_lens=_text(kv))
    if op == "append":
        n = _log(rng, 1, 64)
        new = [1] * n if rng.random() < 0.5 else [_log(rng, 1, 16384 // n) for _ in range(n)]
        return dict(base, lens=_text(rng.choice([0, _log(rng, 1, 4000)]) for _ in range(n)), new=_text(new))
    if op == "cache":
        n = _log(rng, 1, 64)
        top = _log(rng, 64, 262144 // n if n > 1 else 131072)
        return dict(base, heads=heads, lens=_text(rng.randint(0, top) for _ in range(n)),
                    q_len=rng.choice([1, 1, 1, 2, 3, 4, 5, 8]), weights=rng.random() < 0.4)
    n = _log(rng, 1, 8)
    budget = _log(rng, 16, 4096)
    return dict(base, lens=_text(rng.randint(0, 4 * budget) for _ in range(n)), budget=budget,
                sinks=rng.randint(0, budget // 8), recent=rng.randint(0, budget // 4))


# ----------------------------------------------------------------------------------------------------------------------
# The 4-bit format in elementary operations
# ----------------------------------------------------------------------------------------------------------------------

def _quantise(x, sg):
    """x [..., dim] -> (codes uint8 [..., dim] with the sign in bit 3, scales E4M3 [..., dim / 16]); every step one fp32 operation."""
    x = x.float().unflatten(-1, (-1, 16))
    sg = torch.tensor(sg, dtype=torch.float32, device=x.device)
    s = (x.abs().amax(-1) / (sg * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = s.float() * sg
    r = torch.where(step > 0, 1.0 / step, torch.zeros_like(step))
    y = x * r.unsqueeze(-1)
    a = y.abs()
    # nearest, ties to the even code: the borders of 0.5, 1.5, 3 and 6 are open below, those of 1, 2 and 4 closed
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(y).to(torch.uint8) * 8
    return code.flatten(-2), s


def _values(codes, scales):
    """Packed codes [..., dim / 2] and scale bytes [..., dim / 16] -> code * scale in fp32 (exact), [..., dim]."""
    one = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float32, device=codes.device)
    lut = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)  # byte -> (low nibble, high nibble)
    v = lut[codes.int()].flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _split(pages, dim):
    """The four parts of pages [..., page bytes]: key codes, value codes, key scales, value scales, a row per token."""
    a, b = PAGE * dim // 2, PAGE * dim // 16
    part = lambda lo, n, w: pages[..., lo:lo + n].unflatten(-1, (PAGE, w))  # noqa: E731
    return part(0, a, dim // 2), part(a, a, dim // 2), part(2 * a, b, dim // 16), part(2 * a + b, b, dim // 16)


def _rows(part, table, n):
    """part [n_pages, heads, 64, w] through table [S, max_pages] -> the first n rows of every sequence [S, heads, n, w]."""
    x = part[table[:, :max(1, -(-n // PAGE))].long()]  # [S, pages, heads, 64, w]
    return x.transpose(1, 2).flatten(2, 3)[:, :, :n]


# ----------------------------------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * gain).to(dtype)


def _channels(g, heads, dim):
    """Per-channel gains: a few channels of keys are several times the others."""
    u = torch.rand((heads, dim), generator=g, device="cuda")
    return torch.where(u > 0.96, 3.0, 0.5 + u)


def _dev(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def _pool(g, case, lens, spare=0):
    """Random full pages behind a shuffled table: (pages, table, what is left of the shuffle)."""
    heads, dim = case["kv_heads"], case["dim"]
    need = [max(1, -(-x // PAGE)) for x in lens]
    width = max(need)
    n = sum(need) + spare + 3
    page_bytes = PAGE * (dim + dim // 8)
    pages = torch.randint(0, 256, (n, heads, page_bytes), generator=g, device="cuda", dtype=torch.uint8)
    # scales as they come of data: E4M3 codes 0x48 .. 0x6f (4 to 120), none of them NaN or negative
    pages[..., PAGE * dim:] = pages[..., PAGE * dim:] % 40 + 0x48
    order = torch.randperm(n, generator=g, device="cuda").int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(need):  # entries behind a sequence's last page name no page
        table[i, :m] = order[at:at + m]
        at += m
    return pages, table, order[at:]


def prepare(case, seed):
    g = _gen(seed)
    dim, kvh, dtype = case["dim"], case["kv_heads"], DTYPES[case["dtype"]]
    st = dict(case=case, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "prompt":
        heads, ql, kl = case["heads"], _ints(case["q_lens"]), _ints(case["kv_lens"])
        if ql == kl:  # the three are column blocks of one projection's output
            qkv = _normal(g, (sum(ql), heads + 2 * kvh, dim), dtype)
            q, k, v = qkv.split([heads, kvh, kvh], 1)
        else:  # the prefix comes from a cache
            q, k, v = (_normal(g, (n, h, dim), dtype) for n, h in ((sum(ql), heads), (sum(kl), kvh), (sum(kl), kvh)))
        q *= 1.5
        return dict(st, q=q, k=k, v=v, q_lens=ql, kv_lens=kl, cu_q=_dev(_cu(ql)), cu_k=_dev(_cu(kl)))
    if case["op"] == "append":
        lens, new = _ints(case["lens"]), _ints(case["new"])
        pages, table, _ = _pool(g, case, [a + b for a, b in zip(lens, new)])
        gain = _channels(g, kvh, dim)
        k, v = (_normal(g, (sum(new), kvh, dim), torch.float32) for _ in range(2))
        return dict(st, pages=pages, table=table.clamp(min=0), lens=_dev(lens), cu=_dev(_cu(new)),
                    n_new=sum(new), k=(k * gain).to(dtype), v=v.to(dtype))
    lens = _ints(case["lens"])
    if case["op"] == "cache":
        pages, table, _ = _pool(g, case, lens)
        n = len(lens)
        # queries that give the codes' logits a spread of a few units
        q = _normal(g, (n * case["q_len"], case["heads"], dim), dtype, 0.8)
        st.update(pages=pages, table=table, lens=_dev(lens), q=q, longest=max(lens),
                  workspace=torch.empty(96 << 20, dtype=torch.uint8, device="cuda"))
        if case["weights"]:
            st["weights"] = torch.rand((n, kvh, table.shape[1] * PAGE), generator=g, device="cuda")
        return st
    budget = case["budget"]
    kept = [min(x, budget) for x in lens]
    out_pages = max(1, -(-budget // PAGE))
    pages, table, left = _pool(g, case, lens, spare=len(lens) * out_pages)
    w = torch.rand((len(lens), kvh, table.shape[1] * PAGE), generator=g, device="cuda")
    w = w.pow(6) * 8.0  # few keys have most of the weight
    w = torch.where(w < 1e-3, torch.zeros_like(w), w)  # and many have none that counts: ties
    return dict(st, pages=pages, table=table, lens=_dev(lens), weights=w,
                to_table=left[:len(lens) * out_pages].reshape(len(lens), out_pages).contiguous(), cu=_dev(_cu(kept)),
                n_kept=sum(kept), workspace=torch.empty(96 << 20, dtype=torch.uint8, device="cuda"))


# ----------------------------------------------------------------------------------------------------------------------
# The operators
# ----------------------------------------------------------------------------------------------------------------------

def _softmax(s, dead):
    """Over the last axis in fp32; keys that are dead weigh nothing, and a row without keys is 0."""
    s = s.masked_fill_(dead, float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = s.sub_(m).exp_()
    return p.div_(p.sum(-1, keepdim=True).clamp(min=1e-38))


def _prompt(st):
    q, k, v, cu_q, cu_k = st["q"], st["k"], st["v"], st["cu_q"].long(), st["cu_k"].long()
    heads, kvh, dim = q.shape[1], k.shape[1], q.shape[2]
    nq, nk = max(st["q_lens"]), max(st["kv_lens"])
    iq, ik = torch.arange(nq, device=q.device), torch.arange(nk, device=q.device)
    lq, lk = cu_q.diff()[:, None], cu_k.diff()[:, None]
    at_q = (cu_q[:-1, None] + iq).clamp(max=q.shape[0] - 1)
    at_k = (cu_k[:-1, None] + ik).clamp(max=k.shape[0] - 1)
    qf = q.float()[at_q].unflatten(2, (kvh, -1)).permute(0, 2, 3, 1, 4)  # [S, kv head, group, query, dim]
    kf, vf = (x.float()[at_k].transpose(1, 2) for x in (k, v))  # [S, kv head, key, dim]
    s = qf.flatten(2, 3) @ kf.transpose(2, 3)
    s = s.mul_(dim ** -0.5).unflatten(2, (heads // kvh, nq))
    # the last query sees every key; a query sees the keys up to its own place
    dead = ((ik > (iq + lk - lq)[..., None]) | (ik >= lk)[:, None])[:, None, None]
    o = (_softmax(s, dead).flatten(2, 3) @ vf).unflatten(2, (heads // kvh, nq))
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[iq < lq]  # [T, heads, dim] in the prompts' order
    return o.to(q.dtype)


def _append(st):
    pages, table, cu, dim = st["pages"], st["table"].long(), st["cu"].long(), st["k"].shape[2]
    t = torch.arange(st["n_new"], device=pages.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = st["lens"].long()[seq] + t - cu[seq]
    page, row = table[seq, pos // PAGE], pos % PAGE
    parts = _split(pages, dim)
    for i, (x, sg) in enumerate(((st["k"], K_SG), (st["v"], V_SG))):
        c, s = _quantise(x, sg)
        parts[i][page, :, row] = c[..., ::2] | (c[..., 1::2] << 4)
        parts[2 + i][page, :, row] = s.view(torch.uint8)
    kc, vc, ks, vs = (x[page, :, row] for x in parts)
    return tuple((_values(c, s) * torch.tensor(sg, device=pages.device)).to(st["k"].dtype)
                 for c, s, sg in ((kc, ks, K_SG), (vc, vs, V_SG)))


def _cache(st):
    q, lens, n = st["q"], st["lens"].long(), max(1, st["longest"])
    S, (T, heads, dim), kvh = lens.numel(), q.shape, st["pages"].shape[1]
    parts = [_rows(x, st["table"].clamp(min=0), n) for x in _split(st["pages"], dim)]
    m = T // S
    qf = q.float().view(S, m, kvh, heads // kvh, dim).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = qf @ _values(parts[0], parts[2]).transpose(2, 3)
    s = s.mul_(K_SG * dim ** -0.5).unflatten(2, (heads // kvh, m))
    j = torch.arange(n, device=q.device)
    last = lens[:, None] - m + torch.arange(m, device=q.device)  # each new token's own place
    p = _softmax(s, (j > last[..., None])[:, None, None])
    o = (p.flatten(2, 3) @ _values(parts[1], parts[3])) * V_SG
    o = o.unflatten(2, (heads // kvh, m)).permute(0, 3, 1, 2, 4).reshape(T, heads, dim).to(q.dtype)
    if "weights" not in st:
        return o
    st["weights"][..., :n] += p.sum((2, 3))
    return o, st["weights"]


def _evict(st):
    c, w, lens = st["case"], st["weights"], st["lens"].long()
    S, kvh, width = w.shape
    budget = c["budget"]
    j = torch.arange(width, device=w.device)
    n = lens[:, None]
    safe = (j < c["sinks"]) | (j >= n - c["recent"]) | (n <= budget)
    rank = torch.where(safe[:, None], torch.full_like(w, float("inf")), w)
    rank = torch.where((j < n)[:, None], rank, torch.full_like(w, float("-inf")))
    top = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]  # of equal weights the first ones
    if width < budget:
        top = torch.nn.functional.pad(top, (0, budget - width))
    new = lens.clamp(max=budget)
    live = (torch.arange(budget, device=w.device) < new[:, None])[:, None]
    kept = torch.where(live, top, torch.full_like(top, 1 << 40)).sort(-1).values
    at = torch.where(live, kept, torch.zeros_like(kept))
    out_w = torch.zeros((S, kvh, st["to_table"].shape[1] * PAGE), device=w.device)
    out_w[..., :budget] = torch.where(live, w.gather(-1, at), torch.zeros((), device=w.device))
    page = st["table"].long()[torch.arange(S, device=w.device)[:, None, None], at // PAGE]
    h = torch.arange(kvh, device=w.device)[None, :, None]
    parts = [x[page, h, at % PAGE].transpose(1, 2)[live[:, 0]] for x in _split(st["pages"], c["dim"])]
    k, v = ((_values(parts[i], parts[2 + i]) * torch.tensor(sg, device=w.device)).to(DTYPES[c["dtype"]])
            for i, sg in ((0, K_SG), (1, V_SG)))
    return new.int(), torch.where(live, kept, torch.full_like(kept, -1)).int(), out_w, k, v


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"prompt": _prompt, "append": _append, "cache": _cache, "evict": _evict}[op](st)
    from vision_language_model_b200 import vlm
    if op == "prompt":
        return vlm.prompt_attention(st["q"], st["k"], st["v"], st["q_lens"], st["kv_lens"], status=st["status"])
    if op == "append":
        vlm.kv4_append(st["pages"], st["table"], st["lens"], st["k"], st["v"], K_SG, V_SG, cu_new=st["cu"],
                       status=st["status"])
        return vlm.kv4_read(st["pages"], st["table"], K_SG, V_SG, st["cu"], st["n_new"], start=st["lens"],
                            dtype=st["k"].dtype, status=st["status"])
    if op == "cache":
        o = vlm.kv4_attention(st["pages"], st["table"], st["lens"], st["q"], K_SG, V_SG, weights=st.get("weights"),
                              workspace=st["workspace"], status=st["status"])
        return (o, st["weights"]) if "weights" in st else o
    c = st["case"]
    new, kept, w = vlm.kv4_evict(st["pages"], st["table"], st["lens"], st["weights"], st["to_table"], c["budget"],
                                 sinks=c["sinks"], recent=c["recent"], workspace=st["workspace"], status=st["status"])
    k, v = vlm.kv4_read(st["pages"], st["to_table"], K_SG, V_SG, st["cu"], st["n_kept"], dtype=DTYPES[c["dtype"]],
                        status=st["status"])
    return new, kept, w, k, v


# ----------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------------------------------------------------

def work(case):
    dim, kvh = case["dim"], case["kv_heads"]
    row4 = kvh * 2 * (dim // 2 + dim // 16)  # a token's keys and values in the cache
    row16 = kvh * 2 * dim * 2                # and in 16 bits
    if case["op"] == "prompt":
        ql, kl, heads = _ints(case["q_lens"]), _ints(case["kv_lens"]), case["heads"]
        pairs = sum(max(0, min(b, b - a + i + 1)) for a, b in zip(ql, kl) for i in range(a))
        return {"bytes": 2 * sum(ql) * heads * dim * 2 + sum(kl) * row16, "flops": 4 * pairs * heads * dim}
    if case["op"] == "append":
        n = sum(_ints(case["new"]))
        return {"bytes": n * (2 * row16 + 2 * row4), "flops": n * kvh * 2 * dim * 4}
    lens = _ints(case["lens"])
    if case["op"] == "cache":
        m, heads = case["q_len"], case["heads"]
        return {"bytes": sum(lens) * (row4 + (kvh * 8 if case["weights"] else 0)) + len(lens) * m * heads * dim * 4,
                "flops": 4 * sum(lens) * m * heads * dim}
    kept = sum(min(x, case["budget"]) for x in lens)
    return {"bytes": sum(lens) * kvh * 4 + kept * (kvh * 8 + 3 * row4 + row16), "flops": sum(lens) * kvh}


# ----------------------------------------------------------------------------------------------------------------------
# Exact values: every sequence and head for itself, in 64 bits, from the definitions
# ----------------------------------------------------------------------------------------------------------------------

def _round32(x):
    return x.float().double()


def _exact_quantised(x, sg):
    """The values that x [n, dim] stands for once quantised. The definition rounds each step to fp32; in between all is exact."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    sg = float(torch.tensor(sg, dtype=torch.float32))
    six = float(torch.tensor(6.0 * sg, dtype=torch.float32))
    b = x.double().reshape(x.shape[0], -1, 16)
    ratio = _round32(b.abs().amax(2) / six).clamp(max=448.0)
    # E4M3: steps of an eighth of the power of two below, of 2^-9 under 2^-6; ties to even
    step = torch.exp2(torch.floor(torch.log2(ratio.clamp(min=2.0 ** -6))) - 3.0)
    scale = torch.round(ratio / step) * step
    unit = _round32(scale * sg)
    inverse = _round32(torch.where(unit > 0, 1.0 / unit, 0.0))
    y = _round32(b * inverse[..., None])
    off = (y.abs()[..., None] - grid).abs()
    near = off.amin(-1, keepdim=True)
    tied = off == near
    even = torch.arange(8, device=x.device) % 2 == 0
    code = torch.where(tied.sum(-1) > 1, (tied & even).int().argmax(-1), tied.int().argmax(-1))
    return (torch.copysign(grid[code], y) * scale[..., None] * sg).reshape(x.shape)


def _exact_read(pages, table, seq, head, n, dim, which):
    """Keys (which 0) or values (1) of one sequence and head, code * scale, [n, dim] in 64 bits."""
    at = table[seq, :max(1, -(-n // PAGE))].long()
    raw = pages[at, head]
    a, b = PAGE * dim // 2, PAGE * dim // 16
    codes = raw[:, which * a:(which + 1) * a].reshape(-1, dim // 2)[:n].long()
    sc = raw[:, 2 * a + which * b:2 * a + (which + 1) * b].reshape(-1, dim // 16)[:n].long()
    nib = torch.stack([codes & 15, codes >> 4], 2).reshape(n, dim)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=pages.device)
    e, m = (sc >> 3) & 15, (sc & 7).double()
    scale = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e.double() - 7.0) * (1.0 + m / 8.0))
    return torch.where(nib >= 8, -1.0, 1.0) * grid[nib & 7] * scale.repeat_interleave(16, 1)


def _exact_attention(q, k, v, scale, first):
    """q [rows, m, dim] over keys k [n, dim]: query i sees the keys up to first + i. Returns (output, every key's summed weight)."""
    s = torch.einsum("gmd,nd->gmn", q, k) * scale
    see = torch.arange(k.shape[0], device=k.device) <= first + torch.arange(q.shape[1], device=k.device)[:, None]
    top = torch.where(see, s, -math.inf).amax(-1, keepdim=True)
    e = torch.where(see, torch.exp(s - torch.where(top == -math.inf, 0.0, top)), 0.0)
    p = e / torch.where(see.any(-1, keepdim=True), e.sum(-1, keepdim=True), 1.0)
    return torch.einsum("gmn,nd->gmd", p, v), p.sum((0, 1))


def exact(case, seed):
    st = prepare(case, seed)
    dim, kvh = case["dim"], case["kv_heads"]
    ksg, vsg = (float(torch.tensor(x, dtype=torch.float32)) for x in (K_SG, V_SG))
    if case["op"] == "prompt":
        G = case["heads"] // kvh
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        q0 = k0 = 0
        for a, b in zip(st["q_lens"], st["kv_lens"]):
            for h in range(kvh):
                for lo in range(0, a, 1024):  # rows at a time, for memory
                    hi = min(a, lo + 1024)
                    q = st["q"][q0 + lo:q0 + hi, h * G:(h + 1) * G].double().transpose(0, 1)
                    k, v = (st[x][k0:k0 + b, h].double() for x in "kv")
                    out[q0 + lo:q0 + hi, h * G:(h + 1) * G] = _exact_attention(q, k, v, dim ** -0.5, b - a + lo)[0].transpose(0, 1)
            q0, k0 = q0 + a, k0 + b
        return out
    if case["op"] == "append":
        return tuple(_exact_quantised(st[x].reshape(-1, dim), sg).reshape(st[x].shape) for x, sg in (("k", K_SG), ("v", V_SG)))
    lens = _ints(case["lens"])
    if case["op"] == "cache":
        m, G = case["q_len"], case["heads"] // kvh
        out = torch.zeros((len(lens) * m, case["heads"], dim), dtype=torch.float64, device="cuda")
        w = st["weights"].double() if case["weights"] else None
        for i, n in enumerate(lens):
            if n == 0:
                continue
            for h in range(kvh):
                k, v = (_exact_read(st["pages"], st["table"], i, h, n, dim, x) for x in (0, 1))
                q = st["q"][i * m:(i + 1) * m, h * G:(h + 1) * G].double().transpose(0, 1)
                o, p = _exact_attention(q, k, v, dim ** -0.5 * ksg, n - m)
                out[i * m:(i + 1) * m, h * G:(h + 1) * G] = o.transpose(0, 1) * vsg
                if w is not None:
                    w[i, h, :n] += p
        return out if w is None else (out, w)
    budget = case["budget"]
    w = st["weights"].double().cpu()
    new, out_w = [], torch.zeros((len(lens), kvh, st["to_table"].shape[1] * PAGE), dtype=torch.float64)
    kept = torch.full((len(lens), kvh, budget), -1, dtype=torch.int32)
    ks, vs = [], []
    for i, n in enumerate(lens):
        new.append(min(n, budget))
        rows = ([], [])
        for h in range(kvh):
            if n <= budget:
                ids = list(range(n))
            else:
                mid = range(case["sinks"], n - case["recent"])
                wh = w[i, h].tolist()
                best = sorted(mid, key=lambda j: (-wh[j], j))[:budget - case["sinks"] - case["recent"]]
                ids = sorted([*range(case["sinks"]), *best, *range(n - case["recent"], n)])
            at = torch.tensor(ids, dtype=torch.long)
            kept[i, h, :len(ids)] = at.int()
            out_w[i, h, :len(ids)] = w[i, h, at]
            for which, sg in ((0, ksg), (1, vsg)):
                rows[which].append(_exact_read(st["pages"], st["table"], i, h, n, dim, which)[at.cuda()] * sg)
        ks.append(torch.stack(rows[0], 1))
        vs.append(torch.stack(rows[1], 1))
    return torch.tensor(new, dtype=torch.int32), kept, out_w, torch.cat(ks), torch.cat(vs)
