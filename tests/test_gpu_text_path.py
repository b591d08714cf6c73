"""The text side's operators as a serving program uses them together, and how
they behave on streams and in graphs."""
import numpy as np
import pytest
import torch

from oracle import text_oracle as T
from tests import text_util as U
from tests.gpu_util import guarded, guarded_copy, to_np
from vision_language_model_b200 import synth, vlm

pytestmark = pytest.mark.gpu
PAGE, K_SG, V_SG = U.PAGE, U.K_SG, U.V_SG


def test_an_image_prompt_from_its_embeddings_to_an_evicted_cache():
    """Placeholders expanded, image rows scattered, one projection's q, k, v through the prompt's
    attention into the cache, two tokens decoded with weights, the cache thinned, a third token over
    what is left, and a second prompt chunk over the cached prefix read back."""
    heads, kv_heads, dim, width = 8, 2, 64, 256
    scale = dim ** -0.5
    prompts = [synth.text_sequences(1, 1, 40, [[1]]).reshape(-1), synth.text_sequences(2, 1, 9, [[1]]).reshape(-1)]
    counts = [150, 61]
    ids = torch.cat([torch.where(p == 10, 7, p) for p in prompts]).cuda()
    status = vlm.new_status()
    ids = vlm.expand_placeholders(ids, 7, counts, status=status)
    lens = [len(p) - 1 + c for p, c in zip(prompts, counts)]
    n = sum(lens)
    assert ids.numel() == n
    text = synth.text_embeddings(3, n, width).cuda()
    vlm.scatter(ids, synth.randn_bf16(4, "img", (sum(counts), width), 1.0).cuda(), text, 10, status=status)
    w = synth.randn_bf16(5, "w", ((heads + 2 * kv_heads) * dim, width), 0.1).cuda()
    qkv = vlm.gemm(vlm.EPI_BF16, text, w, torch.empty((n, w.shape[0]), dtype=torch.bfloat16, device="cuda"), status=status)
    q, k, v = qkv.view(n, -1, dim).split([heads, kv_heads, kv_heads], 1)

    # the prompt
    out = vlm.prompt_attention(q, k, v, lens, status=status)
    o, a = T.prompt_attention(q.float().cpu(), k.float().cpu(), v.float().cpu(), lens, lens, scale)
    ds = U.logit_error(q.float().cpu().numpy(), k.float().cpu().numpy(), scale)
    U.assert_close(out, o, U.prompt_tolerance(torch.bfloat16, o, a, ds), "prompt")

    # into the cache
    S = 2
    budget, room = 96, [-(-(m + 4) // PAGE) for m in lens]
    n_pages = sum(room) + 2 * S + 1
    pages = vlm.kv4_pages(n_pages, kv_heads, dim)
    order = np.random.default_rng(0).permutation(n_pages).astype(np.int32)
    table = np.full((S, max(room)), -1, np.int32)
    table[0, :room[0]], table[1, :room[1]] = order[:room[0]], order[room[0]:sum(room)]
    to = order[sum(room):sum(room) + 2 * S].reshape(S, 2)
    gt, gto = U.cuda_int(table), U.cuda_int(to)
    cu = U.cuda_int(np.concatenate([[0], np.cumsum(lens)]))
    vlm.kv4_append(pages, gt, None, k, v, K_SG, V_SG, cu_new=cu, status=status)
    ref = np.zeros(tuple(pages.shape), np.uint8)
    for s in range(S):
        rows = slice(int(cu[s]), int(cu[s + 1]))
        T.write(ref, table, s, 0, k[rows].float().cpu().numpy(), v[rows].float().cpu().numpy(), K_SG, V_SG)

    # two tokens, one after the other, every place's weight summed
    weights = torch.zeros((S, kv_heads, table.shape[1] * PAGE), device="cuda")
    want_w = np.zeros(tuple(weights.shape))
    at = np.array(lens)
    for step in range(2):
        tok = U.rand16(10 + step, (S, heads + 2 * kv_heads, dim), torch.bfloat16).cuda()
        tq, tk, tv = tok.split([heads, kv_heads, kv_heads], 1)
        vlm.kv4_append(pages, gt, U.cuda_int(at), tk, tv, K_SG, V_SG, status=status)
        for s in range(S):
            T.write(ref, table, s, at[s], tk[s:s + 1].float().cpu().numpy(), tv[s:s + 1].float().cpu().numpy(), K_SG, V_SG)
        at = at + 1
        got = vlm.kv4_attention(pages, gt, U.cuda_int(at), tq, K_SG, V_SG, weights=weights, status=status)
        o, a, w1 = T.cache_attention(ref, table, list(at), tq.float().cpu().numpy(), 1, K_SG, V_SG, scale)
        want_w += w1
        kk = np.full((1, dim), 6 * 448 * K_SG)
        ds = U.logit_error(tq.float().cpu().numpy(), kk, scale)
        U.assert_close(got, o, U.cache_tolerance(torch.bfloat16, o, a, ds, max(at), 6 * 448 * V_SG), f"token {step}")
    U.assert_close(weights, want_w, 2 * (2 * np.expm1(2 * ds) + 1e-5) * want_w + 1e-6, "weights")

    # thinned by the GPU's own weights
    new, kept, to_w = vlm.kv4_evict(pages, gt, U.cuda_int(at), weights, gto, budget, sinks=4, recent=16, status=status)
    assert vlm.status_sync(status) == vlm.OK
    hw = weights.cpu().numpy()
    thin = ref.copy()
    for s in range(S):
        for h in range(kv_heads):
            ids_ = T.keep(hw[s, h], int(at[s]), budget, 4, 16)
            assert np.array_equal(kept[s, h, :len(ids_)].cpu().numpy(), ids_)
            for i, j in enumerate(ids_):
                for off, _, wd in T._parts(dim):
                    thin[to[s, i // PAGE], h, off + (i % PAGE) * wd:off + (i % PAGE + 1) * wd] = \
                        ref[table[s, j // PAGE], h, off + (j % PAGE) * wd:off + (j % PAGE + 1) * wd]
    tq = U.rand16(20, (S, heads, dim), torch.bfloat16).cuda()
    got = vlm.kv4_attention(pages, gto, new, tq, K_SG, V_SG, weights=to_w, status=status)
    small = [min(int(x), budget) for x in at]
    o, a, _ = T.cache_attention(thin, to, small, tq.float().cpu().numpy(), 1, K_SG, V_SG, scale)
    U.assert_close(got, o, U.cache_tolerance(torch.bfloat16, o, a, ds, budget, 6 * 448 * V_SG), "after eviction")

    # another chunk of the prompts over the prefix read back
    rk, rv = vlm.kv4_read(pages, gto, K_SG, V_SG, U.cuda_int(np.concatenate([[0], np.cumsum(small)])), sum(small),
                          status=status)
    m = 5
    cq, ck, cv = (U.rand16(30 + i, (S * m, hh, dim), torch.bfloat16).cuda() for i, hh in enumerate((heads, kv_heads, kv_heads)))
    parts = []
    for x, y in ((rk, ck), (rv, cv)):
        parts.append(torch.cat([t for s in range(S) for t in (x[sum(small[:s]):sum(small[:s + 1])], y[s * m:(s + 1) * m])]))
    got = vlm.prompt_attention(cq, parts[0], parts[1], [m] * S, [x + m for x in small], status=status)
    o, a = T.prompt_attention(cq.float().cpu(), parts[0].float().cpu(), parts[1].float().cpu(), [m] * S,
                              [x + m for x in small], scale)
    ds = U.logit_error(cq.float().cpu().numpy(), parts[0].float().cpu().numpy(), scale)
    U.assert_close(got, o, U.prompt_tolerance(torch.bfloat16, o, a, ds), "second chunk")
    assert vlm.status_sync(status) == vlm.OK


def _decoder(seed, lens, heads=8, kv_heads=2, dim=128, steps=6):
    S = len(lens)
    room = [n + steps for n in lens]
    pages, table, _ = U.random_pool(seed, room, kv_heads, dim)
    g = torch.Generator("cuda").manual_seed(seed)
    toks = torch.randn((steps, S, heads + 2 * kv_heads, dim), generator=g, device="cuda").bfloat16()
    return dict(pages=torch.from_numpy(pages).cuda(), table=U.cuda_int(table), lens=U.cuda_int(lens), toks=toks,
                weights=torch.zeros((S, kv_heads, table.shape[1] * PAGE), device="cuda"), heads=heads, kv_heads=kv_heads,
                ws=guarded(vlm.kv4_attention_workspace_size(S, heads, kv_heads, dim), torch.uint8),
                out=guarded((S, heads, dim), torch.bfloat16), status=vlm.new_status())


def _step(d, tok, stream=None):
    q, k, v = tok.split([d["heads"], d["kv_heads"], d["kv_heads"]], 1)
    vlm.kv4_append(d["pages"], d["table"], d["lens"], k, v, K_SG, V_SG, status=d["status"], stream=stream)
    d["lens"] += 1
    vlm.kv4_attention(d["pages"], d["table"], d["lens"], q, K_SG, V_SG, weights=d["weights"], out=d["out"],
                      workspace=d["ws"], status=d["status"], stream=stream)


def test_a_captured_decoding_step_replays_with_growing_lengths():
    lens = [63, 0, 500, 1290]
    a, b = _decoder(1, lens), _decoder(1, lens)
    eager = []
    for tok in a["toks"]:
        _step(a, tok)
        eager.append(a["out"].clone())
    slot = b["toks"][0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm up on copies of the state
        w = _decoder(1, lens)
        _step(w, w["toks"][0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(b, slot)
    for i, tok in enumerate(b["toks"]):
        slot.copy_(tok)
        graph.replay()
        assert torch.equal(b["out"], eager[i]), i
    assert torch.equal(a["weights"], b["weights"]) and torch.equal(a["pages"], b["pages"])
    assert vlm.status_sync(a["status"]) == vlm.OK and vlm.status_sync(b["status"]) == vlm.OK


def test_a_captured_prompt_and_eviction_replay_on_new_data():
    heads, kv_heads, dim, lens = 8, 2, 64, [300, 77]
    n = sum(lens)
    q, k, v = (U.rand16(s, (n, h, dim), torch.float16).cuda() for s, h in ((1, heads), (2, kv_heads), (3, kv_heads)))
    out = torch.empty_like(q)
    pages, table, left = U.random_pool(4, lens, kv_heads, dim, spare=4)
    gp, gt, gl, gto = torch.from_numpy(pages).cuda(), U.cuda_int(table), U.cuda_int(lens), U.cuda_int(left[:4].reshape(2, 2))
    w = torch.rand((2, kv_heads, table.shape[1] * PAGE), device="cuda")

    def step():
        vlm.prompt_attention(q, k, v, lens, out=out)
        return vlm.kv4_evict(gp, gt, gl, w, gto, 100, sinks=2, recent=9)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (5, 6):
        q.copy_(U.rand16(seed, tuple(q.shape), torch.float16))
        w.copy_(torch.rand(tuple(w.shape), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        res = [out.clone()] + [x.clone() for x in got]
        want = [vlm.prompt_attention(q, k, v, lens)] + list(step())
        for x, y in zip(res, want):
            assert torch.equal(x, y)


def test_two_streams_with_their_own_workspaces():
    lens = [[700, 3, 64], [1500, 40]]
    ref = []
    for i, n in enumerate(lens):
        d = _decoder(10 + i, n)
        ref.append([])
        for tok in d["toks"]:
            _step(d, tok)
            ref[-1].append(d["out"].clone())
    ds = [_decoder(10 + i, n) for i, n in enumerate(lens)]
    streams = [torch.cuda.Stream() for _ in lens]
    torch.cuda.synchronize()
    got = [[], []]
    for step in range(6):
        for d, s, out in zip(ds, streams, got):
            with torch.cuda.stream(s):
                _step(d, d["toks"][step])
                out.append(d["out"].clone())
    torch.cuda.synchronize()
    for x, y in zip(ref, got):
        for r, g in zip(x, y):
            assert torch.equal(r, g)


def test_a_given_stream_and_buffers_of_the_calls_own():
    # outputs and workspaces that the binding makes belong to the call until the given stream is done
    s = torch.cuda.Stream()
    pages, table, _ = U.random_pool(20, [2000] * 8, 2, 128)
    gp, gt, gl = torch.from_numpy(pages).cuda(), U.cuda_int(table), U.cuda_int([2000] * 8)
    q = U.rand16(21, (8, 8, 128), torch.bfloat16).cuda()
    want = vlm.kv4_attention(gp, gt, gl, q, K_SG, V_SG)
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append(vlm.kv4_attention(gp, gt, gl, q, K_SG, V_SG, stream=s))
        torch.full((4 << 20,), 255, dtype=torch.uint8, device="cuda")  # would take a freed workspace's memory
    s.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_rows_behind_the_last_sequence_stay():
    pages, table, _ = U.random_pool(22, [100, 65], 2, 64)
    q = U.rand16(23, (2, 8, 64), torch.bfloat16).cuda()
    buf = torch.full((5, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    vlm.kv4_attention(torch.from_numpy(pages).cuda(), U.cuda_int(table), U.cuda_int([100, 65]), q, K_SG, V_SG, out=buf[:2])
    assert (buf[2:] == 3).all() and not (buf[:2] == 3).all()


def test_more_sequences_than_one_launch_takes():
    # 4,096 per launch: lengths that differ on both sides of the border
    S = 4100
    lens = np.full(S, 1, np.int64)
    lens[:7], lens[4090:] = [70, 0, 3, 64, 65, 1, 2], [0, 5, 130, 1, 1, 64, 90, 0, 33, 128]
    pages, table, _ = U.random_pool(24, list(lens), 1, 64)
    q = U.rand16(25, (S, 2, 64), torch.float16)
    w = torch.zeros((S, 1, table.shape[1] * PAGE), device="cuda")
    status = vlm.new_status()
    got = vlm.kv4_attention(torch.from_numpy(pages).cuda(), U.cuda_int(table), U.cuda_int(lens), q.cuda(), K_SG, V_SG,
                            weights=w, status=status)
    assert vlm.status_sync(status) == vlm.OK
    pick = [*range(7), *range(4088, S)]
    o, a, ww = T.cache_attention(pages, table[pick], list(lens[pick]), q[pick].float().numpy(), 1, K_SG, V_SG, 0.125)
    ds = U.logit_error(q[pick].float().numpy(), np.full((1, 64), 720.0), 0.125, float(np.float32(K_SG)))
    U.assert_close(got[pick], o, U.cache_tolerance(torch.float16, o, a, ds, 130, 720 * V_SG))
    U.assert_close(w[pick], ww, 2 * (2.0 ** -21 + np.expm1(2 * ds)) * ww + 1e-6)
