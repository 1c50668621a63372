"""Grouped-head attention on the GPU where it can go wrong: contexts that many blocks share, values that are no
numbers, scales of either sign, larger batches of appends, and workspaces and devices shared between calls."""
import pytest
import torch

import compressed_sparse_attention_13_b200 as K
from gqa_reference import assert_within, attend
from test_gpu_gqa import (DT, clean, decode_reference, fill_cache, gen, make, normal, prompt_data, prompt_reference, run_prompt,
                          table_of)

pytestmark = pytest.mark.gpu


def decode(p, n, q, kc, vc, t, lens, sinks, act, ws=None):
    out = torch.full(q.shape, float("nan"), dtype=DT[act], device="cuda")
    if ws is None:
        ws = torch.full((K.gqa_workspace_size(p, K.OP_PAGED_DECODE, n, n, t.shape[1] * p.page_size),), 0xFF, dtype=torch.uint8, device="cuda")
    K.paged_decode_attn(p, n, q, kc, vc, t.cuda(), torch.tensor(lens).cuda() - 1, None if sinks is None else sinks.cuda(), out, ws)
    return out


# One long row, or a long one among short ones: its parts lie in up to all blocks and are joined.
LONG = [
    # act, cache, H, HK, d, page, lens
    ("bf16", "bf16", 1, 1, 128, 16, [20011]),
    ("bf16", "bf16", 16, 2, 64, 8, [30001, 1]),
    ("bf16", "bf16", 8, 1, 256, 100, [9000, 64, 0]),
    ("bf16", "fp8", 8, 1, 128, 64, [25000]),
    ("bf16", "fp8", 3, 1, 192, 16, [12007, 33]),
    ("f32", "f32", 2, 1, 64, 16, [30011]),
    ("f32", "f32", 9, 1, 128, 7, [8009, 2]),
    ("f32", "fp8", 8, 1, 256, 16, [6000]),
    ("f32", "bf16", 1, 1, 192, 3, [5003, 5003]),
]


@pytest.mark.parametrize("flags", [0, K.FLAG_BATCH_INVARIANT], ids=["", "invariant"])
@pytest.mark.parametrize("case", LONG, ids=lambda c: f"{c[0]}-{c[1]}-H{c[2]}x{c[3]}-d{c[4]}-p{c[5]}-{c[6][0]}")
def test_decode_of_rows_that_many_blocks_share(case, flags):
    act, cache, H, HK, d, page, lens = case
    g, _ = gen(51), clean()
    p = make(H, HK, d, act, cache, page_size=page, flags=flags)
    held = [-(-n // page) for n in lens]
    t = table_of(g, held, max(held))
    kc, vc = fill_cache(g, p, sum(held), cache)
    q = normal(g, len(lens), H, d, dt=DT[act]).cuda()
    sinks = normal(g, H)
    ref, tol = decode_reference(p, q, kc, vc, t, lens, sinks, act, cache)
    out = decode(p, len(lens), q, kc, vc, t, lens, sinks, act)
    assert clean() == 0
    assert_within(out, ref, tol, "long")
    assert torch.equal(out, decode(p, len(lens), q, kc, vc, t, lens, sinks, act))


@pytest.mark.parametrize("act,cache", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32"), ("f32", "fp8")])
@pytest.mark.parametrize("n", [40, 5000])
def test_decode_of_a_query_that_is_no_number(act, cache, n):
    """A NaN in a head's query makes that head NaN and no other, in a short row and in one that is joined from parts."""
    p, g = make(4, 2, 128, act, cache, page_size=16), gen(52)
    held = -(-n // 16)
    t = table_of(g, [held, held], held)
    kc, vc = fill_cache(g, p, 2 * held, cache)
    q = normal(g, 2, 4, 128, dt=DT[act])
    ref, tol = decode_reference(p, q, kc, vc, t, [n, n], None, act, cache)
    q[1, 2, 77] = float("nan")
    out = decode(p, 2, q.cuda(), kc, vc, t, [n, n], None, act).cpu()
    assert torch.isnan(out[1, 2].float()).all()
    keep = torch.ones(2, 4, dtype=torch.bool)
    keep[1, 2] = False
    assert_within(out[keep], ref[keep], tol[keep], "other heads")


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sink", [False, True])
def test_prompt_of_a_query_that_is_no_number(act, d, sink):
    g = gen(53)
    wide, kv, cq, ck = prompt_data(g, act, 4, 2, d, [150, 30], [150, 30])
    p = make(4, 2, d, act)
    q, k, v = wide[:, :4 * d].unflatten(1, (4, d)).contiguous(), *(x.unflatten(1, (2, d)).contiguous() for x in kv.split(2 * d, 1))
    sinks = normal(g, 4) if sink else None
    ref, tol = prompt_reference(p, q, k, v, cq, ck, sinks, act)
    q[100, 3, d - 1], q[5, 0, 0] = float("nan"), float("inf")
    out = run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, sinks, act).cpu()
    keep = torch.ones(q.shape[:2], dtype=torch.bool)
    keep[180:] = keep[100, 3] = keep[5, 0] = False
    assert_within(out[keep], ref[keep], tol[keep], "other rows")
    assert torch.isnan(out[100, 3].float()).all()


@pytest.mark.parametrize("scale", [-0.25, 0.0])
@pytest.mark.parametrize("act,cache", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32")])
def test_scales_of_zero_and_below(scale, act, cache):
    g = gen(54)
    p = make(4, 2, 64, act, cache, page_size=16, window=70, scale=scale)
    t = table_of(g, [20, 3], 20)
    kc, vc = fill_cache(g, p, 23, cache)
    q, lens = normal(g, 2, 4, 64, dt=DT[act]).cuda(), [311, 40]
    ref, tol = decode_reference(p, q, kc, vc, t, lens, None, act, cache)
    assert_within(decode(p, 2, q, kc, vc, t, lens, None, act), ref, tol, "decode")
    wide, kv, cq, ck = prompt_data(g, act, 4, 2, 64, [200, 9], [200, 9])
    q, k, v = wide[:, :256].unflatten(1, (4, 64)).contiguous(), *(x.unflatten(1, (2, 64)).contiguous() for x in kv.split(128, 1))
    ref, tol = prompt_reference(p, q, k, v, cq, ck, None, act)
    out = run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, None, act)
    assert_within(out[:209], ref[:209], tol[:209], "prompt")


PROMPTS = [
    # act, H, HK, d, window, lens_q, lens_k: many key tiles, chunks of several sizes, windows that begin inside tiles
    ("f32", 2, 1, 64, 0, [700], [700]),
    ("f32", 2, 2, 128, 0, [300, 40], [520, 650]),
    ("f32", 2, 1, 192, 130, [400], [400]),
    ("bf16", 6, 1, 128, 0, [300, 1, 64], [1100, 700, 64]),
    ("bf16", 2, 2, 128, 300, [900], [900]),
    ("bf16", 1, 1, 64, 100, [129, 700], [400, 700]),
    ("bf16", 2, 1, 192, 65, [500], [700]),
    ("bf16", 2, 2, 256, 0, [300], [900]),
]


@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: f"{c[0]}-H{c[1]}x{c[2]}-d{c[3]}-w{c[4]}-{c[5][0]}-{c[6][0]}")
def test_prompts_over_many_key_tiles(case):
    act, H, HK, d, window, lq, lk = case
    g, _ = gen(55), clean()
    wide, kv, cq, ck = prompt_data(g, act, H, HK, d, lq, lk)
    p = make(H, HK, d, act, window=window)
    q, k, v = wide[:, :H * d].unflatten(1, (H, d)).contiguous(), *(x.unflatten(1, (HK, d)).contiguous() for x in kv.split(HK * d, 1))
    ref, tol = prompt_reference(p, q, k, v, cq, ck, None, act)
    out = run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, None, act)
    n = int(cq[-1])
    assert clean() == 0
    assert_within(out[:n], ref[:n], tol[:n], "tiles")
    assert (out[n:] == 9).all()


@pytest.mark.parametrize("act,cache,d,H,HK,rot,pairs", [("bf16", "bf16", 128, 8, 2, 128, False), ("bf16", "fp8", 192, 3, 1, 48, False),
                                                        ("f32", "f32", 64, 5, 5, 32, True), ("bf16", "fp8", 256, 1, 1, 112, True)])
@pytest.mark.parametrize("n_seq", [3, 40])
def test_append_of_many_tokens_is_that_of_its_tokens_one_by_one(act, cache, d, H, HK, rot, pairs, n_seq):
    """A batch large enough for several tokens a block, and sequences enough for a search, against calls of one token per
    sequence: the same bits everywhere, nothing outside."""
    clean()
    g, page = gen(56), 16
    lens = [1201 // n_seq + (7 * i) % 13 for i in range(n_seq)]
    starts = [(31 * i) % 50 - (1 if i == 1 else 0) for i in range(n_seq)]
    starts[2] = -5                                   # left out
    p = make(H, HK, d, act, cache, page_size=page, rot_dim=rot, flags=K.FLAG_ROT_PAIRS if pairs else 0)
    f = (1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).cuda()
    n, held = sum(lens) + 3, [-(-(a + max(s, 0)) // page) for a, s in zip(lens, starts)]
    t = table_of(g, held, max(held)).cuda()
    q, k, v = (normal(g, n, h, d, dt=DT[act]).cuda() for h in (H, HK, HK))
    cu = torch.tensor([sum(lens[:i]) for i in range(n_seq + 1)], dtype=torch.int32).cuda()

    def fresh():
        kc, vc = K.empty_paged(p, sum(held))
        for x in (kc.data, vc.data, kc.scales, vc.scales):
            if x is not None:
                x.zero_()
        return kc, vc, torch.full_like(q, 7), torch.full_like(k, 7)

    kc, vc, qo, ko = fresh()
    K.paged_append(p, n_seq, n, cu, torch.tensor(starts).cuda(), q, k, v, f, qo, ko, kc, vc, t)
    kc2, vc2, qo2, ko2 = fresh()
    for i in range(max(lens)):
        rows = [int(cu[s]) + i for s in range(n_seq) if i < lens[s]]
        pos = [starts[s] + i if starts[s] >= 0 else -1 for s in range(n_seq) if i < lens[s]]
        pick = [s for s in range(n_seq) if i < lens[s]]
        a, b = torch.full_like(q[rows], 7), torch.full_like(k[rows], 7)
        K.paged_append(p, len(rows), len(rows), None, torch.tensor(pos).cuda(), q[rows], k[rows], v[rows], f, a, b, kc2, vc2,
                       t[pick].contiguous())
        qo2[rows], ko2[rows] = a, b
    assert clean() == 0
    for x, y in ((qo, qo2), (ko, ko2), (kc.data, kc2.data), (vc.data, vc2.data)) + (
            ((kc.scales, kc2.scales), (vc.scales, vc2.scales)) if cache == "fp8" else ()):
        assert torch.equal(x, y)
    left = slice(int(cu[2]), int(cu[3]))
    assert (qo[left] == 7).all() and (qo[n - 3:] == 7).all()


def test_two_captured_graphs_share_a_workspace():
    """Replayed one after the other on a stream, in any order: a workspace carries nothing from call to call."""
    g = gen(57)
    p = make(8, 1, 128, page_size=16)
    shapes = [[9000], [700, 5000, 3, 64]]
    total = max(sum(-(-n // 16) for n in lens) for lens in shapes)
    kc, vc = fill_cache(g, p, total, "bf16")
    ws = torch.empty(K.gqa_workspace_size(p, K.OP_PAGED_DECODE, 4, 4, 9008), dtype=torch.uint8, device="cuda")
    runs = []
    for lens in shapes:
        held = [-(-n // 16) for n in lens]
        t = table_of(g, held, max(held)).cuda()
        q, pos = normal(g, len(lens), 8, 128, dt=torch.bfloat16).cuda(), torch.tensor(lens).cuda() - 1
        want = decode(p, len(lens), q, kc, vc, t, lens, None, "bf16")
        out, graph = torch.zeros_like(q), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            K.paged_decode_attn(p, len(lens), q, kc, vc, t, pos, None, out, ws)
        runs.append((graph, out, want, (q, t, pos)))
    for i in (0, 1, 1, 0, 1, 0):
        graph, out, want, _ = runs[i]
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_a_call_makes_the_device_of_its_tensors_current():
    """The stream is that of the tensors' device, the caller's current device stays."""
    p, g = make(2, 1, 64, page_size=4), gen(58)
    kc, vc = fill_cache(g, p, 4, "bf16")
    q = normal(g, 1, 2, 64, dt=torch.bfloat16).cuda()
    t = torch.arange(4, dtype=torch.int32)[None]
    ref, tol = decode_reference(p, q, kc, vc, t, [13], None, "bf16", "bf16")
    last = torch.cuda.device_count() - 1
    before = torch.cuda.current_device()
    with torch.cuda.device(last):
        out = decode(p, 1, q, kc, vc, t, [13], None, "bf16")
        assert torch.cuda.current_device() == last
    assert torch.cuda.current_device() == before
    assert_within(out, ref, tol, "device")


def test_prompt_with_fewer_keys_than_queries_that_are_all_hidden():
    """Sequences whose keys begin behind all but their last queries, or that have none: rows of 0 beside others."""
    g = gen(59)
    lq, lk = [300, 256, 130], [2, 0, 130]
    for act, d in (("bf16", 128), ("bf16", 64), ("bf16", 256), ("f32", 64)):
        wide, kv, cq, ck = prompt_data(g, act, 2, 1, d, lq, lk)
        p = make(2, 1, d, act)
        q, k, v = wide[:, :2 * d].unflatten(1, (2, d)).contiguous(), *(x.unflatten(1, (1, d)).contiguous() for x in kv.split(d, 1))
        for sinks in (None, normal(g, 2)):
            ref, tol = prompt_reference(p, q, k, v, cq, ck, sinks, act)
            out = run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, sinks, act)
            assert_within(out[:686], ref[:686], tol[:686], "hidden")
            assert (out[:298] == 0).all() and (out[300:556] == 0).all()


def test_attend_reference_of_one_key_is_its_value():
    """The reference itself, on the smallest case: one key, no sink."""
    v = torch.randn(1, 1, 64, dtype=torch.float64)
    o, _ = attend(torch.randn(1, 2, 64, dtype=torch.float64), torch.randn(1, 1, 64, dtype=torch.float64), v, 0.1,
                  torch.ones(1, 1, dtype=torch.bool), None, torch.float32, 0.0)
    assert torch.equal(o, v.expand(1, 2, 64))


def test_prompts_replayed_from_a_graph_with_other_lengths():
    """The lengths are read on the device: a captured call serves any batch that fits its buffers."""
    g = gen(60)
    p = make(4, 2, 128)
    n, n_seq = 700, 5
    q, k, v = (normal(g, n, h, 128, dt=torch.bfloat16).cuda() for h in (4, 2, 2))
    cu, out = torch.zeros(n_seq + 1, dtype=torch.int32, device="cuda"), torch.zeros_like(q)
    ws = torch.empty(K.gqa_workspace_size(p, K.OP_PROMPT_ATTN, n_seq, n, 0), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.prompt_attn(p, n_seq, q, k, v, cu, cu, None, out, ws)
    for lens in ([700, 0, 0, 0, 0], [1, 2, 3, 4, 5], [0, 130, 0, 257, 313], [140] * 5):
        at = torch.tensor([sum(lens[:i]) for i in range(n_seq + 1)], dtype=torch.int32)
        cu.copy_(at)
        out.fill_(9)
        graph.replay()
        ref, tol = prompt_reference(p, q.cpu(), k.cpu(), v.cpu(), at, at, None, "bf16")
        m = sum(lens)
        assert_within(out[:m], ref[:m], tol[:m], str(lens))
        assert (out[m:] == 9).all()
