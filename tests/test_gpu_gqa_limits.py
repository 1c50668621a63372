"""Grouped-head attention on the GPU at the ends of what its arguments and values may be."""
import pytest
import torch

import compressed_sparse_attention_13_b200 as K
from gqa_paged_reference import attend_paged, scale_rows
from gqa_reference import assert_within, paged_rows
from test_gpu_gqa import DT, clean, fill_cache, gen, make, normal, prompt_data, prompt_reference, run_prompt, table_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 200])
@pytest.mark.parametrize("act,H,HK,d", [("bf16", 8, 2, 64), ("bf16", 2, 2, 128), ("bf16", 3, 1, 192), ("bf16", 4, 1, 256),
                                        ("f32", 2, 1, 64), ("f32", 2, 2, 256)])
def test_prompt_with_a_window_that_hides_nothing(act, H, HK, d, window):
    """The longest windows, with fewer keys than queries, so that queries stand before the first key: the same as no window."""
    g, _ = gen(71), clean()
    lq, lk = [300, 300, 40, 7], [120, 295, 40, 0]
    wide, kv, cq, ck = prompt_data(g, act, H, HK, d, lq, lk)
    p = make(H, HK, d, act, window=window)
    q, k, v = wide[:, :H * d].unflatten(1, (H, d)).contiguous(), *(x.unflatten(1, (HK, d)).contiguous() for x in kv.split(HK * d, 1))
    sinks = normal(g, H)
    ref, tol = prompt_reference(p, q, k, v, cq, ck, sinks, act)
    out = run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, sinks, act)
    n = int(cq[-1])
    assert clean() == 0
    assert_within(out[:n], ref[:n], tol[:n], "window")
    assert (out[180:300] != 0).any() and (out[:180] == 0).all()
    p.window = 0
    assert torch.equal(out, run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, sinks, act))


@pytest.mark.parametrize("act,cache", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32")])
@pytest.mark.parametrize("window", [0, 20, 2 ** 31 - 1])
@pytest.mark.parametrize("pages", [12, 200], ids=["whole", "split"])
def test_decode_at_any_position(act, cache, window, pages):
    """Positions at both ends of 64 bits: below 0 a row is 0, past the table it has the places that exist and is flagged."""
    g, _ = gen(72), clean()
    p = make(4, 2, 64, act, cache, page_size=8, window=window)
    cap = 8 * pages
    pos = [-2 ** 63, 50, -2 ** 63 + 7, 2 ** 63 - 1, -1, 2 ** 63 - 9, cap - 1, 2 ** 40, cap + 5]
    t = table_of(g, [pages] * len(pos), pages)
    kc, vc = fill_cache(g, p, pages * len(pos), cache)
    q, sinks = normal(g, len(pos), 4, 64, dt=DT[act]).cuda(), normal(g, 4)
    ws = torch.empty(K.gqa_workspace_size(p, K.OP_PAGED_DECODE, len(pos), len(pos), cap), dtype=torch.uint8, device="cuda")
    for i, at in enumerate(pos):
        out, tab = torch.full((1, 4, 64), float("nan"), dtype=DT[act], device="cuda"), t[i:i + 1].cuda()
        K.paged_decode_attn(p, 1, q[i:i + 1], kc, vc, tab, torch.tensor([at]).cuda(), sinks.cuda(), out, ws)
        assert clean() == (K.DEV_BAD_INDEX if at >= cap else 0)
        lo, n = max(at - window + 1, 0) if window else 0, max(min(at + 1, cap), 0)
        if n <= lo:
            assert (out == 0).all()
            continue
        k, v = (paged_rows(c, t[i], n, 8)[lo:] for c in (kc, vc))
        vs = scale_rows(vc, t[i], n, 8)[lo:] if cache == "fp8" else None
        ref, tol = attend_paged(q[i:i + 1].cpu().double(), k, v, vs, p.scale, sinks, act, cache)
        assert_within(out, ref, tol, str(at))
    every = torch.full_like(q, float("nan"))
    K.paged_decode_attn(p, len(pos), q, kc, vc, t.cuda(), torch.tensor(pos).cuda(), sinks.cuda(), every, ws)
    assert clean() == K.DEV_BAD_INDEX and torch.isfinite(every.float()).all()
    assert all((every[i] == 0).all() for i, at in enumerate(pos) if at < 0)


@pytest.mark.parametrize("n_seq", [3, 40])
def test_append_of_tokens_past_every_table(n_seq):
    """Positions up to the last one of 64 bits: such tokens are flagged and not written, and their queries and keys come out
    as those of a token, not as those of a sequence that is left out."""
    g, _ = gen(73), clean()
    p = make(2, 1, 64, page_size=4)
    starts = [2 ** 63 - 2, 0, 2 ** 40] + [0] * (n_seq - 3)
    lens = [5, 6, 2] + [1] * (n_seq - 3)
    n = sum(lens)
    cu = torch.tensor([sum(lens[:i]) for i in range(n_seq + 1)], dtype=torch.int32)
    t = torch.arange(2 * n_seq, dtype=torch.int32).view(n_seq, 2)
    kc, vc = K.empty_paged(p, 2 * n_seq)
    kc.data.zero_(), vc.data.zero_()
    q, k, v = (normal(g, n, h, 64, dt=torch.bfloat16).cuda() for h in (2, 1, 1))
    qo, ko = torch.full_like(q, 5), torch.full_like(k, 5)
    K.paged_append(p, n_seq, n, cu.cuda(), torch.tensor(starts).cuda(), q, k, v, None, qo, ko, kc, vc, t.cuda())
    assert clean() == K.DEV_BAD_INDEX
    assert torch.equal(qo, q) and torch.equal(ko, k)   # nothing is rotated
    assert torch.equal(kc.data[2:4, 0].flatten(0, 1)[:6], k[5:11, 0]) and torch.equal(vc.data[2:4, 0].flatten(0, 1)[:6], v[5:11, 0])
    assert not kc.data[[0, 1, 4, 5]].any() and not vc.data[[0, 1, 4, 5]].any()
