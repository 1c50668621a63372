"""Grouped-head attention on the GPU at the ends of what its arguments and values may be."""
import pytest
import torch

import compressed_sparse_attention_13_b200 as K
from gqa_reference import assert_within
from test_gpu_gqa import clean, gen, make, normal, prompt_data, prompt_reference, run_prompt

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
