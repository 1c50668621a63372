"""Grouped-head attention on the GPU over values of very different size: logits that grow along a row, FP8 scales over
many powers of two, and values that are no numbers at every head dim."""
import math

import pytest
import torch

import compressed_sparse_attention_13_b200 as K
from gqa_paged_reference import attend_paged, scale_rows
from gqa_reference import assert_within, paged_rows
from test_gpu_gqa import DT, clean, gen, make, normal, prompt_data, prompt_reference, run_prompt, table_of

pytestmark = pytest.mark.gpu
LN2 = math.log(2.0)


def growth(kind, n, g):
    """Logits of a row of n keys, in log2 units.  A block has whole pieces of 512 keys of a row (batch-invariant mode), or
    about as many; a warp takes 16 (8 in full precision) of every 64 (32)."""
    i = torch.arange(n)
    x = 0.5 * torch.randn(n, generator=g, dtype=torch.float64)
    if kind == "shelf":   # many keys near 0, then in each tile one that lies 10 higher: both parts count in the result
        return x + 10.0 * ((i % 512 >= 448) & (i % 8 == 3))
    if kind == "saw":     # three rises of 9.5 and a fall
        return x + 9.5 * (i // 64 % 4)
    if kind == "ramp":    # 12.5 higher each 64 keys: 100 in a piece, then on
        return x - 100.0 + 12.5 * (i // 64)
    assert kind == "cliff"  # up by more than fp32 can hold, and down again
    return x + 300.0 * (i % 256 >= 128)


def grown_cache(g, p, kind, lens, t, cache):
    """Pages whose keys give a query near `u` these logits, and normal values."""
    d, HK, page = p.head_dim, p.n_kv_heads, p.page_size
    kc, vc = K.empty_paged(p, int(t.max()) + 1)
    n_pages = kc.data.shape[0]
    u = torch.randint(0, 2, (HK, d), generator=g) * 2.0 - 1.0
    k = torch.zeros(n_pages, HK, page, d)
    v = normal(g, n_pages, HK, page, d)
    for s, n in enumerate(lens):
        i = torch.arange(n)
        for h in range(HK):
            rows = u[h] * (growth(kind, n, g) * LN2 / d).float()[:, None] + 0.002 * normal(g, n, d)
            k[t[s, i // page].long(), h, i % page] = rows
    for c, x in ((kc, k), (vc, v)):
        x = x.cuda().view(-1, d)
        K.csa_quantize(x, K.Stored(c.fmt, c.data.view(x.shape[0], -1), None if c.scales is None else c.scales.view(x.shape[0], -1)))
    return kc, vc, u


FORMS = [("bf16", "bf16", 64), ("bf16", "bf16", 128), ("bf16", "bf16", 192), ("bf16", "bf16", 256), ("bf16", "fp8", 64),
         ("bf16", "fp8", 128), ("bf16", "fp8", 192), ("bf16", "fp8", 256), ("f32", "f32", 64), ("f32", "bf16", 128),
         ("f32", "fp8", 64), ("f32", "fp8", 256)]


def over_all(p, q, kc, vc, t, lens, sinks, act, cache, what):
    """The call on the whole batch against every row's own 64-bit form."""
    n, (H, d) = len(lens), q.shape[1:]
    out = torch.full((n, H, d), float("nan"), dtype=DT[act], device="cuda")
    ws = torch.empty(K.gqa_workspace_size(p, K.OP_PAGED_DECODE, n, n, t.shape[1] * p.page_size), dtype=torch.uint8, device="cuda")
    K.paged_decode_attn(p, n, q.cuda(), kc, vc, t.cuda(), torch.tensor(lens).cuda() - 1, None if sinks is None else sinks.cuda(), out, ws)
    assert clean() == 0
    refs = []
    for b, m in enumerate(lens):
        k, v = (paged_rows(c, t[b], m, p.page_size) for c in (kc, vc))
        vs = scale_rows(vc, t[b], m, p.page_size) if cache == "fp8" else None
        refs.append(attend_paged(q[b:b + 1].double(), k, v, vs, p.scale, sinks, act, cache))
    assert_within(out, torch.cat([r for r, _ in refs]), torch.cat([e for _, e in refs]), what)
    return out


@pytest.mark.parametrize("flags", [0, K.FLAG_BATCH_INVARIANT], ids=["", "invariant"])
@pytest.mark.parametrize("kind", ["shelf", "saw", "ramp", "cliff"])
@pytest.mark.parametrize("act,cache,d", FORMS)
def test_decode_of_logits_that_grow_along_the_row(act, cache, d, kind, flags):
    """The running maximum is raised after a warp's first tile, by what fp32 holds and by more: the sums and the output so
    far, and the units of FP8 products, follow.  Rows within one block and rows joined from several, with and without sinks."""
    g, _ = gen(81), clean()
    HK, G = (8, 2) if d == 64 else (4, 3)
    lens = [600, 1100, 64, 513, 200, 2300, 130, 17] + [600] * 24
    p = make(HK * G, HK, d, act, cache, page_size=16, scale=1.0, flags=flags)
    held = [-(-n // 16) for n in lens]
    t = table_of(g, held, max(held))
    kc, vc, u = grown_cache(g, p, kind, lens, t, cache)
    q = (u.repeat_interleave(G, 0) * (1 + 0.02 * normal(g, len(lens), HK * G, d))).to(DT[act])
    sinks = normal(g, HK * G) * 5 if kind in ("shelf", "ramp") else None
    over_all(p, q, kc, vc, t, lens, sinks, act, cache, kind)


def test_the_growing_logits_raise_the_maximum_after_a_first_tile():
    """What the test above is for: in every kind, tiles that a warp takes later exceed its earlier ones by more than the 8
    log2 units up to which the maximum stays, by amounts that fp32's exponential holds and, in one, by more."""
    g = gen(82)
    for kind in ("shelf", "saw", "ramp", "cliff"):
        for step, tok in ((64, 16), (32, 8)):
            x = growth(kind, 512, g).view(512 // step, step // tok, tok).amax(2)   # [step][warp]
            for w in range(x.shape[1]):
                m, held, gone = x[0, w], 0, 0
                for y in x[1:, w]:
                    if y > m + 8:
                        held, gone, m = held + (y - m < 120), gone + (y - m >= 126), y
                assert (held >= 1) if kind != "cliff" else (gone >= 1), kind


SPREADS = ["rising", "falling", "groups", "any", "far"]


def spread_scales(kind, shape, g):
    """Scales [n][HK][d/64] as powers of two times 1..2, over the range that the documentation gives (values within 2^100)."""
    n, HK, groups = shape
    i = torch.arange(n, dtype=torch.float64)[:, None, None]
    one = torch.ones(shape, dtype=torch.float64)
    e = {"rising": -60 + 120 * i / n, "falling": 60 - 120 * i / n,
         "groups": one * 40 * (1 - 2 * (torch.arange(groups) % 2)),
         "any": torch.randint(-40, 41, shape, generator=g).double(),
         "far": torch.where(i % 7 == 3, 90.0, -90.0)}[kind]
    return torch.exp2(e * one) * (1 + torch.rand(shape, generator=g, dtype=torch.float64))


@pytest.mark.parametrize("flags", [0, K.FLAG_BATCH_INVARIANT], ids=["", "invariant"])
@pytest.mark.parametrize("kind", SPREADS)
@pytest.mark.parametrize("act,d", [("bf16", 64), ("bf16", 128), ("bf16", 192), ("bf16", 256), ("f32", 64), ("f32", 192)])
def test_decode_of_fp8_scales_over_many_powers_of_two(act, d, kind, flags):
    """Value scales that rise and fall along the row, differ between the groups of 64 channels or jump by 2^180; key scales
    over 2^20."""
    g, _ = gen(83), clean()
    HK, G = (2, 4) if d != 64 else (1, 16)
    lens = [700, 1500, 40, 16, 260, 1, 513, 90]
    p = make(HK * G, HK, d, act, "fp8", page_size=16, flags=flags)
    held = [-(-n // 16) for n in lens]
    t = table_of(g, held, max(held))
    kc, vc = K.empty_paged(p, sum(held))
    for c in (kc, vc):
        codes = torch.randint(0, 127, c.data.shape, generator=g)                   # 127 is NaN
        c.data.copy_((codes + 128 * torch.randint(0, 2, c.data.shape, generator=g)).to(torch.uint8))
        c.scales.fill_(1.0)
    kscale, vscale = torch.ones(kc.scales.shape), torch.ones(vc.scales.shape)
    for s, n in enumerate(lens):
        i = torch.arange(n)
        at = (t[s, i // 16].long(), slice(None), i % 16)
        # (codes are as likely in every binade: |k| is up to 448 and mostly far less)
        kscale[at] = torch.exp2(-7 - 20 * torch.rand(n, HK, d // 64, generator=g))
        vscale[at] = spread_scales(kind, (n, HK, d // 64), g).float()
    kc.scales.copy_(kscale), vc.scales.copy_(vscale)
    q = normal(g, len(lens), HK * G, d, dt=DT[act])
    for sinks in (None, normal(g, HK * G)):
        over_all(p, q, kc, vc, t, lens, sinks, act, "fp8", kind)


@pytest.mark.parametrize("d,H,HK,lens", [(128, 32, 8, [1, 16, 17, 300, 2049]), (64, 6, 2, [1, 7, 8, 400]), (256, 12, 1, [1, 500, 63]),
                                         (192, 9, 3, [33, 800]), (128, 16, 1, [9000, 5])])
def test_decode_over_fp8_pages_rounds_probabilities_to_f16(d, H, HK, lens):
    """Normal keys and values at the kernel's own rounding: P to f16, entries exactly as they are stored."""
    g, _ = gen(84), clean()
    p = make(H, HK, d, "bf16", "fp8", page_size=16)
    held = [-(-n // 16) for n in lens]
    t = table_of(g, held, max(held))
    kc, vc = K.empty_paged(p, sum(held))
    for c in (kc, vc):
        x = normal(g, sum(held) * HK * 16, d).cuda()
        K.csa_quantize(x, K.Stored(c.fmt, c.data.view(x.shape[0], -1), c.scales.view(x.shape[0], -1)))
    over_all(p, normal(g, len(lens), H, d, dt=torch.bfloat16), kc, vc, t, lens, None, "bf16", "fp8", "f16")


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("act,H,HK,d", [("bf16", 4, 2, 64), ("bf16", 3, 1, 64), ("bf16", 4, 2, 128), ("bf16", 2, 1, 192), ("bf16", 7, 1, 192),
                                        ("bf16", 4, 2, 256), ("f32", 2, 1, 64), ("f32", 2, 1, 192), ("f32", 2, 2, 256)])
def test_prompt_values_that_are_no_numbers_at_every_head_dim(act, H, HK, d, window):
    """Values with infinities and NaN in several groups of channels, at keys all over the tiles: they come out in the channels
    where they are, in the rows that see them, as the formula has it, and nowhere else."""
    g, _ = gen(85), clean()
    lq = lk = [20, 330, 40]
    wide, kv, cq, ck = prompt_data(g, act, H, HK, d, lq, lk)
    p = make(H, HK, d, act, window=window)
    q, (k, v) = wide[:, :H * d].unflatten(1, (H, d)).contiguous(), (x.unflatten(1, (HK, d)).contiguous() for x in kv.split(HK * d, 1))
    v = v.clone()
    bad = {}                                             # (sequence, key, head, channel): value
    for key, value in ((3, float("inf")), (63, float("nan")), (64, float("-inf")), (65, float("inf")), (127, float("-inf")),
                       (200, float("inf")), (255, float("nan")), (328, float("inf")), (329, float("-inf"))):
        for c in range(key % 8, d, 64):                  # one channel of each group, others for other keys
            bad[1, key, key % HK, c] = value
    bad[0, 19, 0, 5] = bad[2, 0, HK - 1, d - 1] = float("inf")
    clear = v.clone()
    for (s, key, h, c), value in bad.items():
        v[int(ck[s]) + key, h, c], clear[int(ck[s]) + key, h, c] = value, 0.0
    ref, tol = prompt_reference(p, q, k, clear, cq, ck, None, act)
    G, want = H // HK, {}
    for (s, key, h, c), value in bad.items():
        for i in range(key, min(lq[s], key + window if window else lq[s])):
            for x in range(h * G, (h + 1) * G):
                at = (int(cq[s]) + i, x, c)
                want[at] = want.get(at, 0.0) + value
    out = run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, None, act).cpu()
    n = int(cq[-1])
    assert clean() == 0
    keep = torch.ones(out.shape, dtype=torch.bool)
    for at, value in want.items():
        keep[at] = False
        assert (math.isnan(value) and math.isnan(out[at])) or float(out[at]) == value, (at, value, out[at])
    keep[n:] = False
    assert_within(out[keep], ref[keep], tol[keep], "others")


@pytest.mark.parametrize("act,H,HK,d", [("bf16", 4, 1, 64), ("bf16", 2, 2, 128), ("bf16", 3, 1, 192), ("bf16", 4, 2, 256), ("f32", 2, 1, 64),
                                        ("f32", 2, 1, 128), ("f32", 2, 1, 256)])
@pytest.mark.parametrize("kind", ["shelf", "ramp", "cliff"])
def test_prompt_of_logits_that_grow_along_the_keys(act, H, HK, d, kind):
    """As for the decode: every row's maximum is raised several times, at each head dim's own tiles."""
    g, _ = gen(86), clean()
    n = [520, 300, 33]
    wide, kv, cq, ck = prompt_data(g, act, H, HK, d, n, n)
    p = make(H, HK, d, act, scale=1.0)
    u = torch.randint(0, 2, (HK, d), generator=g) * 2.0 - 1.0
    k, v = (x.unflatten(1, (HK, d)).clone() for x in kv.split(HK * d, 1))
    for s, m in enumerate(n):
        rows = (growth(kind, m, g) * LN2 / d).float()[:, None, None] * u + 0.002 * normal(g, m, HK, d)
        k[int(ck[s]):int(ck[s + 1])] = rows.to(DT[act])
    q = (u.repeat_interleave(H // HK, 0) * (1 + 0.02 * normal(g, wide.shape[0], H, d))).to(DT[act])
    sinks = normal(g, H) * 5 if kind != "cliff" else None
    ref, tol = prompt_reference(p, q, k, v, cq, ck, sinks, act)
    out = run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, sinks, act)
    m = int(cq[-1])
    assert clean() == 0
    assert_within(out[:m], ref[:m], tol[:m], kind)


@pytest.mark.parametrize("act,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 192), ("f32", 256)])
@pytest.mark.parametrize("one", [False, True], ids=["packed", "single"])
def test_append_quantises_as_csa_quantize_does(act, d, one):
    """Rows that are not rotated: the same codes and scales bit for bit, for values of any size and for those that are no
    numbers.  One difference is documented: a group so small that its scale is 0 in fp32 is stored as zeros with scale 1."""
    g, _ = gen(87), clean()
    n, HK, page = 600, 3, 16
    p = make(3, HK, d, act, "fp8", page_size=page)
    x = normal(g, 2, n, HK, d) * torch.exp2(torch.randint(-30, 31, (2, n, HK, 1), generator=g).float())
    x[:, 1] = 0.0
    x[:, 2] *= 1e-38                                     # scales that leave the normal range
    x[:, 3] = torch.exp2(torch.randint(-149, -120, (2, HK, d), generator=g).double()).float()
    x[:, 4] = 3e38
    x[:, 5] = torch.exp2(torch.randint(-9, 1, (2, HK, d), generator=g).float()) * (1 + torch.randint(0, 8, (2, HK, d), generator=g) / 16)
    for i, bad in ((6, float("nan")), (7, float("inf")), (8, float("-inf"))):
        x[:, i, :, i::64] = bad
    x = x.to(DT[act]).cuda()
    pages = -(-n // page) if not one else n
    kc, vc = K.empty_paged(p, pages)
    pos, cu = (torch.zeros(n, dtype=torch.int64), None) if one else (torch.zeros(1, dtype=torch.int64), torch.tensor([0, n], dtype=torch.int32).cuda())
    t = torch.arange(pages, dtype=torch.int32).view(n, 1) if one else torch.arange(pages, dtype=torch.int32)[None]
    K.paged_append(p, len(pos), n, cu, pos.cuda(), None, x[0], x[1], None, None, None, kc, vc, t.cuda())
    i = torch.arange(n)
    at = (i, slice(None), 0 * i) if one else (i // page, slice(None), i % page)
    for c, y in ((kc, x[0]), (vc, x[1])):
        want = K.empty_stored(K.FP8_S64, n * HK, d)
        K.csa_quantize(y.float().reshape(-1, d), want)
        codes, scales = want.data.view(n, HK, -1, 64), want.scales.view(n, HK, -1)
        none = scales == 0        # amax / 448 underflows: here the group counts as one of zeros
        scales = torch.where(none, 1.0, scales)
        assert torch.equal(c.scales[at].view(torch.int32), scales.view(torch.int32))
        got = c.data[at].unflatten(-1, (-1, 64))
        assert torch.equal(got[~none], codes[~none]) and not (got[none] & 0x7F).any()
    assert clean() == 0
