"""Grouped-head attention on the GPU against plain 64-bit forms: appending to the
paged cache, one new token over it, packed prompts, and the three together."""
import pytest
import torch

import compressed_sparse_attention_13_b200 as K
from compressed_sparse_attention_13_b200.paged import PagedLayer
from gqa_reference import HALF, assert_within, attend, causal, paged_rows, partner, rotate

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FMT = {"bf16": K.BF16, "f32": K.F32, "fp8": K.FP8_S64}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dt=torch.float32):
    return torch.randn(*shape, generator=g).to(dt)


def make(H, HK, d, act="bf16", cache=None, **kw):
    return K.gqa_params(H, HK, d, kw.pop("scale", d ** -0.5), act_fmt=FMT[act], cache_fmt=FMT[cache or act], **kw)


def clean():
    return K.csa_device_status(reset=True)


def table_of(g, held, per):
    """Block tables of sequences that hold held[i] pages each, in a random order."""
    order = torch.randperm(sum(held), generator=g).to(torch.int32)
    t, at = torch.full((len(held), per), -1, dtype=torch.int32), 0
    for i, h in enumerate(held):
        t[i, :h] = order[at:at + h]
        at += h
    return t


# ------------------------------------------------------------------ append
APPEND = [
    # act, cache, H, HK, d, page, rot, pairs, lens (None: one token each), starts, strided
    ("bf16", "bf16", 8, 2, 128, 16, 128, False, [5, 0, 33, 1], [0, 7, 100, 15], True),
    ("bf16", "fp8", 6, 3, 128, 8, 64, True, [17, 40], [3, 0], False),
    ("bf16", "f32", 4, 4, 64, 5, 16, False, [9], [1048560], False),
    ("f32", "f32", 4, 1, 256, 16, 256, False, [3, 20], [131071, 2], True),
    ("f32", "bf16", 7, 7, 192, 1, 96, True, [6, 1], [0, 3], False),
    ("f32", "fp8", 2, 2, 192, 64, 192, False, [70], [60], False),
    ("bf16", "bf16", 32, 8, 128, 16, 0, False, None, [0, 15, 16, 4095, -1, 77], False),
    ("bf16", "fp8", 16, 1, 64, 16, 64, True, None, [9, -1, 0], True),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[0]}-{c[1]}-d{c[4]}-r{c[6]}")
def test_append(case):
    act, cache, H, HK, d, page, rot, pairs, lens, starts, strided = case
    g, clean0 = gen(7), clean()
    one = lens is None
    ls = [1] * len(starts) if one else lens
    n, extra = sum(ls), 0 if one else 3
    N = n + extra
    held = [max(0, -(-(a + b) // page)) if a >= 0 else 0 for a, b in zip(starts, ls)]
    far = max(starts) > 100000
    if far:  # only the pages that are written exist: the others are not resident
        held = [(-(-(a + b) // page) - a // page) if a > 1000 else h for a, b, h in zip(starts, ls, held)]
    per = max(-(-(max(a, 0) + b) // page) for a, b in zip(starts, ls)) + 1
    pages = sum(held) + 2
    if far:
        t, at = torch.full((len(ls), per), -1, dtype=torch.int32), 0
        for i, (a, h) in enumerate(zip(starts, held)):
            f = a // page if a > 1000 else 0
            t[i, f:f + h] = torch.arange(at, at + h, dtype=torch.int32)
            at += h
    else:
        t = table_of(g, held, per)
    p = make(H, HK, d, act, cache, page_size=page, rot_dim=rot, flags=K.FLAG_ROT_PAIRS if pairs else 0)
    wide = normal(g, N, (H + 2 * HK) * d + (8 if strided else 0), dt=DT[act])
    q, k, v = (x.unflatten(1, (-1, d)) for x in wide[:, :(H + 2 * HK) * d].split([H * d, HK * d, HK * d], 1))
    dev = wide.cuda()
    qd, kd, vd = (x.unflatten(1, (-1, d)) for x in dev[:, :(H + 2 * HK) * d].split([H * d, HK * d, HK * d], 1))
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    kc, vc = K.empty_paged(p, pages)
    for c in (kc, vc):
        c.data.view(torch.uint8).fill_(0x55)
        if c.scales is not None:
            c.scales.fill_(7.0)
    before = [c.data.clone() for c in (kc, vc)]
    qo, ko = torch.full((N, H, d), 5.0, dtype=DT[act], device="cuda"), torch.full((N, HK, d), 5.0, dtype=DT[act], device="cuda")
    cu = [0]
    for m in ls:
        cu.append(cu[-1] + m)
    K.paged_append(p, len(ls), N, None if one else torch.tensor(cu, dtype=torch.int32).cuda(),
                   torch.tensor(starts, dtype=torch.int64).cuda(), qd, kd, vd, f.cuda(), qo, ko, kc, vc, t.cuda())
    torch.cuda.synchronize()
    assert clean() == 0
    written = [torch.zeros(c.data.shape[:3], dtype=torch.bool) for c in (kc, vc)]
    u = HALF[DT[act]]
    for s, (a, m) in enumerate(zip(starts, ls)):
        sl = slice(cu[s], cu[s + 1])
        if a < 0:
            assert (qo[sl] == 5).all() and (ko[sl] == 5).all()
            continue
        if m == 0:
            continue
        pos = torch.arange(a, a + m)
        # fp32 cosines, two products and a sum: 2^-22 of |a| + |b|; the angle's own rounding, |turn| 2^-24, is in it
        for got, x, lab in ((qo[sl], q[sl], "q"), (ko[sl], k[sl], "k")):
            ref = rotate(x.double(), pos, f, rot, pairs)
            assert_within(got, ref, u * ref.abs() + 2.0 ** -21 * partner(x.double(), rot, pairs), lab)
        ids, off = t[s, pos // page].long(), pos % page
        for c, x, w, rotated in ((kc, k[sl], written[0], True), (vc, v[sl], written[1], False)):
            ref = rotate(x.double(), pos, f, rot, pairs) if rotated else x.double()
            err = 2.0 ** -21 * partner(x.double(), rot if rotated else 0, pairs)
            rows = c.data.cpu()[ids, :, off]
            w[ids, :, off] = True
            if cache == "fp8":
                sc = c.scales.cpu()[ids, :, off].double()
                top = ref.unflatten(-1, (-1, 64)).abs().amax(-1)
                assert ((sc - top / 448).abs() <= 2.0 ** -20 * top / 448 + err.unflatten(-1, (-1, 64)).amax(-1) / 448).all()
                val = rows.view(torch.float8_e4m3fn).double() * sc.repeat_interleave(64, -1)
                assert_within(val, ref, 2.0 ** -4 * ref.abs() * (1 + 2.0 ** -18) + sc.repeat_interleave(64, -1) * 2.0 ** -10 + 2 * err, "fp8")
            else:
                assert_within(rows, ref, HALF[rows.dtype] * ref.abs() + err, "cache")
    if extra:
        assert (qo[n:] == 5).all() and (ko[n:] == 5).all()
    for c, b, w in zip((kc, vc), before, written):
        assert torch.equal(c.data.cpu()[~w].view(torch.uint8), b.cpu()[~w].view(torch.uint8)), "another row was written"


def test_append_in_place_and_without_queries():
    p, g = make(4, 2, 64, page_size=16, rot_dim=64), gen(3)
    q, k, v = normal(g, 6, 4, 64, dt=torch.bfloat16).cuda(), normal(g, 6, 2, 64, dt=torch.bfloat16).cuda(), normal(g, 6, 2, 64, dt=torch.bfloat16).cuda()
    f = (100.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).cuda()
    pos, t = torch.arange(6, dtype=torch.int64).cuda() * 3, torch.arange(6, dtype=torch.int32).view(6, 1).cuda()
    t2 = torch.cat([t, t + 6], 1)[:, :2].contiguous()
    outs = []
    for in_place in (False, True):
        kc, vc = K.empty_paged(p, 12)
        kc.data.zero_(), vc.data.zero_()
        a, b = (q.clone(), k.clone())
        qo, ko = (a, b) if in_place else (torch.empty_like(a), torch.empty_like(b))
        K.paged_append(p, 6, 6, None, pos, a, b, v, f, qo, ko, kc, vc, t2)
        outs.append((qo, ko, kc.data, vc.data))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    kc, vc = K.empty_paged(p, 12)
    kc.data.zero_(), vc.data.zero_()
    K.paged_append(p, 6, 6, None, pos, None, k, v, f, None, None, kc, vc, t2)
    assert torch.equal(kc.data, outs[0][2]) and torch.equal(vc.data, outs[0][3])


@pytest.mark.parametrize("bad", [-1, 4, 2 ** 31 - 1, -2 ** 31])
def test_bad_pages_are_flagged_and_skipped(bad):
    clean()
    p, g = make(2, 1, 64, page_size=4), gen(4)
    kc, vc = K.empty_paged(p, 4)
    kc.data.zero_(), vc.data.zero_()
    x = normal(g, 8, 1, 64, dt=torch.bfloat16).cuda()
    t = torch.tensor([[2, bad]], dtype=torch.int32).cuda()
    cu, pos0 = torch.tensor([0, 8], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int64).cuda()
    K.paged_append(p, 1, 8, cu, pos0, None, x, x, None, None, None, kc, vc, t)
    assert clean() == K.DEV_BAD_INDEX
    assert torch.equal(kc.data[2, 0], x[:4, 0]) and not kc.data[[0, 1, 3]].any()
    q = normal(g, 1, 2, 64, dt=torch.bfloat16).cuda()
    out, ws = torch.empty_like(q), torch.empty(K.gqa_workspace_size(p, K.OP_PAGED_DECODE, 1, 1, 8), dtype=torch.uint8, device="cuda")
    for pos in (7, 2 ** 40):  # the bad page's tokens, or all past the table, are left out
        K.paged_decode_attn(p, 1, q, kc, vc, t, torch.tensor([pos]).cuda(), None, out, ws)
        assert clean() == K.DEV_BAD_INDEX
        ref, tol = attend(q.cpu().double(), x[:4].cpu().double(), x[:4].cpu().double(), 0.125, torch.ones(1, 4, dtype=torch.bool), None,
                          torch.bfloat16, 2.0 ** -8)
        assert_within(out, ref, tol, "bad page")


# ------------------------------------------------------------------ decode
DECODE = [
    # act, cache, H, HK, d, page, window, sink, lens
    ("bf16", "bf16", 32, 8, 128, 16, 0, False, [1, 2, 15, 16, 17, 31, 33, 64, 100, 1001]),
    ("bf16", "bf16", 8, 8, 64, 16, 0, True, [0, 5, 513, 0, 4097]),
    ("bf16", "bf16", 7, 1, 128, 100, 0, True, [1, 99, 100, 101, 2000]),
    ("bf16", "bf16", 16, 1, 256, 8, 128, True, [1, 127, 128, 129, 700]),
    ("bf16", "bf16", 48, 3, 192, 64, 0, False, [65, 1, 1333]),
    ("bf16", "bf16", 64, 1, 64, 1, 33, False, [1, 33, 34, 500]),
    ("bf16", "bf16", 20, 1, 128, 24, 1, True, [1, 24, 1000]),
    ("bf16", "bf16", 128, 1, 64, 16, 0, False, [77, 300]),
    ("bf16", "fp8", 32, 8, 128, 16, 0, False, [1, 16, 17, 300, 2049]),
    ("bf16", "fp8", 6, 2, 64, 7, 50, True, [1, 7, 8, 400, 0]),
    ("bf16", "fp8", 12, 1, 256, 64, 0, True, [1, 500, 63]),
    ("bf16", "fp8", 9, 3, 192, 16, 0, False, [33, 800]),
    ("bf16", "f32", 4, 2, 128, 16, 0, False, [3, 200]),
    ("f32", "f32", 8, 8, 64, 16, 128, True, [1, 2, 60, 127, 128, 900, 5000, 0]),
    ("f32", "f32", 16, 2, 128, 32, 0, False, [1, 700, 33]),
    ("f32", "f32", 5, 1, 256, 16, 0, True, [250, 17]),
    ("f32", "f32", 6, 2, 192, 10, 0, False, [250, 9]),
    ("f32", "bf16", 8, 1, 128, 16, 0, False, [500, 1]),
    ("f32", "fp8", 4, 1, 64, 16, 0, True, [310, 15]),
]


def fill_cache(g, p, held_pages, cache):
    """A paged cache with normal values; the raw tensors are on the device."""
    kc, vc = K.empty_paged(p, held_pages)
    for c in (kc, vc):
        x = normal(g, held_pages * p.n_kv_heads * p.page_size, p.head_dim).cuda()
        st = K.Stored(c.fmt, c.data.view(x.shape[0], -1), None if c.scales is None else c.scales.view(x.shape[0], -1))
        K.csa_quantize(x, st)
    return kc, vc


def decode_reference(p, q, kc, vc, t, lens, sinks, act, cache):
    outs, tols = [], []
    # 8-bit entries take part as they are or scaled and rounded once more to 16 bits: one more half step on each product
    half = 0.0 if act == "f32" or cache == "f32" else 2.0 ** -8 if cache == "bf16" else 3 * 2.0 ** -8
    for b, n in enumerate(lens):
        k, v = (paged_rows(c, t[b], n, p.page_size) for c in (kc, vc))
        see = causal(1, n, p.window) if n else torch.zeros(1, 0, dtype=torch.bool)
        o, e = attend(q[b:b + 1].cpu().double(), k, v, p.scale, see, sinks, DT[act], half)
        outs.append(o)
        tols.append(e)
    return torch.cat(outs), torch.cat(tols)


@pytest.mark.parametrize("flags", [0, K.FLAG_BATCH_INVARIANT], ids=["", "invariant"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{c[0]}-{c[1]}-H{c[2]}x{c[3]}-d{c[4]}-p{c[5]}-w{c[6]}")
def test_decode(case, flags):
    act, cache, H, HK, d, page, window, sink, lens = case
    g, _ = gen(11), clean()
    p = make(H, HK, d, act, cache, page_size=page, window=window, flags=flags)
    held = [-(-n // page) for n in lens]
    per = max(held) + 1
    t = table_of(g, held, per)
    kc, vc = fill_cache(g, p, sum(held), cache)
    wide = normal(g, len(lens), H * d + 16, dt=DT[act])
    dev = wide.cuda()
    q = dev[:, :H * d].unflatten(1, (H, d))   # strided rows
    sinks = normal(g, H) if sink else None
    ref, tol = decode_reference(p, q, kc, vc, t, lens, sinks, act, cache)
    # rows behind a sequence's last token hold what nobody may see: NaN
    for b, n in enumerate(lens):
        if n % page:
            last = int(t[b, n // page])
            for c in (kc, vc):
                if c.scales is not None:
                    c.data[last, :, n % page:] = 0x7F
                    c.scales[last, :, n % page:] = float("inf")
                else:
                    c.data[last, :, n % page:] = float("nan")
    out = torch.full((len(lens), H, d), float("nan"), dtype=DT[act], device="cuda")
    ws = torch.full((K.gqa_workspace_size(p, K.OP_PAGED_DECODE, len(lens), len(lens), per * page),), 0xFF, dtype=torch.uint8, device="cuda")
    pos = torch.tensor(lens, dtype=torch.int64).cuda() - 1
    for _ in range(2):  # the second call finds the first one's workspace
        K.paged_decode_attn(p, len(lens), q, kc, vc, t.cuda(), pos, None if sinks is None else sinks.cuda(), out, ws)
        assert clean() == 0
        assert_within(out, ref, tol, "decode")


def test_decode_sees_nothing_before_the_window_and_nothing_of_other_pages():
    """Entries that are out of the window, NaN and infinities among them, do not reach the output."""
    p, g = make(4, 2, 128, page_size=8, window=20), gen(5)
    t = table_of(g, [12], 12)
    kc, vc = fill_cache(g, p, 12, "bf16")
    q = normal(g, 1, 4, 128, dt=torch.bfloat16).cuda()
    ref, tol = decode_reference(p, q, kc, vc, t, [90], None, "bf16", "bf16")
    for c in (kc, vc):
        c.data[t[0, :8].long().cuda()] = float("nan")            # tokens 0..63
        c.data[int(t[0, 8]), :, :6] = float("inf")               # tokens 64..69: 70 is the first visible one
        c.data[int(t[0, 11]), :, 2:] = float("-inf")             # tokens 90..
    out, ws = torch.empty_like(q), torch.empty(K.gqa_workspace_size(p, K.OP_PAGED_DECODE, 1, 1, 96), dtype=torch.uint8, device="cuda")
    K.paged_decode_attn(p, 1, q, kc, vc, t.cuda(), torch.tensor([89]).cuda(), None, out, ws)
    assert_within(out, ref, tol, "window")


@pytest.mark.parametrize("act,cache", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32")])
def test_decode_is_the_same_in_every_batch_when_asked(act, cache):
    """CSA_FLAG_BATCH_INVARIANT: a row's bits do not depend on the other rows; both modes repeat bit for bit."""
    p, g = make(8, 2, 128, act, cache, page_size=16, flags=K.FLAG_BATCH_INVARIANT), gen(6)
    lens = [3000, 1, 700, 9000, 16, 4500, 128, 2500]
    held = [-(-n // 16) for n in lens]
    t = table_of(g, held, max(held))
    kc, vc = fill_cache(g, p, sum(held), cache)
    q = normal(g, len(lens), 8, 128, dt=DT[act]).cuda()

    def go(rows, flags):
        p.flags = flags
        n = len(rows)
        ws = torch.empty(K.gqa_workspace_size(p, K.OP_PAGED_DECODE, n, n, max(held) * 16), dtype=torch.uint8, device="cuda")
        out = torch.empty(n, 8, 128, dtype=DT[act], device="cuda")
        K.paged_decode_attn(p, n, q[rows].contiguous(), kc, vc, t[rows].contiguous().cuda(), torch.tensor([lens[r] - 1 for r in rows]).cuda(),
                            None, out, ws)
        return out

    every = go(list(range(8)), K.FLAG_BATCH_INVARIANT)
    for rows in ([0], [3], [5, 2], [7, 6, 5, 4, 3, 2, 1, 0], [3] * 40):
        assert torch.equal(go(rows, K.FLAG_BATCH_INVARIANT), every[rows])
    assert torch.equal(go(list(range(8)), 0), go(list(range(8)), 0))


def test_decode_reaches_rows_past_32_bit_offsets():
    """A cache of more than 2^32 elements, of which the last pages are used."""
    clean()
    n_pages = 2 ** 32 // (8 * 16 * 128) + 10
    p, g = make(32, 8, 128, page_size=16), gen(8)
    kc, vc = K.empty_paged(p, n_pages)
    t = torch.tensor([[n_pages - 1, 3, n_pages - 7, n_pages - 2]], dtype=torch.int32)
    x = normal(g, 2, 50, 8, 128, dt=torch.bfloat16)
    cu, pos0 = torch.tensor([0, 50], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int64).cuda()
    K.paged_append(p, 1, 50, cu, pos0, None, x[0].cuda(), x[1].cuda(), None, None, None, kc, vc, t.cuda())
    q = normal(g, 1, 32, 128, dt=torch.bfloat16).cuda()
    out, ws = torch.empty_like(q), torch.empty(K.gqa_workspace_size(p, K.OP_PAGED_DECODE, 1, 1, 64), dtype=torch.uint8, device="cuda")
    K.paged_decode_attn(p, 1, q, kc, vc, t.cuda(), torch.tensor([49]).cuda(), None, out, ws)
    assert clean() == 0
    ref, tol = attend(q.cpu().double(), x[0].double(), x[1].double(), p.scale, causal(1, 50, 0), None, torch.bfloat16, 2.0 ** -8)
    assert_within(out, ref, tol, "far pages")


# ------------------------------------------------------------------ prompt
PROMPT = [
    # act, H, HK, d, window, sink, lens_q, lens_k (None: the same)
    ("bf16", 8, 2, 64, 0, False, [1, 17, 64, 200], None),
    ("bf16", 8, 2, 128, 0, True, [128, 129, 127, 1, 0, 300], None),
    ("bf16", 4, 4, 128, 0, False, [255, 256, 257, 513], None),
    ("bf16", 7, 1, 128, 40, True, [100, 333], None),
    ("bf16", 6, 2, 192, 0, True, [65, 200], None),
    ("bf16", 4, 1, 256, 0, False, [130, 31, 260], None),
    ("bf16", 16, 1, 256, 100, True, [90, 210], None),
    ("bf16", 32, 1, 64, 1, False, [1, 70], None),
    ("bf16", 128, 1, 64, 0, False, [33], None),
    ("bf16", 100, 1, 64, 0, True, [40, 3], None),
    ("bf16", 8, 2, 128, 0, False, [20, 1, 60, 5, 9], [500, 129, 60, 3, 0]),   # later chunks; fewer keys than queries; none
    ("bf16", 4, 4, 64, 64, True, [200, 300], [250, 120]),
    ("bf16", 4, 2, 128, 256, False, [1000], None),
    ("f32", 8, 8, 64, 0, False, [1, 64, 65, 200], None),
    ("f32", 4, 2, 128, 50, True, [100, 33, 129], None),
    ("f32", 3, 1, 256, 0, False, [70], None),
    ("f32", 4, 2, 192, 0, True, [66, 7], [100, 5]),
]


def prompt_data(g, act, H, HK, d, lq, lk, pad=5):
    nq, nk = sum(lq) + pad, sum(lk) + pad
    wide = normal(g, nq, H * d + 8, dt=DT[act])
    kv = normal(g, nk, 2 * HK * d, dt=DT[act])
    cu = [torch.tensor([sum(x[:i]) for i in range(len(x) + 1)], dtype=torch.int32) for x in (lq, lk)]
    return wide, kv, *cu


def prompt_reference(p, q, k, v, cq, ck, sinks, act):
    H, d = q.shape[1:]
    out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for s in range(len(cq) - 1):
        a, b, c, e = int(cq[s]), int(cq[s + 1]), int(ck[s]), int(ck[s + 1])
        out[a:b], tol[a:b] = attend(q[a:b].double(), k[c:e].double(), v[c:e].double(), p.scale, causal(b - a, e - c, p.window), sinks,
                                    DT[act], 0.0 if act == "f32" else 2.0 ** -8)
    return out, tol


def run_prompt(p, q, k, v, cq, ck, sinks, act, out=None, stream=None):
    n = len(cq) - 1
    out = torch.full(q.shape, 9.0, dtype=DT[act], device="cuda") if out is None else out
    ws = torch.full((K.gqa_workspace_size(p, K.OP_PROMPT_ATTN, n, q.shape[0], 0),), 0xFF, dtype=torch.uint8, device="cuda")
    K.prompt_attn(p, n, q, k, v, cq.cuda(), ck.cuda(), None if sinks is None else sinks.cuda(), out, ws, stream=stream)
    return out


@pytest.mark.parametrize("case", PROMPT, ids=lambda c: f"{c[0]}-H{c[1]}x{c[2]}-d{c[3]}-w{c[4]}-{'k' if c[7] else ''}{c[6][0]}")
def test_prompt(case):
    act, H, HK, d, window, sink, lq, lk = case
    g, _ = gen(21), clean()
    lk_ = lk or lq
    wide, kv, cq, ck = prompt_data(g, act, H, HK, d, lq, lk_)
    p = make(H, HK, d, act, window=window)
    sinks = normal(g, H) if sink else None
    n, m = int(cq[-1]), int(ck[-1])
    wide[n:] = float("nan")   # rows behind the last sequence
    kv[m:] = float("nan")
    q, (k, v) = wide[:, :H * d].unflatten(1, (H, d)), (x.unflatten(1, (HK, d)) for x in kv.split(HK * d, 1))
    wd, kvd = wide.cuda(), kv.cuda()
    qd, (kd, vd) = wd[:, :H * d].unflatten(1, (H, d)), (x.unflatten(1, (HK, d)) for x in kvd.split(HK * d, 1))
    ref, tol = prompt_reference(p, q, k, v, cq, ck, sinks, act)
    out = run_prompt(p, qd, kd, vd, cq, ck, sinks, act)
    assert clean() == 0
    assert_within(out[:n], ref[:n], tol[:n], "prompt")
    assert (out[n:] == 9).all(), "rows behind the last sequence were written"


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window", [0, 90])
def test_prompt_what_a_query_does_not_see_does_not_reach_it(act, bad, window):
    """A token's own non-finite key and value show in the queries that see it and nowhere else."""
    g, at = gen(22), 150
    wide, kv, cq, ck = prompt_data(g, act, 4, 2, 128, [20, 300, 40], [20, 300, 40])
    p = make(4, 2, 128, act, window=window)
    q, k, v = wide[:, :512].unflatten(1, (4, 128)), *(x.unflatten(1, (2, 128)).contiguous() for x in kv.split(256, 1))
    ref, tol = prompt_reference(p, q, k, v, cq, ck, None, act)
    k, v = k.clone(), v.clone()
    k[20 + at, 1, 3], v[20 + at, 0, 7], v[20 + at, 1, 7] = bad, bad, bad
    out = run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, None, act)
    sees = torch.zeros(q.shape[0], dtype=torch.bool)
    sees[20 + at:20 + (min(300, at + window) if window else 300)] = True
    n = int(cq[-1])
    rest = ~sees[:n]
    assert_within(out[:n][rest], ref[:n][rest], tol[:n][rest], "others")
    assert not torch.isfinite(out[:n][sees[:n]][:, 0, 7].float()).any()


def test_prompt_large_logits_and_extreme_sinks():
    """Logits of hundreds (the running maximum rises often), sinks that take all or nothing."""
    g = gen(23)
    wide, kv, cq, ck = prompt_data(g, "bf16", 4, 1, 128, [400], [400])
    p = make(4, 1, 128, scale=1.0)
    q, k, v = wide[:, :512].unflatten(1, (4, 128)), *(x.unflatten(1, (1, 128)).contiguous() for x in kv.split(128, 1))
    k *= torch.linspace(0.1, 4, 405).bfloat16()[:, None, None]
    sinks = torch.tensor([0.0, -1e30, 1e4, float("-inf")])
    ref, tol = prompt_reference(p, q, k, v, cq, ck, sinks, "bf16")
    out = run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, sinks, "bf16")
    assert_within(out[:400], ref[:400], tol[:400], "large")


def test_prompt_many_sequences():
    """More sequences than one warp's search step, most of them short, some empty."""
    g = gen(24)
    lens = [(7 * i) % 23 for i in range(1100)]
    wide, kv, cq, ck = prompt_data(g, "bf16", 4, 2, 64, lens, lens)
    p = make(4, 2, 64)
    q, k, v = wide[:, :256].unflatten(1, (4, 64)), *(x.unflatten(1, (2, 64)).contiguous() for x in kv.split(128, 1))
    ref, tol = prompt_reference(p, q, k, v, cq, ck, None, "bf16")
    out = run_prompt(p, q.cuda(), k.cuda(), v.cuda(), cq, ck, None, "bf16")
    n = int(cq[-1])
    assert_within(out[:n], ref[:n], tol[:n], "many")


def test_prompt_of_a_long_sequence_at_sampled_rows():
    """40,000 tokens: some rows against their own 64-bit value."""
    g, n = gen(25), 40000
    qkv = torch.randn(n, 4, 128, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    q, k, v = qkv[:, :2], qkv[:, 2:3], qkv[:, 3:4]
    p = make(2, 1, 128)
    cu = torch.tensor([0, n], dtype=torch.int32)
    out = run_prompt(p, q, k, v, cu, cu, None, "bf16")
    for i in (0, 1, 127, 128, 4095, 20000, 33333, n - 1):
        ref, tol = attend(q[i:i + 1].cpu().double(), k[:i + 1].cpu().double(), v[:i + 1].cpu().double(), p.scale,
                          torch.ones(1, i + 1, dtype=torch.bool), None, torch.bfloat16, 2.0 ** -8)
        assert_within(out[i:i + 1], ref, tol, f"row {i}")


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("act,cache,d,H,HK", [("f32", "f32", 64, 4, 2), ("bf16", "bf16", 128, 8, 2), ("bf16", "fp8", 128, 8, 1)])
def test_prompts_then_tokens_through_the_paged_layer(act, cache, d, H, HK):
    """Prompts and eight decode steps of three sequences, one of which is released and started anew: each output against
    full attention over the rotated queries and the cache as stored (the rotation itself is tested above)."""
    clean()
    g, page = gen(31), 16
    p = make(H, HK, d, act, cache, page_size=page, rot_dim=d // 2)
    f = (1e6 ** (-torch.arange(0, d // 2, 2, dtype=torch.float64) / (d // 2))).cuda()
    lay = PagedLayer(p, 3, 40, 12, f)
    sinks = normal(g, H)

    def rotated(x, pos):
        kc, vc = K.empty_paged(p, 1)
        o, n = torch.empty_like(x), x.shape[0]
        full = make(x.shape[1], x.shape[1], d, act, cache, page_size=page, rot_dim=d // 2)
        c2 = K.empty_paged(full, n)
        K.paged_append(full, n, n, None, torch.tensor(pos).cuda(), x, x, x, f, o, None, *c2,
                       torch.arange(n, dtype=torch.int32)[:, None].expand(n, 200).contiguous().cuda())
        return o

    def tokens(n):
        return [normal(g, n, h, d, dt=DT[act]).cuda() for h in (H, HK, HK)]

    def check_prompt(lens):
        n = sum(lens)
        q, k, v = tokens(n)
        out = torch.empty_like(q)
        lay.prefill(lens, q, k, v, sinks.cuda(), out)
        pos = [i for m in lens for i in range(m)]
        cu = torch.tensor([sum(lens[:i]) for i in range(4)], dtype=torch.int32)
        ref, tol = prompt_reference(p, rotated(q, pos).cpu(), rotated(k, pos).cpu(), v.cpu(), cu, cu, sinks, act)
        assert_within(out, ref, tol, "prompt")

    check_prompt([37, 0, 16])
    for step in range(8):
        if step == 4:
            lay.release(2)
            check_prompt_of = [0, 0, 21]
            lens = lay.lens
            q, k, v = tokens(21)
            out = torch.empty_like(q)
            lay.prefill(check_prompt_of, q, k, v, sinks.cuda(), out)
            assert lay.lens[2] == 21 and lens[0] == 41
        q, k, v = tokens(3)
        out = torch.empty_like(q)
        lay.decode(q, k, v, sinks.cuda(), out)
        pos = [n - 1 for n in lay.lens]
        qr = rotated(q, [max(x, 0) for x in pos])
        ref, tol = decode_reference(p, qr, lay.k_cache, lay.v_cache, lay.table.cpu(), lay.lens, sinks, act, cache)
        assert_within(out, ref, tol, f"step {step}")
    assert clean() == 0 and lay.lens == [45, 0, 25]


def test_decode_steps_replayed_from_a_graph():
    """Two layers with a workspace each, captured once and replayed while the lengths grow; the eager steps give the same bits."""
    p = make(8, 2, 128, page_size=16, rot_dim=128)
    f = (1e4 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).cuda()
    runs = []
    for graphed in (False, True):
        g = gen(33)
        lays = [PagedLayer(p, 4, 64, 16, f) for _ in range(2)]
        lens = [100, 1, 33, 0]
        n = sum(lens)
        for lay in lays:
            q, k, v = (normal(g, n, h, 128, dt=torch.bfloat16).cuda() for h in (8, 2, 2))
            lay.prefill(lens, q, k, v, None, torch.empty_like(q))
        q, k, v = (torch.zeros(4, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))
        outs, rot = [torch.empty_like(q) for _ in lays], [torch.empty_like(q) for _ in lays]

        def steps():
            for lay, o, r in zip(lays, outs, rot):
                lay.step(q, k, v, None, o, r)

        graph = None
        if graphed:
            # captured with no sequence active: nothing is written by the warm-up
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            held = [lay.pos.clone() for lay in lays]
            for lay in lays:
                lay.pos.fill_(-1)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                steps()
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                steps()
            for lay, h in zip(lays, held):
                lay.pos.copy_(h)
        got = []
        for _ in range(20):
            for x, h in ((q, 8), (k, 2), (v, 2)):
                x.copy_(normal(g, 4, h, 128, dt=torch.bfloat16).cuda())
            for lay in lays:
                lay.advance()
            graph.replay() if graph else steps()
            got += [o.clone() for o in outs]
        runs.append(torch.stack(got))
    assert torch.equal(*runs)
    assert (runs[0][:, 3] == 0).all()


def test_two_streams_at_once_with_a_workspace_each():
    g = gen(34)
    p = make(8, 2, 128, page_size=16)
    lens = [3000, 2000, 1]
    held = [-(-n // 16) for n in lens]
    t = table_of(g, held, max(held))
    kc, vc = fill_cache(g, p, sum(held), "bf16")
    qs = [normal(g, 3, 8, 128, dt=torch.bfloat16).cuda() for _ in range(2)]
    pos, td = torch.tensor(lens).cuda() - 1, t.cuda()
    size = K.gqa_workspace_size(p, K.OP_PAGED_DECODE, 3, 3, max(held) * 16)
    want = []
    for q in qs:
        want.append(torch.empty_like(q))
        K.paged_decode_attn(p, 3, q, kc, vc, td, pos, None, want[-1], torch.empty(size, dtype=torch.uint8, device="cuda"))
    streams, ws = [torch.cuda.Stream() for _ in qs], [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in qs]
    got = [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(50):
        for q, s, w, o in zip(qs, streams, ws, got):
            K.paged_decode_attn(p, 3, q, kc, vc, td, pos, None, o, w, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
