"""Grouped-head attention: what the entry points refuse, before any CUDA call
(these run on the CPU, where a CUDA call would fail)."""
import ctypes as C

import pytest
import torch

import compressed_sparse_attention_13_b200 as K

FAKE, ODD = C.c_void_p(0x1000), C.c_void_p(0x1008)


def P(**kw):
    a = dict(n_heads=8, n_kv_heads=2, head_dim=128, scale=0.1, page_size=16)
    a.update(kw)
    return K.gqa_params(**a)


def append(p, n_seq=2, n_tok=5, cu=FAKE, pos0=FAKE, q=FAKE, q_ld=1024, k=FAKE, k_ld=256, v=FAKE, v_ld=256, f=FAKE, qo=FAKE,
           ko=None, kc=FAKE, ks=None, vc=FAKE, vs=None, n_pages=9, table=FAKE, max_pages=4):
    return K.lib().paged_append(C.byref(p), n_seq, n_tok, cu, pos0, q, q_ld, k, k_ld, v, v_ld, f, qo, ko, kc, ks, vc, vs,
                                n_pages, table, max_pages, None)


def decode(p, batch=2, q=FAKE, q_ld=1024, kc=FAKE, ks=None, vc=FAKE, vs=None, n_pages=9, table=FAKE, max_pages=4, pos=FAKE,
           sinks=None, out=FAKE, ws=FAKE, wb=1 << 40):
    return K.lib().paged_decode_attn(C.byref(p), batch, q, q_ld, kc, ks, vc, vs, n_pages, table, max_pages, pos, sinks, out,
                                     ws, wb, None)


def prompt(p, n_seq=2, q=FAKE, q_ld=1024, n_q=9, k=FAKE, k_ld=256, v=FAKE, v_ld=256, n_k=9, cq=FAKE, ck=FAKE, out=FAKE,
           ws=FAKE, wb=1 << 40):
    return K.lib().prompt_attn(C.byref(p), n_seq, q, q_ld, n_q, k, k_ld, v, v_ld, n_k, cq, ck, None, out, ws, wb, None)


BAD_PARAMS = [(dict(n_heads=0), -1), (dict(n_kv_heads=0), -1), (dict(n_kv_heads=3), -1), (dict(head_dim=0), -1),
              (dict(head_dim=96), -1), (dict(head_dim=320), -3), (dict(n_heads=258, n_kv_heads=2), -3), (dict(window=-1), -1),
              (dict(scale=float("nan")), -1), (dict(act_fmt=K.FP8_S64), -1), (dict(flags=0x40), -1),
              (dict(flags=K.FLAG_QI_BF16), -1)]


@pytest.mark.parametrize("kw,want", BAD_PARAMS)
def test_bad_parameters(kw, want):
    p = P(**kw)
    big = dict(q_ld=1 << 20)
    assert append(p, **big) == want and decode(p, **big) == want and prompt(p, **big) == want
    assert K.gqa_workspace_size(p, K.OP_PROMPT_ATTN, 1, 1, 1) == 0


@pytest.mark.parametrize("kw,want", [(dict(page_size=0), -1), (dict(cache_fmt=K.MXFP4), -1)])
def test_bad_cache_parameters_concern_the_paged_calls(kw, want):
    assert append(P(**kw)) == want and decode(P(**kw)) == want
    assert prompt(P(**kw), n_seq=0) == 0
    assert K.gqa_workspace_size(P(**kw), K.OP_PAGED_DECODE, 1, 1, 1) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(n_seq=-1), -1), (dict(n_tok=-1), -1), (dict(n_tok=1 << 31), -3), (dict(cu=None), -1), (dict(pos0=None), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(qo=None), -1), (dict(q_ld=1023), -1), (dict(q_ld=1028), -2),
    (dict(k_ld=255), -1), (dict(v_ld=260), -2), (dict(q=ODD), -2), (dict(k=ODD), -2), (dict(qo=ODD), -2), (dict(kc=ODD), -2),
    (dict(kc=None), -1), (dict(table=None), -1), (dict(n_pages=-1), -1), (dict(max_pages=-1), -1),
    (dict(n_pages=1 << 31), -3), (dict(k=C.c_void_p(0x2000), ko=C.c_void_p(0x2000), k_ld=512), -1),
    (dict(qo=FAKE, q_ld=2048), -1)])
def test_append_refuses(kw, want):
    assert append(P(), **kw) == want


@pytest.mark.parametrize("rot,want", [(-2, -1), (7, -1), (144, -1), (24, -3)])
def test_append_refuses_rotations(rot, want):
    assert append(P(rot_dim=rot)) == want


def test_append_needs_frequencies_and_scales():
    assert append(P(rot_dim=64), f=None) == -1
    assert append(P(cache_fmt=K.FP8_S64), ks=None, vs=FAKE) == -1


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), -1), (dict(q=None), -1), (dict(pos=None), -1), (dict(out=None), -1), (dict(q_ld=1000), -1),
    (dict(q_ld=1028), -2), (dict(out=ODD), -2), (dict(ws=ODD), -2), (dict(wb=0), -4), (dict(ws=None), -1), (dict(vc=None), -1),
    (dict(batch=1 << 30), -3)])
def test_decode_refuses(kw, want):
    assert decode(P(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(n_seq=-1), -1), (dict(n_q=-1), -1), (dict(n_k=-1), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(cq=None), -1),
    (dict(ck=None), -1), (dict(out=None), -1), (dict(q_ld=8), -1), (dict(k_ld=260), -2), (dict(v=ODD), -2), (dict(wb=0), -4),
    (dict(ws=None), -1), (dict(n_q=1 << 31), -3), (dict(n_k=1 << 31), -3), (dict(n_q=1 << 29), -3)])
def test_prompt_refuses(kw, want):
    assert prompt(P(), **kw) == want


def test_nothing_to_do():
    assert append(P(), n_seq=0) == 0 and append(P(), n_tok=0) == 0
    assert decode(P(), batch=0) == 0
    assert prompt(P(), n_seq=0) == 0 and prompt(P(), n_q=0) == 0


def test_workspace_grows_with_the_heads_and_is_never_zero():
    for op in (K.OP_PAGED_DECODE, K.OP_PROMPT_ATTN):
        small, large = (K.gqa_workspace_size(P(n_heads=h), op, 8, 8, 4096) for h in (2, 64))
        assert 0 < small <= large < 1 << 30
    assert K.gqa_workspace_size(P(), K.OP_HCA_ATTN, 1, 1, 1) == 0
    assert K.gqa_workspace_size(P(), K.OP_PAGED_DECODE, -1, 1, 1) == 0


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    p, x = P(), torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        K._rows_of(x, 2, 8, p, "q")
    fake = type("T", (), dict(is_cuda=True, dtype=torch.bfloat16, shape=(2, 8, 64), stride=lambda self: (512, 64, 1)))()
    with pytest.raises(ValueError, match=r"\[2\]\[8\]\[128\]"):
        K._rows_of(fake, 2, 8, p, "q")
    fake.shape, fake.dtype = (2, 8, 128), torch.float32
    with pytest.raises(ValueError, match="bfloat16"):
        K._rows_of(fake, 2, 8, p, "q")
    fake.dtype = torch.bfloat16
    with pytest.raises(ValueError, match="dense"):
        K._rows_of(fake, 2, 8, p, "q")
    with pytest.raises(ValueError, match="int32"):
        K._dense(torch.zeros(3, dtype=torch.int64), (3,), torch.int32, "cu_q")


def test_a_paged_layer_hands_out_and_takes_back_pages():
    from compressed_sparse_attention_13_b200.paged import PagedLayer
    lay = PagedLayer(P(page_size=4), n_seq=2, n_pages=5, max_pages=4, device="cpu")
    lay.reserve(0, 9)
    lay.lens[0] = 9
    lay.reserve(1, 8)
    lay.lens[1] = 8
    assert sorted(lay.table[lay.table >= 0].tolist()) == [0, 1, 2, 3, 4]
    with pytest.raises(RuntimeError, match="no room"):
        lay.reserve(1, 1)
    lay.release(0)
    assert (lay.table[0] == -1).all()
    lay.advance()
    assert lay.lens == [0, 9] and lay.pos.tolist() == [-1, 8] and (lay.table[1] >= 0).sum() == 3
    with pytest.raises(RuntimeError, match="no room"):
        lay.reserve(1, 8)   # the pool has pages left, the table has not


def test_the_binding_refuses_tensors_of_different_devices():
    class On:
        is_cuda, shape, dtype = True, (2,), torch.int32

        def __init__(self, i):
            self.i, self.device = i, f"cuda:{i}"

        def get_device(self):
            return self.i

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 16 * self.i

    spec = ((2,), torch.int32, "cu_q")
    assert K._check(1, (On(1), *spec), (None, *spec), (On(1), *spec)) == [16, None, 16]
    with pytest.raises(ValueError, match="different devices: cu_q on cuda:0, another on cuda:1"):
        K._check(1, (On(1), *spec), (On(0), *spec))
    with pytest.raises(ValueError, match="int64"):
        K._check(1, (On(1), (2,), torch.int64, "cu_q"))


@pytest.mark.parametrize("kw,want", [(dict(max_pages=1 << 27), -3), (dict(n_pages=1 << 27), -3), (dict(max_pages=(1 << 27) - 1, wb=0), -4),
                                     (dict(n_pages=(1 << 27) - 1, wb=0), -4)])
def test_decode_counts_rows_in_32_bits(kw, want):
    """Pages of 16 tokens and two key heads: 2^27 of them are one too many, either way."""
    assert decode(P(), **kw) == want
