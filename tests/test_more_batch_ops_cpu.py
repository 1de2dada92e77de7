"""4-bit pages, page pools and adjusted logits without a GPU: every refusal of their
arguments happens on the host, before anything is enqueued, with a status and a reason;
calls with nothing to do succeed."""
import ctypes

import pytest

import llama_decode_forward_gb300 as L
from llama_decode_forward_gb300 import binding as B
from test_batch_ops_cpu import BAD, BAD_PAGES, BAD_POINTERS, P, UNSUP, append, attend, pages, ref, refused


def read(**kw):
    base = dict(dtype=L.LLM_F16, k_out=P, v_out=P, k_stride=128, v_stride=128)
    return B.llm_read(**{**base, **kw})


def pool(**kw):
    base = dict(n_seqs=2, page_size=16, n_pages=4, max_pages=2, page_table=P, lens=P, refs=P, err=None, n_layers=2, k_pages=P,
                v_pages=P, page_bytes=4096, row_bytes=256, layer_stride=4 * 4096)
    return B.llm_pool(**{**base, **kw})


def adjust(**kw):
    base = dict(n_rows=2, vocab=100, dtype=L.LLM_F32, out_dtype=L.LLM_F16, logits=P, stride=100, out=2 * P, out_stride=100, history=P,
                history_lens=P, history_stride=50, max_history=50, window=0, repetition=P, frequency=P, presence=P, bias_ids=P, bias=P,
                n_bias=3, n_masks=2, masks=P, mask_stride=4, mask_of=P)
    return B.llm_adjust(**{**base, **kw})


Q4 = [(dict(page_size=4), UNSUP), (dict(page_size=1), UNSUP), (dict(head_dim=40), UNSUP), (dict(head_dim=8), UNSUP),
      (dict(page_size=1 << 20, max_pages=1, n_kv_heads=1 << 10), UNSUP)]


@pytest.mark.parametrize("kw,status", BAD_PAGES + BAD_POINTERS + Q4)
def test_pages_of_4_bits_refused(kw, status):
    refused(B._lib.llm_kv_append_q4(ref(pages(**kw)), ref(append()), None), status)
    refused(B._lib.llm_attend_batch_q4(ref(pages(**kw)), ref(attend()), None), status)
    refused(B._lib.llm_kv_read_q4(ref(pages(**kw)), ref(read()), None), status)
    if (kw, status) not in BAD_POINTERS:
        refused(B._lib.llm_attend_batch_q4_workspace(ref(pages(**kw)), ref(attend())), status)
    if (kw, status) not in Q4:
        refused(B._lib.llm_kv_read(ref(pages(**kw)), ref(read()), None), status)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=L.LLM_Q8_0), UNSUP), (dict(k_out=None), BAD), (dict(v_out=None), BAD), (dict(k_out=P + 8), BAD),
    (dict(v_out=P + 2), BAD), (dict(k_stride=64), BAD), (dict(v_stride=132), BAD), (dict(k_stride=-128), BAD),
])
def test_read_refused(kw, status):
    refused(B._lib.llm_kv_read(ref(pages()), ref(read(**kw)), None), status)
    refused(B._lib.llm_kv_read_q4(ref(pages()), ref(read(**kw)), None), status)


def test_attend_of_4_bits_refuses_a_small_workspace():
    p = pages(prefix_len=100)
    need = B._lib.llm_attend_batch_q4_workspace(ref(p), ref(attend()))
    assert need > 0
    for kw in (dict(workspace=None), dict(workspace=P + 128), dict(workspace_bytes=need - 1)):
        refused(B._lib.llm_attend_batch_q4(ref(p), ref(attend(**kw)), None), BAD)


@pytest.mark.parametrize("page,n_kv,hd,want", [(16, 8, 64, 16 * 8 * 40), (8, 1, 16, 96), (8, 2, 48, 512), (32, 32, 128, 32 * 32 * 80),
                                               (8, 1, 96, 8 * 60), (16, 1, 80, 16 * 52)])
def test_page_bytes(page, n_kv, hd, want):
    assert B._lib.llm_q4_page_bytes(page, n_kv, hd) == want


@pytest.mark.parametrize("args,status", [((0, 1, 64), BAD), ((24, 1, 64), BAD), ((4, 1, 64), UNSUP), ((16, 0, 64), BAD), ((16, 1, 40), UNSUP),
                                         ((16, 1, 144), UNSUP), ((1 << 30, 1, 64), UNSUP)])
def test_page_bytes_refused(args, status):
    refused(B._lib.llm_q4_page_bytes(*args), status)


BAD_POOL = [
    (dict(n_seqs=-1), BAD), (dict(n_pages=-1), BAD), (dict(max_pages=-1), BAD), (dict(n_layers=-1), BAD), (dict(page_size=0), BAD),
    (dict(page_size=12), BAD), (dict(n_seqs=4097), UNSUP), (dict(max_pages=1 << 27), UNSUP), (dict(n_pages=(1 << 31) - 1), UNSUP),
    (dict(page_bytes=0), BAD), (dict(page_bytes=4100), BAD), (dict(row_bytes=-16), BAD), (dict(row_bytes=100), BAD),
    (dict(row_bytes=272), BAD), (dict(layer_stride=4 * 4096 - 16), BAD), (dict(layer_stride=4 * 4096 + 8), BAD), (dict(layer_stride=-4 * 4096), BAD),
    (dict(n_layers=1 << 15, page_bytes=1 << 31, row_bytes=0, layer_stride=1 << 40), UNSUP),
]
BAD_POOL_POINTERS = [
    (dict(page_table=None), BAD), (dict(lens=None), BAD), (dict(refs=None), BAD), (dict(k_pages=None), BAD), (dict(v_pages=None), BAD),
    (dict(page_table=P + 2), BAD), (dict(lens=P + 1), BAD), (dict(refs=P + 2), BAD), (dict(err=P + 2), BAD), (dict(k_pages=P + 8), BAD),
    (dict(v_pages=P + 4), BAD),
]


@pytest.mark.parametrize("kw,status", BAD_POOL + BAD_POOL_POINTERS)
def test_pool_refused(kw, status):
    p = pool(**kw)
    refused(B._lib.llm_pages_update(ref(p), P, P, P, 1 << 40, None), status)
    refused(B._lib.llm_pages_compact(ref(p), P, P, 2 * P, P, P, 1 << 40, None), status)
    if (kw, status) in BAD_POOL:
        refused(B._lib.llm_pages_update_workspace(ref(p)), status)
        refused(B._lib.llm_pages_compact_workspace(ref(p)), status)


def test_pool_calls_refuse_their_own_arguments():
    p = pool()
    u, c = B._lib.llm_pages_update_workspace(ref(p)), B._lib.llm_pages_compact_workspace(ref(p))
    assert u > 0 and c > 0
    for ws, n in ((None, u), (P + 128, u), (P, u - 1), (P, -1)):
        refused(B._lib.llm_pages_update(ref(p), P, P, ws, n, None), BAD)
    for ws, n in ((None, c), (P + 64, c), (P, c - 1)):
        refused(B._lib.llm_pages_compact(ref(p), P, P, 2 * P, P, ws, n, None), BAD)
    for args in ((P + 2, P), (P, P + 1)):
        refused(B._lib.llm_pages_update(ref(p), *args, P, 1 << 40, None), BAD)
    for args in ((None, P, 2 * P, P), (P, None, 2 * P, P), (P, P, None, P), (P, P, 2 * P, None), (P + 2, P, 2 * P, P), (P, P, P, P),
                 (P, 3 * P, 3 * P, P), (P, P, 2 * P, P + 1)):
        refused(B._lib.llm_pages_compact(ref(p), *args, P, 1 << 40, None), BAD)
    refused(B._lib.llm_pages_update(None, P, P, P, 1 << 40, None), BAD)
    refused(B._lib.llm_pages_compact(None, P, P, 2 * P, P, P, 1 << 40, None), BAD)


@pytest.mark.parametrize("kw,status", [
    (dict(n_rows=-1), BAD), (dict(vocab=0), BAD), (dict(vocab=(1 << 30) + 1), UNSUP), (dict(max_history=-1), BAD), (dict(window=-1), BAD),
    (dict(n_bias=-1), BAD), (dict(n_masks=-1), BAD), (dict(dtype=L.LLM_Q8_0), UNSUP), (dict(out_dtype=3), UNSUP), (dict(logits=None), BAD),
    (dict(out=None), BAD), (dict(history_lens=None), BAD), (dict(bias_ids=None), BAD), (dict(bias=None), BAD), (dict(masks=None), BAD),
    (dict(logits=P + 2), BAD), (dict(out=P + 1), BAD), (dict(history=P + 2), BAD), (dict(history_lens=P + 2), BAD),
    (dict(repetition=P + 2), BAD), (dict(frequency=P + 1), BAD), (dict(presence=P + 2), BAD), (dict(bias_ids=P + 2), BAD),
    (dict(bias=P + 3), BAD), (dict(masks=P + 2), BAD), (dict(mask_of=P + 2), BAD), (dict(stride=99), BAD), (dict(out_stride=-100), BAD),
    (dict(history_stride=49), BAD), (dict(mask_stride=3), BAD), (dict(out=P), BAD), (dict(out=P, out_dtype=L.LLM_F32, out_stride=104), BAD),
    (dict(n_rows=1 << 28, vocab=1 << 17, stride=1 << 17, out_stride=1 << 17, mask_stride=1 << 12), UNSUP),
])
def test_adjust_refused(kw, status):
    refused(B._lib.llm_logits_adjust(ref(adjust(**kw)), None), status)


def test_null_structs_refused():
    refused(B._lib.llm_logits_adjust(None, None), BAD)
    for f, a in ((B._lib.llm_kv_append_q4, append()), (B._lib.llm_attend_batch_q4, attend()), (B._lib.llm_kv_read, read()), (B._lib.llm_kv_read_q4, read())):
        refused(f(None, ref(a), None), BAD)
        refused(f(ref(pages()), None, None), BAD)
    refused(B._lib.llm_pages_update_workspace(None), BAD)
    refused(B._lib.llm_pages_compact_workspace(None), BAD)


def test_nothing_to_do():
    none = pages(n_seqs=0, k_pages=None, v_pages=None, page_table=None, lens=None)
    for f, a in ((B._lib.llm_kv_append_q4, append()), (B._lib.llm_attend_batch_q4, attend()), (B._lib.llm_kv_read, read()), (B._lib.llm_kv_read_q4, read())):
        assert f(ref(none), ref(a), None) == L.LLM_OK
    assert B._lib.llm_logits_adjust(ref(adjust(n_rows=0, logits=None)), None) == L.LLM_OK
    assert B._lib.llm_pages_update(ref(pool(n_seqs=0, page_table=None, lens=None)), None, None, P, 1 << 40, None) == L.LLM_OK


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    x, one = torch.zeros(2, L.binding._lib.llm_q4_page_bytes(16, 2, 64), dtype=torch.uint8), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="is on cpu"):
        L.PagedBatchQ4(x, x, one.view(1, 1), one, 16, 2, 64)
    with pytest.raises(TypeError, match="uint8"):
        L.PagedBatchQ4(x.half(), x, one.view(1, 1), one, 16, 2, 64)
    with pytest.raises(L.LlmError):
        L.PagedBatchQ4(x, x, one.view(1, 1), one, 4, 2, 64)
    with pytest.raises(L.LlmError):
        L.q4_pages(3, 16, 2, 40)
    with pytest.raises(ValueError, match="is on cpu"):
        L.PagePool(None, None, one.view(1, 1), one, one, page_size=16)
    with pytest.raises(TypeError):
        L.PagePool(None, None, one.view(1, 1), one, one.float(), page_size=16)
    with pytest.raises(ValueError, match="is on cpu"):
        L.AdjustLogits(torch.zeros(2, 10))
    with pytest.raises(TypeError):
        L.AdjustLogits(torch.zeros(2, 10, dtype=torch.float64))


def test_binding_refuses_sizes_that_32_bits_do_not_hold():
    torch = pytest.importorskip("torch")
    x, one, big = torch.zeros(2, 16, dtype=torch.uint8), torch.ones(1, dtype=torch.int32), (1 << 32) + 8
    for kw in (dict(prefix_len=big), dict(n_new=big)):
        with pytest.raises(ValueError, match="32-bit"):
            L.PagedBatchQ4(x, x, one.view(1, 1), one, 16, 2, 64, **kw)
    for args in ((big, 2, 64), (16, big, 64), (16, 2, big)):
        with pytest.raises(ValueError, match="32-bit"):
            L.PagedBatchQ4(x, x, one.view(1, 1), one, *args)
        with pytest.raises(ValueError, match="32-bit"):
            L.q4_pages(1, *args)
    with pytest.raises(ValueError, match="32-bit"):
        L.AdjustLogits(torch.zeros(2, 10), window=big)


def test_decode_batch_of_4_bits_refuses_a_dead_handle():
    b = B.llm_batch(n_seqs=1, n_new=1)
    for h in (None, 0x1000):
        assert B._lib.llm_decode_batch_q4(h, ctypes.addressof(b)) == BAD
        assert B._lib.llm_batch_q4_pages_bytes(h, 1, 16) == BAD
