"""The operators of batched decoding without a GPU: every refusal of their
arguments happens on the host, before anything is enqueued, with a status and
a reason (llm_last_error(NULL)); calls with nothing to do succeed."""
import ctypes

import pytest

import llama_decode_forward_gb300 as L
from llama_decode_forward_gb300 import binding as B

P = 0x10000          # a 16-byte aligned address that no refused call reads


def pages(**kw):
    base = dict(n_seqs=2, n_new=1, prefix_len=0, page_size=16, n_pages=4, max_pages=2, n_kv_heads=2, head_dim=64,
                k_pages=P, v_pages=P, page_table=P, lens=P, err=None)
    return B.llm_pages(**{**base, **kw})


def append(**kw):
    base = dict(n_heads=4, rope_dims=64, rope_neox=0, table_rows=64, dtype=L.LLM_F32, q_out_dtype=L.LLM_F16, q=P, k=P,
                v=P, q_stride=256, k_stride=128, v_stride=128, q_out=2 * P, q_out_stride=256, cos_sin=P)
    return B.llm_append(**{**base, **kw})


def attend(**kw):
    base = dict(n_heads=4, q_dtype=L.LLM_F32, out_dtype=L.LLM_F16, scale=0.0, q=P, q_stride=256, out=P, out_stride=256,
                prefix_k=P, prefix_v=P, prefix_stride=128, workspace=P, workspace_bytes=1 << 40)
    return B.llm_attend(**{**base, **kw})


def logprobs(**kw):
    base = dict(n_rows=2, vocab=100, dtype=L.LLM_F32, n_targets=1, top=5, logits=P, stride=100, targets=P, logprob=P,
                entropy=P, top_id=P, top_logprob=P)
    return B.llm_logprobs_args(**{**base, **kw})


ref = ctypes.byref
BAD, UNSUP = L.LLM_ERR_INVALID_ARG, L.LLM_ERR_UNSUPPORTED

BAD_PAGES = [
    (dict(n_seqs=-1), BAD), (dict(n_new=0), BAD), (dict(n_new=-3), BAD), (dict(prefix_len=-1), BAD),
    (dict(page_size=0), BAD), (dict(page_size=24), BAD), (dict(page_size=-16), BAD), (dict(n_pages=-1), BAD),
    (dict(max_pages=-1), BAD), (dict(n_kv_heads=0), BAD), (dict(head_dim=0), BAD), (dict(head_dim=60), UNSUP),
    (dict(head_dim=136), UNSUP), (dict(n_seqs=1 << 20, n_new=1 << 20), UNSUP),
    (dict(max_pages=1 << 30, page_size=16), UNSUP), (dict(n_kv_heads=1 << 30), UNSUP),
]
BAD_POINTERS = [
    (dict(lens=None), BAD), (dict(page_table=None), BAD), (dict(k_pages=None), BAD), (dict(v_pages=None), BAD),
    (dict(k_pages=P + 8), BAD), (dict(v_pages=P + 2), BAD), (dict(page_table=P + 2), BAD), (dict(lens=P + 1), BAD),
    (dict(err=P + 2), BAD),
]


def refused(rc, status):
    assert rc == status
    assert L.llm_last_error(None)


@pytest.mark.parametrize("kw,status", BAD_PAGES + BAD_POINTERS)
def test_pages_refused(kw, status):
    refused(B._lib.llm_kv_append(ref(pages(**kw)), ref(append()), None), status)
    refused(B._lib.llm_attend_batch(ref(pages(**kw)), ref(attend()), None), status)


@pytest.mark.parametrize("kw,status", BAD_PAGES)
def test_workspace_query_refuses_bad_sizes(kw, status):
    refused(B._lib.llm_attend_batch_workspace(ref(pages(**kw)), ref(attend())), status)


@pytest.mark.parametrize("kw,status", [
    (dict(n_heads=-1), BAD), (dict(table_rows=-1), BAD), (dict(rope_dims=63), BAD), (dict(rope_dims=66), BAD),
    (dict(rope_dims=-2), BAD), (dict(dtype=L.LLM_Q8_0), UNSUP), (dict(dtype=2), UNSUP),
    (dict(q_out_dtype=L.LLM_Q8_0), UNSUP), (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD),
    (dict(q_out=None), BAD), (dict(cos_sin=None), BAD), (dict(cos_sin=P + 8), BAD), (dict(q=P + 4), BAD),
    (dict(k=P + 8), BAD), (dict(v=P + 8), BAD), (dict(q_out=P + 8), BAD), (dict(q_stride=252), BAD),
    (dict(k_stride=130), BAD), (dict(k_stride=64), BAD), (dict(v_stride=-128), BAD), (dict(q_out_stride=248), BAD),
    (dict(q_out=P), BAD),                                                      # q itself, but of another type
    (dict(q_out=P, q_out_dtype=L.LLM_F32, q_out_stride=512), BAD),             # or of another stride
])
def test_append_refused(kw, status):
    refused(B._lib.llm_kv_append(ref(pages()), ref(append(**kw)), None), status)


@pytest.mark.parametrize("kw", [dict(n_seqs=4097), dict(n_seqs=4096, max_pages=1 << 20)])
def test_attend_refuses_what_append_takes(kw):
    for rc in (B._lib.llm_attend_batch(ref(pages(**kw)), ref(attend()), None),
               B._lib.llm_attend_batch_workspace(ref(pages(**kw)), ref(attend()))):
        refused(rc, UNSUP)


@pytest.mark.parametrize("kw,status", [
    (dict(n_heads=0), BAD), (dict(n_heads=3), BAD), (dict(q_dtype=L.LLM_Q8_0), UNSUP), (dict(out_dtype=7), UNSUP),
    (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(q=None), BAD),
    (dict(out=None), BAD), (dict(q=P + 4), BAD), (dict(out=P + 8), BAD), (dict(q_stride=258), BAD),
    (dict(q_stride=252), BAD), (dict(out_stride=128), BAD),
])
def test_attend_refused(kw, status):
    refused(B._lib.llm_attend_batch(ref(pages()), ref(attend(**kw)), None), status)


@pytest.mark.parametrize("kw", [dict(workspace=None), dict(workspace=P + 128), dict(workspace_bytes=0),
                                dict(workspace_bytes=-1)])
def test_attend_refuses_a_bad_workspace(kw):
    refused(B._lib.llm_attend_batch(ref(pages(prefix_len=100)), ref(attend(**kw)), None), BAD)
    need = B._lib.llm_attend_batch_workspace(ref(pages(prefix_len=100)), ref(attend()))
    assert need > 0
    refused(B._lib.llm_attend_batch(ref(pages(prefix_len=100)), ref(attend(workspace_bytes=need - 1)), None), BAD)


@pytest.mark.parametrize("kw", [dict(prefix_k=None), dict(prefix_v=None), dict(prefix_k=P + 8), dict(prefix_v=P + 2),
                                dict(prefix_stride=64), dict(prefix_stride=132)])
def test_attend_refuses_bad_prefix(kw):
    refused(B._lib.llm_attend_batch(ref(pages(prefix_len=100)), ref(attend(**kw)), None), BAD)


@pytest.mark.parametrize("kw,status", [
    (dict(n_rows=-1), BAD), (dict(vocab=0), BAD), (dict(n_targets=-1), BAD), (dict(top=-1), BAD),
    (dict(top=33), UNSUP), (dict(vocab=4, top=5), BAD), (dict(dtype=L.LLM_Q8_0), UNSUP), (dict(logits=None), BAD),
    (dict(targets=None), BAD), (dict(logprob=None), BAD), (dict(top_id=None), BAD), (dict(top_logprob=None), BAD),
    (dict(logits=P + 2), BAD), (dict(logits=P + 1, dtype=L.LLM_F16), BAD), (dict(targets=P + 2), BAD),
    (dict(logprob=P + 2), BAD), (dict(entropy=P + 1), BAD), (dict(top_id=P + 2), BAD), (dict(top_logprob=P + 2), BAD),
    (dict(stride=99), BAD), (dict(stride=-100), BAD),
])
def test_logprobs_refused(kw, status):
    refused(B._lib.llm_logprobs(ref(logprobs(**kw)), None), status)


@pytest.mark.parametrize("args", [(None, 0, 4, 64, 1e4), (P, -1, 4, 64, 1e4), (P, 0, -1, 64, 1e4), (P, 0, 4, 63, 1e4),
                                  (P, 0, 4, 0, 1e4), (P, 0, 4, 64, 0.0), (P, 0, 4, 64, float("nan")),
                                  (P, (1 << 31) - 1, 4, 64, 1e4)])
def test_rope_table_refused(args):
    refused(B._lib.llm_rope_table(*args, None, None), BAD)


def test_attend_refuses_a_prefix_at_the_end_of_32_bits():
    for n, status in (((1 << 31) - 1, UNSUP), ((1 << 31) - 64, UNSUP)):
        refused(B._lib.llm_attend_batch_workspace(ref(pages(prefix_len=n)), ref(attend())), status)
    assert B._lib.llm_attend_batch_workspace(ref(pages(prefix_len=(1 << 31) - 65)), ref(attend())) > 0


def test_null_structs_refused():
    refused(B._lib.llm_kv_append(None, ref(append()), None), BAD)
    refused(B._lib.llm_kv_append(ref(pages()), None, None), BAD)
    refused(B._lib.llm_attend_batch(None, ref(attend()), None), BAD)
    refused(B._lib.llm_attend_batch(ref(pages()), None, None), BAD)
    refused(B._lib.llm_attend_batch_workspace(None, ref(attend())), BAD)
    refused(B._lib.llm_attend_batch_workspace(ref(pages()), None), BAD)
    refused(B._lib.llm_logprobs(None, None), BAD)


def test_decode_batch_refuses_a_dead_handle():
    b = B.llm_batch(n_seqs=1, n_new=1)
    assert B._lib.llm_decode_batch(None, ctypes.addressof(b)) == BAD
    assert B._lib.llm_decode_batch(0x1000, ctypes.addressof(b)) == BAD
    assert B._lib.llm_batch_pages_bytes(None, 1, 16) == BAD


def test_nothing_to_do():
    """No sequences, rows or positions: success without a launch (no GPU here)."""
    none = pages(n_seqs=0, k_pages=None, v_pages=None, page_table=None, lens=None)
    assert B._lib.llm_kv_append(ref(none), ref(append()), None) == L.LLM_OK
    assert B._lib.llm_attend_batch(ref(none), ref(attend()), None) == L.LLM_OK
    assert B._lib.llm_logprobs(ref(logprobs(n_rows=0, logits=None)), None) == L.LLM_OK
    assert B._lib.llm_rope_table(P, 0, 0, 64, 1e4, None, None) == L.LLM_OK


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 16, 2, 64, dtype=torch.float16)
    lens = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="is on cpu"):
        L.PagedBatch(x, x, torch.zeros(1, 1, dtype=torch.int32), lens)
    with pytest.raises(TypeError, match="float16"):
        L.PagedBatch(x.float(), x, torch.zeros(1, 1, dtype=torch.int32), lens)
    with pytest.raises(ValueError, match="is on cpu"):
        L.LogProbs(torch.zeros(2, 10))
    with pytest.raises(TypeError):
        L.LogProbs(torch.zeros(2, 10, dtype=torch.float64))


def test_binding_refuses_sizes_that_32_bits_do_not_hold():
    """A C int32 would keep the low bits of these: 2^32 + 5 would be 5."""
    torch = pytest.importorskip("torch")
    x, one = torch.zeros(2, 16, 2, 64, dtype=torch.float16), torch.ones(1, dtype=torch.int32)
    big = (1 << 32) + 5
    for kw in (dict(prefix_len=big), dict(n_new=big), dict(prefix_len=-big)):
        with pytest.raises(ValueError, match="32-bit"):
            L.PagedBatch(x, x, one.view(1, 1), one, **kw)
    with pytest.raises(ValueError, match="32-bit"):
        L.LogProbs(torch.zeros(2, 10), top=big)
    for args in ((big, 64, 1e4), (4, big, 1e4)):
        with pytest.raises(ValueError, match="32-bit"):
            L.rope_table(*args)
    with pytest.raises(ValueError, match="32-bit"):
        L.rope_table(4, 64, 1e4, pos0=1 << 31)
    for args in ((big, 16, 0), (1, big, 0), (1, 16, big), (1, 16, 0, big), (1, 16, 0, 1, big)):
        with pytest.raises(ValueError, match="32-bit"):
            L.BatchDecoder(None, *args)
    with pytest.raises(ValueError, match="positive"):
        L.BatchDecoder(None, 1, 16, 0, 1, 0)
    for args in ((big, 16), (3, big)):
        with pytest.raises(ValueError, match="32-bit"):
            L.llm_batch_pages_bytes(None, *args)


@pytest.mark.parametrize("args,freqs,status", [((P + 2, 0, 4, 64, 1e4), None, BAD), ((P, 0, 4, 64, 1e4), P + 1, BAD),
                                               ((P, 0, 1, 1026, 1e4), None, UNSUP), ((P, 0, 1, 1 << 30, 1e4), None, UNSUP)])
def test_rope_table_refuses_what_its_kernel_cannot_take(args, freqs, status):
    refused(B._lib.llm_rope_table(*args, freqs, None), status)


@pytest.mark.parametrize("kw,heads", [
    (dict(n_seqs=2, prefix_len=(1 << 31) - 65, n_kv_heads=16384, head_dim=8), 16384),            # 2^39 tiles of the prefix
    (dict(n_seqs=1, n_new=512, max_pages=(1 << 27) - 1, n_kv_heads=16384, head_dim=8), 16384),   # 2^46 pieces of the pages
])
def test_attend_refuses_shares_beyond_32_bits(kw, heads):
    refused(B._lib.llm_attend_batch_workspace(ref(pages(**kw)), ref(attend(n_heads=heads))), UNSUP)
