"""What the context-free operators refuse before any device call (no GPU needed: the addresses are never read)."""
import ctypes

import pytest

import persistent_sm_decode_02_b200 as pkg
from persistent_sm_decode_02_b200 import dec as D_

P = 1 << 20  # an aligned address


@pytest.fixture(autouse=True)
def _library():
    import os
    if not os.path.exists(pkg.LIB_PATH):
        import persistent_sm_decode_02_b200.build as b
        b.build()


def cache(**over):
    a = dict(k_pages=P, v_pages=P, k_scales=P, v_scales=P, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64)
    a.update(over)
    return D_.dec_paged_cache(**a)


def append(c=None, rope=None, **over):
    a = dict(dtype=D_.DEC_BF16, q=P, k=P, v=P, q_out=P, k_out=None, q_stride=256, k_stride=128, v_stride=128,
             q_out_stride=256, k_out_stride=128, n_heads=4, n_seqs=1, n_tokens=3, max_new=3, cu_new=P, seq_lens=P, page_table=P, table_stride=2, status=None,
             stream=None)
    a.update(over)
    return D_.dec_kv_append(cache() if c is None else c, D_.dec_rope(P, 64, 0, 1.0) if rope is None else rope, *a.values())


def attention(c=None, **over):
    a = dict(dtype=D_.DEC_BF16, q=P, out=P + 4096, q_stride=256, out_stride=256, n_heads=4, n_seqs=1, seq_lens=P, page_table=P,
             table_stride=2, scale=0.125, workspace=P, workspace_bytes=1 << 30, status=None, stream=None)
    a.update(over)
    return D_.dec_attention_paged(cache() if c is None else c, *a.values())


def prefill(**over):
    a = dict(dtype=D_.DEC_BF16, q=P, k=P, v=P, out=P + 4096, q_stride=256, k_stride=128, v_stride=128, out_stride=256, n_heads=4,
             n_kv_heads=2, head_dim=64, n_seqs=1, n_q=3, n_k=3, max_q=3, cu_q=P, cu_k=P, causal=1, scale=0.125, status=None,
             stream=None)
    a.update(over)
    return D_.dec_attention_prefill(*a.values())


INVALID, UNSUPPORTED = D_.DEC_ERR_INVALID_ARG, D_.DEC_ERR_UNSUPPORTED


def test_good_arguments_reach_the_device():
    """Without a GPU the same calls end at the first device call, not at a check."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (append, attention, prefill):
        assert call() == D_.DEC_ERR_CUDA


BAD_CACHE = [(dict(k_pages=None), INVALID), (dict(v_scales=None), INVALID), (dict(k_pages=P + 8), INVALID),
             (dict(k_scales=P + 2), INVALID), (dict(n_pages=0), INVALID), (dict(page_size=0), INVALID),
             (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
             (dict(n_kv_heads=3), UNSUPPORTED), (dict(n_kv_heads=0), INVALID)]


@pytest.mark.parametrize("over,rc", BAD_CACHE, ids=str)
def test_cache_is_checked(over, rc):
    assert append(cache(**over)) == rc
    assert attention(cache(**over)) == rc
    n = ctypes.c_size_t(0)
    assert D_.dec_attention_paged_workspace(cache(**over), 1, 4, ctypes.byref(n)) == rc


@pytest.mark.parametrize("over", [dict(dtype=D_.DEC_FP8_E4M3_B128), dict(dtype=9), dict(k=None), dict(v=None), dict(q=None),
                                  dict(q_out=None), dict(cu_new=None), dict(seq_lens=None), dict(page_table=None),
                                  dict(q=P + 2), dict(k=P + 8), dict(v=P + 4), dict(k_out=P + 8),
                                  dict(k_out=P, k_out_stride=120), dict(q_out=P + 8), dict(cu_new=P + 1),
                                  dict(status=P + 2), dict(q_stride=248), dict(q_stride=257), dict(k_stride=127),
                                  dict(v_stride=132), dict(q_out_stride=0), dict(n_seqs=-1), dict(n_tokens=-1),
                                  dict(max_new=-1), dict(table_stride=-1)], ids=str)
def test_append_is_checked(over):
    assert append(**over) == INVALID


@pytest.mark.parametrize("rope,rc", [((None, 64, 0, 1.0), INVALID), ((P + 4, 64, 0, 1.0), INVALID), ((P, 80, 0, 1.0), INVALID),
                                     ((P, -16, 0, 1.0), INVALID), ((P, 24, 0, 1.0), UNSUPPORTED), ((P, 64, 2, 1.0), INVALID),
                                     ((P, 64, 0, float("nan")), INVALID), ((P, 64, 0, float("inf")), INVALID)], ids=str)
def test_rope_is_checked(rope, rc):
    assert append(rope=D_.dec_rope(*rope)) == rc


@pytest.mark.parametrize("over,rc", [(dict(n_heads=3), UNSUPPORTED), (dict(n_heads=18), UNSUPPORTED), (dict(n_heads=0), INVALID)],
                         ids=str)
def test_heads_are_checked(over, rc):
    assert append(**over) == rc
    assert attention(**over) == rc
    assert prefill(**over) == rc


@pytest.mark.parametrize("over", [dict(dtype=2), dict(q=None), dict(out=None), dict(seq_lens=None), dict(page_table=None),
                                  dict(workspace=None), dict(workspace_bytes=0), dict(workspace=P + 8), dict(q=P + 8),
                                  dict(out=P + 2), dict(out=P), dict(seq_lens=P + 2), dict(q_stride=255), dict(out_stride=260),
                                  dict(n_seqs=-1), dict(table_stride=-1), dict(scale=0.0), dict(scale=-1.0),
                                  dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38)], ids=str)
def test_attention_is_checked(over):
    assert attention(**over) == INVALID


@pytest.mark.parametrize("over,rc", [(dict(dtype=2), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
                                     (dict(v=None), INVALID), (dict(out=None), INVALID), (dict(out=P), INVALID), (dict(cu_q=None), INVALID),
                                     (dict(cu_k=P + 2), INVALID), (dict(q=P + 8), INVALID), (dict(k_stride=120), INVALID),
                                     (dict(v_stride=129), INVALID), (dict(n_q=-1), INVALID), (dict(max_q=-1), INVALID),
                                     (dict(n_k=-1), INVALID), (dict(n_seqs=-1), INVALID), (dict(head_dim=80), UNSUPPORTED),
                                     (dict(head_dim=0), INVALID), (dict(n_kv_heads=3), UNSUPPORTED), (dict(scale=0.0), INVALID),
                                     (dict(scale=float("inf")), INVALID)], ids=str)
def test_prefill_is_checked(over, rc):
    assert prefill(**over) == rc


def test_sizes_past_what_is_counted_in_32_bits_are_refused():
    assert attention(n_seqs=1 << 16, table_stride=1 << 16) == UNSUPPORTED  # 2^16 * 2 * 2^16 tiles of 16
    assert prefill(n_seqs=1 << 30, n_q=1 << 30, max_q=1 << 20) == UNSUPPORTED
    assert append(n_seqs=1 << 30, n_tokens=1 << 30, max_new=1 << 20) == UNSUPPORTED


def test_nothing_to_do_is_no_error():
    assert append(n_seqs=0, k=None, v=None, cu_new=None) == D_.DEC_OK
    assert append(n_tokens=0, k=None, v=None) == D_.DEC_OK
    assert attention(n_seqs=0, q=None, workspace=None, workspace_bytes=0) == D_.DEC_OK
    assert prefill(n_seqs=0) == D_.DEC_OK and prefill(n_q=0) == D_.DEC_OK


def test_workspace_size_grows_with_nothing_on_the_device():
    """The size goes by head counts and the batch, not by what lengths the device holds."""
    n = ctypes.c_size_t(0)
    assert D_.dec_attention_paged_workspace(cache(), 5, 4, ctypes.byref(n)) == D_.DEC_OK and n.value > 0
    assert D_.dec_attention_paged_workspace(cache(), -1, 4, ctypes.byref(n)) == INVALID
    assert D_.dec_attention_paged_workspace(cache(), 1, 4, None) == INVALID


def test_convenience_class_raises():
    c = pkg.PagedCache(P, P, P, P, n_pages=4, page_size=48, n_kv_heads=2, head_dim=64)
    with pytest.raises(pkg.DecError) as e:
        c.workspace_bytes(1, 4)
    assert e.value.code == UNSUPPORTED
