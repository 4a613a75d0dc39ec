"""Sizes that the packed-sequence operators state, and what they ask of them (no GPU needed)."""
import ctypes

import pytest

import persistent_sm_decode_02_b200 as pkg
from persistent_sm_decode_02_b200 import dec as D_
from test_operators_host import INVALID, P, _library, attention, cache  # noqa: F401


def _bytes(c, n_seqs, n_heads):
    n = ctypes.c_size_t(0)
    assert D_.dec_attention_paged_workspace(c, n_seqs, n_heads, ctypes.byref(n)) == D_.DEC_OK
    return n.value


def test_workspace_size_goes_by_the_head_size_alone():
    """A buffer made once serves every batch and every head count: the work is cut into as many pieces whatever it is."""
    small = _bytes(cache(), 1, 4)
    assert small == _bytes(cache(), 5000, 16) == _bytes(cache(n_pages=1000, page_size=128, n_kv_heads=4), 3, 4)
    assert small < _bytes(cache(head_dim=128), 1, 4) < 4 << 20


def test_workspace_of_one_byte_too_few_is_refused():
    need = _bytes(cache(), 1, 4)
    assert attention(workspace_bytes=need - 1) == INVALID
    import torch
    if not torch.cuda.is_available():  # with a GPU the addresses are refused instead
        assert attention(workspace_bytes=need) == D_.DEC_ERR_CUDA


@pytest.mark.parametrize("given,held", [({}, 0), (dict(wait_timeout_us=250), 250)])
def test_cache_carries_its_wait_limit(given, held):
    c = pkg.PagedCache(P, P, P, P, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, **given)
    assert c.c.wait_timeout_us == held
    assert ctypes.sizeof(D_.dec_paged_cache) == 56
