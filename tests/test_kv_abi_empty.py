"""Host-side check of the paged cache's C entry points for calls without tokens (no GPU needed)."""

import pytest

import block_quantized_matvec_gq_gb300 as gq
from test_kv_abi import ENTRIES, call, lib  # noqa: F401 (lib: builds and loads the library)


@pytest.mark.parametrize("name,good", ENTRIES)
def test_without_tokens_the_token_arrays_may_be_null(name, good):
    none = {p: None for p in ("K", "V", "Q", "O") if p in good}
    assert call(name, good, n_tokens=0, **none) == gq.GQ_OK
    assert call(name, good, n_tokens=1, **none) == gq.GQ_ERR_NULL
    for p in ("cache", "table", "kv_len", "q_start"):
        assert call(name, good, n_tokens=0, **{p: None}) == gq.GQ_ERR_NULL, p
