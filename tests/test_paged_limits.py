"""Sizes that the paged calls' helpers let pass or not (CPU)."""
import pytest


@pytest.fixture(scope="module")
def qi():
    import diffusion_transformer_text_gb300 as q
    q.build()
    q.lib()
    return q


def test_a_cache_has_pages_that_the_calls_take(qi):
    """Pages of more than 65536 rows are refused by both calls, so none are made."""
    assert qi.paged_kv(1, 65536, 1, device="cpu").k.shape == (1, 65536, 1, 128)
    for rows in (2 ** 17, 2 ** 20):
        with pytest.raises(ValueError, match="65536"):
            qi.paged_kv(1, rows, 1, device="cpu")


def test_a_table_past_the_longest_length_wants_a_bound(qi):
    """The calls take lengths of up to 2^24. Behind a table that reaches further a longer kv_len would be cut to that
    without a word, so the bound has to be the caller's."""
    import torch
    q, cache = torch.zeros(2, 1, 2, 128, dtype=torch.float16), qi.paged_kv(4, 64, 2, torch.float16, device="cpu")
    n = torch.zeros(2, dtype=torch.int32)
    for width, max_len, bound in ((2 ** 18, None, 2 ** 24), (2 ** 18 + 1, None, 0), (2 ** 18 + 1, 2 ** 24, 2 ** 24),
                                  (2 ** 18 + 1, 100, 100), (3, None, 192)):
        table = torch.zeros(2, width, dtype=torch.int32)
        check = lambda: qi._check_paged(object(), q, cache, table, n, None, max_len, True, None, None)
        if bound:
            assert qi._PAGED_TAIL.unpack(check()[1])[-1] == bound
        else:
            with pytest.raises(ValueError, match="max_len"):
                check()
