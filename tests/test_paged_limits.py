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
