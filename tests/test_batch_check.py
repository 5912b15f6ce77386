"""The batch operators' status call and its test hook, as far as they go without a GPU."""
import pytest


@pytest.fixture(scope="module")
def qi():
    import diffusion_transformer_text_gb300 as q
    q.build()
    q.lib()
    return q


def test_stall_hook_needs_no_handle(qi):
    assert qi.STATUS[qi.lib().qi_debug_inject(None, 3, 0)] == "QI_OK"
    assert qi.STATUS[qi.lib().qi_debug_inject(None, 0, 0)] == "QI_OK"


def test_check_without_a_device_is_an_error(qi):
    import torch
    if torch.cuda.is_available():
        pytest.skip("there is a device")
    assert qi.STATUS[qi.lib().qi_prefix_attention_check(None)] == "QI_ERR_CUDA"
    assert "qi_prefix_attention_check" in qi.lib().qi_last_error().decode()
