"""A workspace tensor too small to hold an aligned byte is one of no bytes: a negative number would reach the C ABI as a huge
size and pass its check (no GPU needed)."""
import pytest
import torch


def _slices():
    t = torch.zeros(4096, dtype=torch.uint8)
    at = -t.data_ptr() % 256
    return [t[at + 3:at + 10], t[at + 1:at + 1], t[at + 255:at + 256], t[at + 1:at + 256], t[at:at + 1], t[at + 1:at + 300], t[at:at + 512]]


@pytest.mark.parametrize("i", range(7))
def test_sizes_are_those_of_the_aligned_part(i, monkeypatch):
    from bit_moe_expert_router_gb300 import attention, binding
    monkeypatch.setattr(binding, "_need", lambda *a, **k: None)  # (a CPU tensor stands in)
    ws = _slices()[i]
    end = ws.data_ptr() + ws.numel()
    view, view_size = binding._ws_view(ws)
    for at, size in (attention._aligned(ws), (view.value or 0, view_size)):
        assert at % 256 == 0 and size >= 0
        assert size == max(0, end - at)


def test_a_workspace_of_no_bytes_is_refused(cuda_lib):
    import ctypes

    from bit_moe_expert_router_gb300 import attention
    from test_attention_abi import FAKE, _attend, _batch
    lib = attention._load()
    at, size = attention._aligned(_slices()[0])
    assert _attend(lib, _batch(), ws=FAKE, nbytes=ctypes.c_size_t(size)) == 3
