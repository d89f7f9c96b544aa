"""What the Python calls on paged caches and trees refuse before anything is enqueued (CPU only)."""
import pytest
import torch

from long_context_self_gb300 import binding


@pytest.fixture
def stand_in(monkeypatch):
    """Tensors without storage pass for CUDA ones of the current device, so that a call's own checks run."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(binding, "_current_device", lambda: None)


def empty(*shape, t=torch.int32):
    return torch.empty(shape, dtype=t, device="meta")


def test_batches_that_ctypes_would_cut_short(stand_in):
    B = (1 << 32) + 2                    # to a C int: 2
    with pytest.raises(ValueError, match=f"B is {B}"):
        binding.magicdec_tree_accept(empty(B, 1, 1, t=torch.float32), empty(B, 1))
    kp = empty(4, 16, 2, 64, t=torch.bfloat16)
    with pytest.raises(ValueError, match=f"B is {B}"):
        binding.magicdec_tree_commit(kp, kp, empty(B, 1), empty(B), empty(B, 1), empty(B))
    kp = empty(B, 1, 1, 64, t=torch.bfloat16)
    with pytest.raises(ValueError, match=r"k_pages.shape\[0\] is"):
        binding.magicdec_tree_commit(kp, kp, empty(2, 1), empty(2), empty(2, 1), empty(2))


def test_a_stream_of_another_device(stand_in):
    """It would become the current one with its device, and the call would go to the tensors'
    device's own current stream."""
    class Stream:
        cuda_stream, device = 7, torch.device("cuda", 1)

    class Here(Stream):
        device = torch.device("meta")

    x, p = empty(2, 4, 8, 128, t=torch.bfloat16), empty(20, 16, 8, 128, t=torch.bfloat16)
    lens = empty(2)
    calls = (lambda s: binding.magicdec_paged_append(x, x, p, p, empty(2, 10), lens, stream=s),
             lambda s: binding.magicdec_tree_attn(x, p, p, empty(2, 10), lens, stream=s),
             lambda s: binding.magicdec_tree_accept(empty(2, 4, 9, t=torch.float32), empty(2, 4), stream=s),
             lambda s: binding.magicdec_tree_commit(p, p, empty(2, 10), lens, empty(2, 4), lens, stream=s))
    for call in calls:
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call(Stream())
        with pytest.raises(Exception) as e:                 # goes on to select the device, of which there is none
            call(Here())
        assert "stream is on" not in str(e.value)


def test_pools_of_single_rows_past_32_bits():
    """Pages of 1 to 3 rows are gathered by their rows' numbers in the pool."""
    from long_context_self_gb300 import build
    build.build()
    lib, P = binding.lib(), binding.ctypes.c_void_p
    for page in (1, 2, 3):
        most = ((1 << 31) - 2) // page
        for n_pages, ok in ((most, True), (most + 1, page * (most + 1) < (1 << 31) - 1)):
            s = binding.paged_shape(1, 8, 1, 64, page, n_pages, 10)
            size = lib.magicdec_tree_attn_workspace_size(s, 4)
            assert (size > 0) == ok
            if not ok:
                x = P(0x10000)
                assert lib.magicdec_tree_attn(s, 4, x, x, x, x, x, P(0), P(0), x, x, 1 << 40, P(0)) == -5
    assert lib.magicdec_tree_attn_workspace_size(binding.paged_shape(1, 8, 1, 64, 4, 1 << 30, 10), 4) > 0
