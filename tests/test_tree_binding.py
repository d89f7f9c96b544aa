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
