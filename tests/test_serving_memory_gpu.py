"""The serving calls where memory runs out."""
import pytest
import torch

from gpu_parity import free_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_blackwell_gb300 import build
    build.build()
    yield
    free_cuda()


def test_out_of_memory_is_the_error_of_torch():
    """As from the calls whose outputs torch.empty makes."""
    from attention_forward_blackwell_gb300 import binding
    parents = torch.full((4096, 1024), -1, dtype=torch.int32, device="cuda")   # 512 MB of masks
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (64 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            binding.tree_mask(parents)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    mask = binding.tree_mask(parents)
    assert mask.shape == (4096, 1024, 32)
    assert bool((mask[17, 40] == torch.tensor([0, 1 << 8] + [0] * 30, device="cuda")).all())
