"""What rglru_paged_kv_read_q4 returns are two tensors of their own."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("given", [None, "k", "v"])
def test_outputs_take_part_in_a_graph(gpu_lib, dtype, given):
    cache = [torch.full((3, 2, 8, 64 // (32 if c % 2 else 2)), 0x22 if c % 2 == 0 else 127, dtype=torch.uint8, device="cuda") for c in range(4)]
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    own = {} if given is None else {given: torch.empty(5, 2, 64, dtype=dtype, device="cuda")}
    k, v = gpu_lib.rglru_paged_kv_read_q4(*cache, slots, dtype=dtype, **own)
    assert bool((k == 1).all()) and bool((v == 1).all())   # code 2 is 1
    w = torch.full_like(k, 3.0, requires_grad=True)
    k.add_(w)
    (k * v).sum().backward()
    assert bool((v == 1).all()) and bool((w.grad == 1).all()) and not v.requires_grad
    assert k.untyped_storage().data_ptr() != v.untyped_storage().data_ptr() and k.untyped_storage().nbytes() < k.nbytes + 512
