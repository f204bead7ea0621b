"""Which outputs of the norm share an allocation, and that none can grow into another."""
import pytest

pytestmark = pytest.mark.gpu


def _outputs(T, H):
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    x = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").bfloat16()
    return api.add_rms_norm_fp8(x, x, torch.ones(H, device="cuda"))


@pytest.mark.parametrize("T,H", [(1, 4096), (33, 272), (3000, 2048)])
def test_the_residual_has_an_allocation_of_its_own(T, H):
    q, scales, y, s = _outputs(T, H)
    own = s.untyped_storage()
    assert own.nbytes() == 2 * T * H and s.storage_offset() == 0
    assert all(t.untyped_storage().data_ptr() != own.data_ptr() for t in (q, scales, y))


def test_no_output_can_grow_into_another():
    import torch
    outs = _outputs(33, 272)
    before, kept = [t.clone() for t in outs], [t.detach() for t in outs]
    size = outs[0].untyped_storage().nbytes()
    for t in outs[:3]:  # torch raises after it has changed t's shape: t itself is not looked at again
        with pytest.raises(RuntimeError):
            t.resize_(1 << 20)
    outs[3].resize_(1 << 20).zero_()  # of its own: as any tensor
    assert kept[0].untyped_storage().nbytes() == size
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(kept[:3], before))
