"""The binding's own checks, on CPU tensors (a call that passes them all is refused for its device)."""
import pytest
import torch

from adaptive_block_sparse_hilbert_b200 import fva


@pytest.mark.parametrize("backward", [False, True])
def test_masks_as_tensors_or_as_the_struct(backward):
    """Like the other entry points, the training ones take a Mask or a filled fva_mask."""
    s = fva.make_shape(1, 2, 64, 1, 8, 10)
    x = [torch.zeros(1, 2, 80, 64, dtype=torch.bfloat16) for _ in range(8)]
    lse, ws = torch.zeros(1, 2, 80), torch.zeros(1 << 16, dtype=torch.uint8)
    mask = fva.Mask.allocate(s, "cpu")
    for m in (mask, mask.c()):
        with pytest.raises(ValueError, match="expected a CUDA device"):
            if backward:
                fva.fva_sparse_attn_bwd(s, *x[:5], lse, m, *x[5:], ws)
            else:
                fva.fva_sparse_attn_lse(s, *x[:3], m, x[3], lse)
    small = fva.Mask.allocate(fva.make_shape(1, 1, 64, 1, 8, 8), "cpu")
    with pytest.raises(ValueError, match="another shape"):
        fva.fva_sparse_attn_lse(s, *x[:3], small, x[3], lse)


def test_a_cache_keeps_to_its_buffers():
    """The struct that the calls pass on names the buffers the object shows: others need another object."""
    c = fva.Cache.allocate(4, 2, 64, device="cpu")
    for name in ("k", "v", "key_mean", "mass"):
        with pytest.raises(AttributeError):
            setattr(c, name, torch.zeros_like(getattr(c, name)))
        assert getattr(c.c(), name) == getattr(c, name).data_ptr()
    assert fva.Cache(c.k, c.v, c.key_mean).c().mass is None
