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


def test_a_cache_passes_on_the_buffers_it_shows():
    """The struct names the buffers that the object holds, also after one was replaced; one that does
    not fit the others is refused and changes nothing."""
    c = fva.Cache.allocate(4, 2, 64, device="cpu", mass=False)
    assert c.c().mass is None
    c.mass = torch.zeros(4, 2, 64)
    c.mass *= 2
    for name in ("k", "v", "key_mean", "mass"):
        setattr(c, name, torch.zeros_like(getattr(c, name)))
        for bad in (getattr(c, name)[:3], getattr(c, name).to("meta")):
            with pytest.raises(ValueError):
                setattr(c, name, bad)
        assert all(getattr(c.c(), n) == getattr(c, n).data_ptr() for n in ("k", "v", "key_mean", "mass"))
        assert c.c().n_pages == 4
    c.mass = None
    assert c.c().mass is None
