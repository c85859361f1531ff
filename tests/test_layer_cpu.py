"""SparseAttentionLayer.backward's refusals: made on the host, before anything is enqueued."""
import pytest
import torch

from adaptive_block_sparse_hilbert_b200 import fva, pipeline


def _layer(B=2, N=70, H=3, d=64):
    """A training layer behind a forward, without its device buffers."""
    layer = object.__new__(pipeline.SparseAttentionLayer)
    layer.shape, layer.N, layer.train, layer.scale = fva.make_shape(B, H, d, 1, 7, 10), N, True, 0.0
    layer.dtype = torch.bfloat16
    layer.perm = torch.empty(N, dtype=torch.int32)
    for name in ("doh", "qh", "kh", "vb", "oh", "lse", "mask", "dqh", "dkh", "dvh", "bwd_workspace", "dev_status"):
        setattr(layer, name, None)
    return layer


BAD = {
    "a stride of 0": lambda x: x[:1, :1].expand_as(x),       # the gradient of a sum
    "heads before tokens": lambda x: x.transpose(1, 2).contiguous().transpose(1, 2),
    "every second row": lambda x: x.repeat_interleave(2, 1)[:, ::2],
    "too few tokens": lambda x: x[:, :-1].contiguous(),
    "Hilbert order's shape": lambda x: x.transpose(1, 2).contiguous(),
    "another type": lambda x: x.float(),
    "another device": lambda x: x.to("meta"),
}


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("bad", BAD)
def test_backward_refuses_what_it_would_read_or_write_wrongly(monkeypatch, which, bad):
    layer = _layer()
    ran = []
    for name in ("fva_reorder", "fva_sparse_attn_bwd"):
        monkeypatch.setattr(fva, name, lambda *a, **k: ran.append(a))
    x = [torch.ones(2, 70, 3, 64, dtype=torch.bfloat16) for _ in range(4)]
    layer.backward(*x)
    assert len(ran) == 5
    x[which] = BAD[bad](x[which])
    with pytest.raises(ValueError):
        layer.backward(*x)
    assert len(ran) == 5
