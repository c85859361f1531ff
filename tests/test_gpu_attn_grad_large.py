"""The gradient at layers of a real clip's size: more than 128 blocks a head, rows and columns of
more than 64 and 128 entries, more tiles than SMs. The float64 formula runs on the device;
the bounds are those of test_gpu_attn_grad.py."""
import numpy as np
import pytest

from tests.test_gpu_attn_grad import _mask

pytestmark = pytest.mark.gpu

LARGE = [  # H, T, Hg, Wg, d, dtype, blocks a head
    (2, 1, 17, 491, 64, "bf16", 131),   # an odd block count, the last block of 27 rows
    (2, 1, 17, 491, 128, "bf16", 131),
    (1, 5, 31, 61, 128, "bf16", 148),   # 74 tiles: all resident, in their own order
    (2, 2, 36, 62, 64, "f32", 70),
    (1, 1, 67, 67, 128, "f32", 71),
    (2, 3, 38, 38, 32, "f32", 68),
]


def _blocks(H, nB, rng):
    """Per head: rows that keep from nothing to everything, columns that nobody or everybody keeps."""
    share = rng.choice([0.05, 0.3, 0.7, 0.97], (H, nB, 1))
    keep = rng.random((H, nB, nB)) < share
    keep[:, 10:, 66], keep[:, :, nB - 2] = True, True
    keep[:, 3], keep[:, -1] = True, True
    keep[:, 4], keep[:, 6:8] = False, False    # a pair's first row, and a whole pair
    keep[:, :, 65] = False
    return keep


class Large:
    def __init__(self, H, T, Hg, Wg, d, dtype, nB, seed=0):
        import torch
        from adaptive_block_sparse_hilbert_b200 import fva
        self.fva, self.H, self.d, self.N = fva, H, d, T * Hg * Wg
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        assert -(-self.N // 64) == nB
        self.s = fva.make_shape(1, H, d, T, Hg, Wg, dtype)
        rng = np.random.default_rng(seed)
        self.keep = _blocks(H, nB, rng)
        self.mask = _mask(fva, self.s, self.keep)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q, self.k, self.v, self.do = (torch.randn(1, H, self.N, d, device="cuda", generator=g).to(self.dt) for _ in range(4))
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        # as the forward leaves them: o rounded to the type, lse to float32
        heads = [self.formula(h) for h in range(H)]
        self.o = torch.stack([(p @ self.v[0, h].double()).to(self.dt) for h, (p, _) in enumerate(heads)])[None]
        self.lse = torch.stack([lse.float() for _, lse in heads])[None]
        self.ws = torch.full((fva.fva_sparse_attn_bwd_workspace_bytes(self.s),), 255, dtype=torch.uint8, device="cuda")

    def formula(self, h):
        """P and the log-sum-exp of a head; 0 and -infinity for rows that keep nothing."""
        import torch
        block = torch.arange(self.N, device="cuda") // 64
        seen = torch.from_numpy(self.keep[h]).cuda()[block][:, block]
        q, k = self.q[0, h].double(), self.k[0, h].double()
        s = torch.where(seen, q @ k.T / self.d ** 0.5, torch.full((), -torch.inf, dtype=torch.float64, device="cuda"))
        lse = torch.logsumexp(s, 1)
        return torch.exp(s - torch.where(lse.isfinite(), lse, 0.0)[:, None]), lse

    def forward(self):
        import torch
        o, lse = torch.empty_like(self.q), torch.full((1, self.H, self.N), float("nan"), device="cuda")
        self.fva.fva_sparse_attn_lse(self.s, self.q, self.k, self.v, self.mask, o, lse, dev_status=self.st)
        assert int(self.st.item()) == 0
        return lse

    def backward(self):
        import torch
        out = [torch.full_like(self.q, float("nan")) for _ in range(3)]
        self.fva.fva_sparse_attn_bwd(self.s, self.q, self.k, self.v, self.o, self.do, self.lse, self.mask, *out, self.ws,
                                     dev_status=self.st)
        assert int(self.st.item()) == 0
        return out

    def check(self, lse_got, out, p_rel=None):
        """p_rel: o and lse are the forward's own, whose weights have this rounding (0: fp32)."""
        import torch
        bf, scale = self.dt == torch.bfloat16, 1 / self.d ** 0.5
        for h in range(self.H):
            q, k, v, do, o = (x[0, h].double() for x in (self.q, self.k, self.v, self.do, self.o))
            p, lse = self.formula(h)
            rows, got = lse.isfinite(), lse_got[0, h].double()
            score = scale * (q.abs() @ k.abs().T)
            # scores: d products; the sum of N weights, each 2^-21 off; the logarithm's own rounding
            limit = 2.0 ** -24 * ((self.d + 16) * score.max(1).values + self.N + 16) + 2.0 ** -20
            assert bool((got[~rows] == -torch.inf).all()) and bool(((got - lse).abs() <= limit)[rows].all())
            dp, adp = do @ v.T, do.abs() @ v.abs().T
            delta, ad = (p * dp).sum(1, keepdim=True), (do.abs() * o.abs()).sum(1, keepdim=True)
            ds = p * (dp - delta)
            if bf:
                rel, small, n_out = 2.0 ** -8, 2.0 ** -11, 2.0 ** -8
                e_p = p * (rel + small)
                e_ds = rel * ds.abs() + p * (rel * ad + small * (adp + ad))
            else:
                n = 2.0 ** -24
                e_s = n * (self.d + 8) * score + 4 * n * (1 + torch.where(rows, lse, 0.0).abs())[:, None]
                e_p = p * (2 * e_s + 4 * n)
                e_ds = e_p * (dp - delta).abs() + p * n * (self.d + 8) * (adp + 2 * ad) + 4 * n * ds.abs()
                n_out = n * (self.N + 8)
            if p_rel is not None:
                # lse is off by `limit` at most, which scales a row's P; o by its weights' roundings, their scores'
                # errors and a sum of N: both enter D
                e_w = p * ((p_rel + 2 * limit)[:, None] + 2.0 ** -24 * (2 * (self.d + 8) * score + self.N + 64))
                e_d = (e_w * adp).sum(1, keepdim=True)
                e_ds = e_ds + p * (2 * limit[:, None] * (dp - delta).abs() + 2 * e_d)
                e_p = e_p + 2 * p * limit[:, None]
            want = (scale * ds @ k, scale * ds.T @ q, p.T @ do)
            bounds = (scale * e_ds @ k.abs(), scale * e_ds.T @ q.abs(), e_p.T @ do.abs())
            sums = (scale * ds.abs() @ k.abs(), scale * ds.abs().T @ q.abs(), p.T @ do.abs())
            for name, x, w, e, total in zip(("dq", "dk", "dv"), out, want, bounds, sums):
                limit_x = e + (n_out * w.abs() + 2.0 ** -16 * total if bf else n_out * total) + 1e-30
                over = ((x[0, h].double() - w).abs() / limit_x).max()
                assert float(over) <= 1.0, (name, h, float(over))


@pytest.mark.parametrize("case", LARGE, ids=str)
def test_gradient_of_a_large_layer(case):
    import torch
    c = Large(*case)
    out = c.backward()
    c.check(c.forward(), out)
    assert all(torch.equal(a, b) for a, b in zip(out, c.backward()))


@pytest.mark.parametrize("B,H,T,Hg,Wg,d,dtype,v_fp16,curve", [
    (2, 2, 3, 10, 13, 64, "bf16", True, 0), (1, 3, 3, 10, 13, 128, "bf16", False, 0), (1, 2, 4, 16, 17, 128, "bf16", True, 1),
    (2, 2, 3, 10, 13, 64, "f32", True, 0), (1, 2, 3, 11, 12, 32, "f32", False, 1), (1, 2, 3, 10, 13, 128, "f32", True, 0),
    (1, 1, 1, 1, 1, 64, "bf16", True, 0)])
def test_layers_of_every_kind_train(B, H, T, Hg, Wg, d, dtype, v_fp16, curve):
    """SparseAttentionLayer(train=True): both types, V kept as fp16 or not, both token orders, batches;
    forward and gradients in raster order, the mask as routed."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import fva, pipeline
    s = fva.make_shape(B, H, d, T, Hg, Wg, dtype)
    layer = pipeline.SparseAttentionLayer(s, 0.6, 1, v_fp16=v_fp16, curve=curve, train=True)
    N, nB = layer.N, layer.nB
    g = torch.Generator(device="cuda").manual_seed(N + d)
    q, k, v, do = (torch.randn(B, N, H, d, device="cuda", generator=g).to(layer.dtype) for _ in range(4))
    grads = [torch.full_like(q, float("nan")) for _ in range(3)]
    o = layer.forward(2 * q, k, v, torch.empty_like(q))
    layer.backward(do, *grads)
    assert int(layer.dev_status.item()) == 0
    along = lambda x: x[:, layer.perm.long()].transpose(1, 2).reshape(1, B * H, N, d)  # noqa: E731
    assert torch.equal(along(2 * q), layer.qh.view(1, B * H, N, d)) and torch.equal(along(o), layer.oh.view(1, B * H, N, d))
    c = object.__new__(Large)
    c.H, c.N, c.d, c.dt, c.keep = B * H, N, d, layer.dtype, np.zeros((B * H, nB, nB), dtype=bool)
    c.q, c.k, c.v, c.do, c.o = along(2 * q), along(k), along(v), along(do), layer.oh.view(1, B * H, N, d)
    rp, ci = layer.mask.row_ptr.cpu().numpy(), layer.mask.col_idx.cpu().numpy()
    for r in range(B * H * nB):
        c.keep[r // nB, r % nB, ci[rp[r]:rp[r + 1]]] = True
    assert nB == 1 or not c.keep.all()
    p_rel = 0.0 if dtype == "f32" else 2.0 ** -11 if v_fp16 else 2.0 ** -8
    c.check(layer.lse.view(1, B * H, N), [along(x) for x in grads], p_rel)
