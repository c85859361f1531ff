"""Gradient of block-sparse attention (fva_sparse_attn_lse, fva_sparse_attn_bwd) against the
float64 formula, at masks with empty rows and unused key blocks, ragged ends, both head dims.

The bounds are elementwise and come from the roundings the kernels make. bf16: P and dS are
rounded once each (2^-8 relative, half a step), O arrives rounded (2^-8), the gradients are
rounded once; fp32 sums and exponentials add less than 2^-11 of the same magnitudes. fp32: each
sum of n products is off by at most n 2^-24 of the sum of their magnitudes, a score's error
multiplies P."""
import numpy as np
import pytest

from oracle import grad_oracle as GO

pytestmark = pytest.mark.gpu

CASES = [  # B, H, T, Hg, Wg, d, dtype, mask
    (1, 1, 1, 1, 1, 64, "bf16", "full"),
    (1, 2, 1, 8, 8, 128, "bf16", "full"),
    (1, 2, 1, 5, 13, 64, "bf16", "full"),
    (2, 3, 3, 12, 17, 128, "bf16", "random"),
    (2, 3, 3, 12, 17, 64, "bf16", "random"),
    (1, 2, 4, 16, 16, 128, "bf16", "holes"),
    (1, 2, 4, 16, 17, 64, "bf16", "holes"),
    (1, 2, 4, 16, 17, 128, "bf16", "diagonal"),
    (1, 1, 3, 11, 12, 128, "bf16", "none"),
    (1, 2, 13, 10, 10, 128, "bf16", "one column"),
    (1, 1, 1, 1, 1, 32, "f32", "full"),
    (1, 2, 1, 5, 13, 128, "f32", "full"),
    (2, 3, 3, 12, 17, 64, "f32", "random"),
    (1, 2, 4, 16, 17, 32, "f32", "holes"),
    (1, 2, 3, 11, 12, 128, "f32", "holes"),
]


def _blocks(kind, BH, nB, rng):
    keep = rng.random((BH, nB, nB)) < 0.5
    if kind == "full":
        keep[:] = True
    if kind == "holes":
        keep[:, 1::3] = False
        keep[:, :, ::4] = False
    if kind == "diagonal":
        keep[:] = np.eye(nB, dtype=bool)
    if kind == "none":
        keep[:] = False
    if kind == "one column":
        keep[:] = False
        keep[:, :, -1] = True
    return keep


def _mask(fva, s, keep):
    import torch
    BH, nB, _ = keep.shape
    m = fva.Mask.allocate(s)
    rows = keep.reshape(BH * nB, nB)
    m.row_ptr.copy_(torch.from_numpy(np.concatenate([[0], rows.sum(1).cumsum()]).astype(np.int32)))
    cols = rows.nonzero()[1].astype(np.int32)
    m.col_idx[:cols.size] = torch.from_numpy(cols)
    ws = torch.empty(fva.fva_tiles_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fva.fva_build_tiles(s, m, ws, dev_status=st)
    assert int(st.item()) == 0
    return m


class Case:
    def __init__(self, B, H, T, Hg, Wg, d, dtype, kind, seed=0):
        import torch
        from adaptive_block_sparse_hilbert_b200 import fva
        self.fva, self.dt = fva, torch.bfloat16 if dtype == "bf16" else torch.float32
        self.s = fva.make_shape(B, H, d, T, Hg, Wg, dtype)
        self.N, self.B, self.H, self.d = T * Hg * Wg, B, H, d
        nB = (self.N + 63) // 64
        rng = np.random.default_rng(seed)
        self.keep = _blocks(kind, B * H, nB, rng)
        self.mask = _mask(fva, self.s, self.keep)
        make = lambda: torch.from_numpy(rng.standard_normal((B, H, self.N, d)).astype(np.float32)).to(self.dt).cuda()  # noqa: E731
        self.q, self.k, self.v, self.do = (make() for _ in range(4))
        self.seen = [GO.token_mask(self.keep[i], self.N) for i in range(B * H)]
        f = [x.double().cpu().numpy().reshape(B * H, self.N, d) for x in (self.q, self.k, self.v, self.do)]
        self.f = f
        fwd = [GO.attention(f[0][i], f[1][i], f[2][i], self.seen[i]) for i in range(B * H)]
        self.o_want = np.stack([x[0] for x in fwd])
        self.lse_want = np.stack([x[1] for x in fwd])
        four = (B, H, self.N, d)
        self.o = torch.from_numpy(self.o_want.reshape(four)).float().to(self.dt).cuda()
        self.lse = torch.from_numpy(self.lse_want.reshape(four[:3])).float().cuda()
        n = fva.fva_sparse_attn_bwd_workspace_bytes(self.s)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # what is in it does not matter
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def backward(self, **kw):
        import torch
        out = [torch.full_like(self.q, float("nan")) for _ in range(3)]
        self.fva.fva_sparse_attn_bwd(self.s, self.q, self.k, self.v, self.o, self.do, self.lse, self.mask, *out, self.ws,
                                     dev_status=self.st, **kw)
        return out

    def check(self, out):
        assert int(self.st.item()) == 0
        q, k, v, do = self.f
        scale = 1 / np.sqrt(self.d)
        o = self.o.double().cpu().numpy().reshape(-1, self.N, self.d)
        bf = out[0].element_size() == 2
        for i in range(self.B * self.H):
            _, lse, p = GO.attention(q[i], k[i], v[i], self.seen[i])
            want = GO.attention_grad(q[i], k[i], v[i], do[i], self.seen[i])
            dp = do[i] @ v[i].T
            delta = (p * dp).sum(1, keepdims=True)
            ds = p * (dp - delta)
            score = scale * np.abs(q[i]) @ np.abs(k[i]).T
            adp = np.abs(do[i]) @ np.abs(v[i]).T
            ad = (np.abs(do[i]) * np.abs(o[i])).sum(1, keepdims=True)
            if bf:
                rel, small, n_out = 2.0 ** -8, 2.0 ** -11, 2.0 ** -8
                e_p = p * (rel + small)
                e_ds = rel * np.abs(ds) + p * (rel * ad + small * (adp + ad))
            else:
                n = 2.0 ** -24
                e_s = n * (self.d + 8) * score + 4 * n * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))[:, None]
                e_p = p * (2 * e_s + 4 * n)
                e_ds = e_p * np.abs(dp - delta) + p * n * (self.d + 8) * (adp + 2 * ad) + 4 * n * np.abs(ds)
                n_out = n * (self.N + 8)
            bounds = (scale * e_ds @ np.abs(k[i]), scale * e_ds.T @ np.abs(q[i]), e_p.T @ np.abs(do[i]))
            sums = (scale * np.abs(ds) @ np.abs(k[i]), scale * np.abs(ds).T @ np.abs(q[i]), p.T @ np.abs(do[i]))
            for name, got, w, e, total in zip(("dq", "dk", "dv"), out, want, bounds, sums):
                got = got.double().cpu().numpy().reshape(-1, self.N, self.d)[i]
                limit = e + (n_out * np.abs(w) + 2.0 ** -16 * total if bf else n_out * total) + 1e-30
                over = np.abs(got - w) / limit
                assert not np.isnan(got).any() and over.max() <= 1.0, (name, i, float(over.max()))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradient(case):
    c = Case(*case)
    c.check(c.backward())


@pytest.mark.parametrize("case", [CASES[3], CASES[4], CASES[5], CASES[8], CASES[12], CASES[14]], ids=str)
def test_forward_lse(case):
    """The forward's lse, and its output equal to fva_sparse_attn's bit for bit."""
    import torch
    c = Case(*case)
    o, o2 = torch.full_like(c.q, float("nan")), torch.empty_like(c.q)
    lse = torch.full((c.B, c.H, c.N), float("nan"), device="cuda")
    c.fva.fva_sparse_attn_lse(c.s, c.q, c.k, c.v, c.mask, o, lse, dev_status=c.st)
    c.fva.fva_sparse_attn(c.s, c.q, c.k, c.v, c.mask, o2, dev_status=c.st)
    assert int(c.st.item()) == 0 and torch.equal(o, o2)
    got = lse.double().cpu().numpy().reshape(-1, c.N)
    rows = np.isfinite(c.lse_want)
    assert (np.isneginf(got) == ~rows).all()
    # scores: d products; the sum of N weights, each 2^-21 off; the logarithm's own rounding
    score = np.stack([(np.abs(c.f[0][i]) @ np.abs(c.f[1][i]).T).max(1) for i in range(c.B * c.H)]) / np.sqrt(c.d)
    limit = 2.0 ** -24 * ((c.d + 16) * score + c.N + 16) + 2.0 ** -20
    assert (np.abs(got[rows] - c.lse_want[rows]) <= limit[rows]).all()


def test_equal_inputs_give_equal_bits():
    import torch
    c = Case(2, 3, 3, 12, 17, 128, "bf16", "random")
    first = c.backward()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, c.backward()))


def test_other_scale_other_stream():
    import torch
    c = Case(1, 2, 3, 12, 17, 64, "bf16", "random")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out = c.backward(scale=0.125)
    torch.cuda.current_stream().wait_stream(st)
    c.check(out)  # 1 / sqrt(64)
    assert all(torch.equal(a, b) for a, b in zip(out, c.backward()))


def test_captured_and_replayed_with_new_inputs():
    import torch
    c, n = Case(1, 2, 3, 12, 17, 128, "bf16", "random", 1), Case(1, 2, 3, 12, 17, 128, "bf16", "holes", 2)
    c.backward()
    torch.cuda.synchronize()
    out = [torch.empty_like(c.q) for _ in range(3)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.fva.fva_sparse_attn_bwd(c.s, c.q, c.k, c.v, c.o, c.do, c.lse, c.mask, *out, c.ws, dev_status=c.st)
    for x in ("q", "k", "v", "o", "do", "lse"):
        getattr(c, x).copy_(getattr(n, x))
    for x in ("row_ptr", "col_idx", "tile_ptr", "tile_col", "worklist"):
        getattr(c.mask, x).copy_(getattr(n.mask, x))
    g.replay()
    torch.cuda.synchronize()
    n.check(out)


def test_layer_trains():
    """A layer's backward against differences of its own oracle: raster order in and out, the
    routed mask held fixed."""
    import torch
    import oracle as O
    from adaptive_block_sparse_hilbert_b200 import pipeline, synth
    from tests import _common as C
    wl = synth.custom_workload(3, 10, 13, 2, 128, "bf16", seed=61)
    L = synth.make_layer(wl)
    layer = pipeline.SparseAttentionLayer(C.shape_of(wl), wl.p, wl.k_floor, train=True)
    q, k, v = C.to_device(L)
    o, do = torch.empty_like(q), torch.randn_like(q)
    grads = [torch.empty_like(q) for _ in range(3)]
    layer.forward(q, k, v, o)
    layer.backward(do, *grads)
    assert int(layer.dev_status.item()) == 0
    plain = pipeline.SparseAttentionLayer(C.shape_of(wl), wl.p, wl.k_floor)
    assert torch.equal(o, plain.forward(q, k, v, torch.empty_like(q)))
    perm, _ = O.hilbert_perm(wl.T, wl.Hg, wl.Wg)
    rp = layer.mask.row_ptr.cpu().numpy()
    ci = layer.mask.col_idx.cpu().numpy()
    f = [O.reorder(x.double().cpu().numpy(), perm) for x in (q, k, v, do)]
    for h in range(wl.H):
        keep = np.zeros((wl.nB, wl.nB), dtype=bool)
        for a in range(wl.nB):
            r = h * wl.nB + a
            keep[a, ci[rp[r]:rp[r + 1]]] = True
        want = GO.attention_grad(*(x[0, h] for x in f), GO.token_mask(keep, wl.N))
        for g, w in zip(grads, want):
            got = O.reorder(g.double().cpu().numpy(), perm)[0, h]
            # P, dS, O and the result rounded to bf16, each 2^-8 at most, in the 2-norm
            assert np.linalg.norm(got - w) <= 4 * 2.0 ** -8 * np.linalg.norm(w)


def test_backward_needs_a_training_layer():
    import torch
    from adaptive_block_sparse_hilbert_b200 import fva, pipeline
    layer = pipeline.SparseAttentionLayer(fva.make_shape(1, 1, 64, 1, 8, 8), 0.9, 2)
    x = torch.empty(1, 64, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError):
        layer.backward(x, x, x, x)


@pytest.mark.parametrize("d", [64, 128])
def test_wait_that_runs_out_is_reported(d):
    """With the first loads withheld and a 20 ms limit the gradient kernels report a timeout and
    leave the device usable; the next call is right."""
    c = Case(1, 2, 3, 12, 17, d, "bf16", "random")
    c.fva.fva_set_diagnostics(20_000_000, c.fva.FVA_DIAG_WITHHOLD_Q)
    try:
        c.backward()
        assert int(c.st.item()) == c.fva.FVA_DEVERR_TIMEOUT
    finally:
        c.fva.fva_set_diagnostics(0, 0)
    c.st.zero_()
    c.check(c.backward())


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "f32")])
def test_bad_list_entries_are_reported(d, dtype):
    """Tile entries and work-list entries that name nothing are reported, not followed."""
    c = Case(1, 2, 3, 12, 17, d, dtype, "random")
    good = c.mask.tile_col[5].clone()
    c.mask.tile_col[5] = 4 * 4000 + 3
    c.backward()
    assert int(c.st.item()) == c.fva.FVA_DEVERR_BAD_LIST
    c.mask.tile_col[5] = good
    c.st.zero_()
    if dtype == "bf16":
        good = c.mask.worklist[1].clone()
        c.mask.worklist[1] = 4000
        c.backward()
        assert int(c.st.item()) == c.fva.FVA_DEVERR_BAD_LIST
        c.mask.worklist[1] = good
        c.st.zero_()
    c.check(c.backward())


@pytest.mark.parametrize("d", [64, 128])
def test_short_wait_limits_end(d):
    """Whatever waits run out, in some of the warps or none, the calls end and the next is right."""
    c = Case(1, 2, 3, 12, 17, d, "bf16", "random")
    for limit in (1, 2000, 20000):
        c.fva.fva_set_diagnostics(limit, 0)
        try:
            for _ in range(10):
                c.backward()
                assert int(c.st.item()) in (0, c.fva.FVA_DEVERR_TIMEOUT)
        finally:
            c.fva.fva_set_diagnostics(0, 0)
    c.st.zero_()
    c.check(c.backward())


def test_training_layer_refusals():
    """A gradient before any forward, and a forward with the mask of another shape."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import fva, pipeline
    s = fva.make_shape(1, 1, 64, 1, 8, 16)
    layer = pipeline.SparseAttentionLayer(s, 0.9, 2, train=True)
    x = torch.zeros(1, 128, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError):
        layer.backward(x, x, x, x)
    small = fva.Mask.allocate(fva.make_shape(1, 1, 64, 1, 8, 8))
    t = [torch.zeros(1, 1, 128, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    with pytest.raises(ValueError):
        fva.fva_sparse_attn_lse(s, *t[:3], small, t[3], torch.zeros(1, 1, 128, device="cuda"))
