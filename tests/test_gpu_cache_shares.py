"""Attention of single queries where the lists are cut into equal shares, one per CTA (large calls;
small ones have a cluster per unit, see test_gpu_cache.py): units inside a share, units that cross
many, units of more than 16 query heads, and the second launch that joins and accumulates.
Bounds as in test_gpu_cache.py.

A table of more than 192 blocks keeps a call from the clusters. `by_shares` shows which path a call
took: without accumulation the clusters write nothing into the workspace, and the shares do."""
import numpy as np
import pytest

from tests.test_gpu_cache import Streams

pytestmark = pytest.mark.gpu

WIDE = 400
KINDS = [("bf16", 128, 2, 4), ("bf16", 128, 1, 40), ("bf16", 64, 2, 1), ("bf16", 64, 1, 128), ("f16", 128, 1, 2), ("f16", 64, 2, 3),
         ("f16", 64, 1, 20), ("f16", 128, 1, 17), ("f32", 32, 2, 2), ("f32", 32, 1, 20), ("f32", 64, 3, 1), ("f32", 64, 1, 17),
         ("f32", 128, 1, 8), ("f32", 128, 2, 1), ("f32", 128, 1, 20)]


def by_shares(s, q, kept=None, n=None):
    ws = s.ws(s.fva.fva_cache_attn_workspace_bytes(s.cache, s.B, s.max_blocks, s.H, False))
    s.fva.fva_cache_attn(s.cache, s.table, s.length, q, kept, n, s.torch.empty_like(s.dev(s.q)), ws, dev_status=s.st)
    return bool((ws != 255).any())


def lengths(kind):
    if kind == "long":  # about 370 blocks a key head: one unit crosses most of the shares
        return [20001, 0, 1, 65, 3000]
    # units inside a share, with empty ones between them and at both ends
    lens = np.random.default_rng(7).integers(0, 300, 400)
    lens[::7] = 0
    return [0, *lens.tolist(), 700, 0]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("streams", ["long", "many"])
@pytest.mark.parametrize("dtype,d,Hkv,G", KINDS)
def test_attention_by_shares(dtype, d, Hkv, G, streams, accumulate):
    s = Streams(lengths(streams), Hkv * G, Hkv, d, dtype, max_blocks=WIDE).fill()
    s.cache.mass.uniform_(0, 3)
    q = s.query(wide=1)
    assert by_shares(s, q)
    for every in (True, False):
        before = s.cache.mass.double().cpu().numpy()
        kept = n = None
        blocks = [[np.arange(-(-m // 64))] * Hkv for m in s.lens]
        if not every:
            kept, n = s.route(q, 0.5, 2, 1)
            blocks = s.want_route(0.5, 2, 1)
        o, lse = s.attn(q, kept, n, accumulate=accumulate)
        s.ok()
        s.check_attn(o, lse, blocks, before if accumulate else None)


def test_a_narrow_table_takes_the_clusters():
    """What by_shares tells apart."""
    s = Streams([64, 700], 4, 2, 64, "bf16").fill()
    assert not by_shares(s, s.query())


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f32", 64)])
def test_large_scores_by_shares(dtype, d):
    s = Streams([9000, 257], 4, 1, d, dtype, scale_k=40.0, max_blocks=WIDE).fill()
    q = s.query()
    assert by_shares(s, q)
    o, lse = s.attn(q, None, None)
    s.ok()
    s.check_attn(o, lse, [[np.arange(-(-m // 64))] for m in s.lens])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f16", 64), ("f32", 32), ("f32", 128)])
@pytest.mark.parametrize("streams", ["long", "many"])
def test_weightless_rows_are_zero_whatever_their_values(dtype, d, streams):
    """Heads whose every score is -infinity give 0 and -infinity also where the values are
    infinite or NaN, in units inside a share and in those that cross several."""
    s = Streams(lengths(streams), 2, 1, d, dtype, max_blocks=WIDE)
    for k, v in zip(s.k, s.v):
        k[:, 0, 0] = -np.inf
        v[::3, 0, 1], v[1::3, 0, 2] = np.inf, np.nan
    s.fill()
    q = np.abs(s.draw(s.B, 2, d))
    q[:, :, 0] = 1.0
    q = s.query(q)
    assert by_shares(s, q)
    for accumulate in (False, True):
        o, lse = s.attn(q, None, None, accumulate=accumulate)
        s.ok()
        assert bool((o == 0).all()) and bool(lse.isneginf().all())


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("H,Hkv,d,dtype", [(8, 2, 128, "bf16"), (20, 1, 64, "f16"), (3, 3, 32, "f32"), (8, 2, 128, "f32")])
def test_wait_that_runs_out_is_reported(H, Hkv, d, dtype, accumulate):
    """With the loads withheld and a 20 ms limit the call reports a timeout, ends and leaves the
    device usable; the next call is right."""
    s = Streams([700, 64, 0, 15000], H, Hkv, d, dtype, max_blocks=WIDE).fill()
    q = s.query()
    assert by_shares(s, q)
    s.fva.fva_set_diagnostics(20_000_000, s.fva.FVA_DIAG_WITHHOLD_Q)
    try:
        s.attn(q, None, None, accumulate=accumulate)
        s.ok(s.fva.FVA_DEVERR_TIMEOUT)
    finally:
        s.fva.fva_set_diagnostics(0, 0)
    s.cache.mass.zero_()
    before = s.cache.mass.double().cpu().numpy()
    o, lse = s.attn(q, None, None, accumulate=accumulate)
    s.ok()
    s.check_attn(o, lse, [[np.arange(-(-n // 64))] * Hkv for n in s.lens], before if accumulate else None)
