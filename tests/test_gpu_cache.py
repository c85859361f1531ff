"""The paged cache (append, routing of single queries, their attention, eviction) against the
float64 oracle. Caches are filled with NaN wherever nothing was written, table entries behind a
sequence's last block name no page, and workspaces start out as 0xff bytes.

Bounds: a 16-bit output is rounded once (eps / 2); scores are sums of d products in fp32, so a
score is off by at most (d + 16) 2^-24 of the sum of their magnitudes, which multiplies a
weight; the weighted sum of n values adds (n + 64) 2^-24; 16-bit caches may split a weight into
two 16-bit parts (2^-15 of it at most)."""
import numpy as np
import pytest

from oracle import cache_oracle as CO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": "bfloat16", "f16": "float16", "f32": "float32"}


class Streams:
    """A cache, its page table and a host copy of every stream's tokens in the stored type."""

    def __init__(self, lens, H, Hkv, d, dtype, seed=0, max_blocks=None, spare=2, scale_k=1.0):
        import torch
        from adaptive_block_sparse_hilbert_b200 import fva
        self.fva, self.torch, self.dt = fva, torch, getattr(torch, DT[dtype])
        self.rng = np.random.default_rng(seed)
        self.H, self.Hkv, self.G, self.d, self.B = H, Hkv, H // Hkv, d, len(lens)
        need = [-(-n // 64) for n in lens]
        self.max_blocks = max_blocks or max(1, max(need)) + 1
        n_pages = sum(need) + spare
        nan = float("nan")
        self.cache = fva.Cache(*(torch.full((n_pages, Hkv, 64, d), nan, dtype=self.dt, device="cuda") for _ in range(2)),
                               torch.full((n_pages, Hkv, d), nan, device="cuda"),
                               torch.full((n_pages, Hkv, 64), nan, device="cuda"))
        ids = self.rng.permutation(n_pages)
        self.free = ids[sum(need):].tolist()
        self.table_np = np.full((self.B, self.max_blocks), -12345, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table_np[b, :n] = ids[at:at + n]
            at += n
        self.table = torch.from_numpy(self.table_np).cuda()
        self.lens = list(lens)
        self.length = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.k, self.v = ([self.draw(n, Hkv, d, by=s) for n in lens] for s in (scale_k, 1.0))
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def draw(self, *shape, by=1.0):
        x = self.torch.from_numpy((by * self.rng.standard_normal(shape)).astype(np.float32)).to(self.dt)
        return x.double().numpy()

    def dev(self, x):
        return self.torch.from_numpy(np.ascontiguousarray(x)).to(self.dt).cuda()

    def ws(self, n):
        return self.torch.full((max(16, n),), 255, dtype=self.torch.uint8, device="cuda")

    def append(self, counts, lens_after, fused=0):
        """Store the tokens lens_after - counts .. lens_after - 1 of every stream."""
        torch = self.torch
        rows = [np.concatenate([x[b][n - c:n] for b, (c, n) in enumerate(zip(counts, lens_after))]) for x in (self.k, self.v)]
        tok = rows[0].shape[0]
        wide = torch.full((max(1, tok), fused + 2 * self.Hkv, self.d), float("nan"), dtype=self.dt, device="cuda")
        wide[:tok, fused:fused + self.Hkv], wide[:tok, fused + self.Hkv:] = self.dev(rows[0]), self.dev(rows[1])
        ptr = torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), device="cuda")
        length = torch.tensor(lens_after, dtype=torch.int32, device="cuda")
        self.fva.fva_cache_append(self.cache, self.table, length, wide[:tok, fused:fused + self.Hkv],
                                  wide[:tok, fused + self.Hkv:], ptr, max(counts), self.st)
        self.ok()

    def fill(self):
        self.append(self.lens, self.lens)
        self.cache.mass.nan_to_num_(nan=0.0)
        return self

    def ok(self, code=0):
        assert int(self.st.item()) == code
        self.st.zero_()

    def query(self, q=None, wide=0):
        """Queries [B, H, d]; `wide`: as a slice of rows with that many more heads."""
        torch = self.torch
        self.q = self.draw(self.B, self.H, self.d) if q is None else q
        x = torch.full((self.B, self.H + wide, self.d), float("nan"), dtype=self.dt, device="cuda")
        x[:, wide:] = self.dev(self.q)
        return x[:, wide:]

    def route(self, q, p, floor, recent, table=None, length=None):
        torch, i32 = self.torch, dict(dtype=self.torch.int32, device="cuda")
        kept = torch.full((self.B, self.Hkv, self.max_blocks), -7, **i32)
        n = torch.full((self.B, self.Hkv), -7, **i32)
        ws = self.ws(self.fva.fva_cache_route_workspace_bytes(self.cache, self.B, self.max_blocks, self.H))
        self.fva.fva_cache_route(self.cache, self.table if table is None else table,
                                 self.length if length is None else length, q, p, floor, recent, kept, n, ws,
                                 dev_status=self.st)
        return kept, n

    def attn(self, q, kept, n, accumulate=False, scale=0.0):
        torch = self.torch
        o = torch.full((self.B, self.H, self.d), float("nan"), dtype=self.dt, device="cuda")
        lse = torch.full((self.B, self.H), float("nan"), device="cuda")
        ws = self.ws(self.fva.fva_cache_attn_workspace_bytes(self.cache, self.B, self.max_blocks, self.H, accumulate))
        self.fva.fva_cache_attn(self.cache, self.table, self.length, q, kept, n, o, ws, lse, scale, accumulate, self.st)
        return o, lse

    # ---- oracle
    def want_route(self, p, floor, recent):
        return [[CO.route(self.q[b, g * self.G:(g + 1) * self.G], CO.block_means(self.k[b][:, g]), p, floor, recent)
                 for g in range(self.Hkv)] for b in range(self.B)]

    def check_route(self, kept, n, want):
        kept, n = kept.cpu().numpy(), n.cpu().numpy()
        for b in range(self.B):
            for g in range(self.Hkv):
                assert n[b, g] == len(want[b][g]), (b, g)
                assert kept[b, g, :n[b, g]].tolist() == want[b][g].tolist()
                assert (kept[b, g, n[b, g]:] == -1).all()

    def check_attn(self, o, lse, blocks, mass_before=None):
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        mass = self.cache.mass.double().cpu().numpy()
        eps = self.torch.finfo(self.dt).eps / 2
        split = 2.0 ** -15 if self.dt != self.torch.float32 else 0.0
        seen = np.zeros(mass.shape, dtype=bool)
        for b in range(self.B):
            for g in range(self.Hkv):
                heads = slice(g * self.G, (g + 1) * self.G)
                q, k, v = self.q[b, heads], self.k[b][:, g], self.v[b][:, g]
                want, l_want, w, at = CO.attention(q, k, v, blocks[b][g])
                if at.size == 0:
                    assert not o[b, heads].any() and np.isneginf(lse[b, heads]).all()
                    continue
                score = (np.abs(q) @ np.abs(k[at]).T).max(1, keepdims=True) / np.sqrt(self.d)
                rel = 2 * (self.d + 16) * U * score + (at.size + 64) * U + 16 * U * np.abs(l_want)[:, None] + split
                limit = eps * np.abs(want) + rel * (w @ np.abs(v[at]))
                if self.dt == self.torch.float16:
                    limit = limit + 2.0 ** -25  # half a step of the subnormal numbers
                assert (np.abs(o[b, heads] - want) <= limit).all(), (b, g, np.abs(o[b, heads] - want).max())
                assert (np.abs(lse[b, heads] - l_want) <= rel[:, 0] + 4 * U * np.abs(l_want)).all(), (b, g)
                if mass_before is not None:
                    page, slot = self.table_np[b, at // 64], at % 64
                    seen[page, g, slot] = True
                    want_m = mass_before[page, g, slot] + w.sum(0)
                    limit = (rel.max() + 4 * U) * w.sum(0) + 2 * U * want_m
                    assert (np.abs(mass[page, g, slot] - want_m) <= limit).all(), (b, g)
        if mass_before is not None:
            assert (mass[~seen] == mass_before[~seen]).all()


# ------------------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype,d,Hkv", [("bf16", 128, 3), ("f16", 64, 2), ("f32", 32, 1), ("f32", 128, 2)])
def test_append_in_pieces(dtype, d, Hkv):
    """Ragged pieces (none, one, up to a page's end, over several pages) leave the same cache as
    one piece: tokens in place, untouched slots untouched, means of whole and partial pages."""
    import torch
    lens = [0, 1, 64, 65, 200, 130]
    s = Streams(lens, Hkv, Hkv, d, dtype)
    steps = [[0, 1, 3, 64, 63, 1], [0, 0, 0, 0, 1, 63], [0, 0, 61, 1, 70, 0], [0, 0, 0, 0, 66, 66]]
    total = np.zeros(6, dtype=int)
    for c in steps:
        total += c
        s.append(c, total.tolist(), fused=5)
    assert total.tolist() == lens
    one = Streams(lens, Hkv, Hkv, d, dtype).fill()
    for x in ("k", "v", "key_mean"):
        a, b = getattr(s.cache, x), getattr(one.cache, x)
        assert torch.equal(a.nan_to_num(nan=-777.0), b.nan_to_num(nan=-777.0)), x
    k, mean, mass = s.cache.k.double().cpu().numpy(), s.cache.key_mean.cpu().numpy(), s.cache.mass.cpu().numpy()
    v = s.cache.v.double().cpu().numpy()
    written = np.zeros(mass.shape[::2], dtype=bool)
    for b, n in enumerate(lens):
        at = np.arange(n)
        page = s.table_np[b, at // 64]
        written[page, at % 64] = True
        assert (k[page, :, at % 64] == s.k[b]).all() and (v[page, :, at % 64] == s.v[b]).all()
        assert (mass[page, :, at % 64] == 0).all()
        for g in range(Hkv):
            want = CO.block_means(s.k[b][:, g])
            got = mean[s.table_np[b, :len(want)], g]
            # sums of 64 values in float64 are exact but for the last bits of wide fp32 values
            assert (got == want).all() if dtype != "f32" else (np.abs(got - want) <= U * np.abs(want)).all()
    assert np.isnan(np.moveaxis(k, 2, 1)[~written]).all() and np.isnan(np.moveaxis(mass, 2, 1)[~written]).all()


def test_append_reports_and_skips():
    """A count above max_new, a count above the length, a page out of range, a length out of
    range: each is reported, the other streams are stored."""
    import torch
    s = Streams([70, 70, 70, 70], 1, 1, 64, "bf16")
    rows = s.dev(np.concatenate(s.k))
    ptr = torch.tensor([0, 70, 140, 210, 280], dtype=torch.int32, device="cuda")

    def go(length, table=s.table, most=70, ptr=ptr):
        s.cache.k.fill_(5)
        s.fva.fva_cache_append(s.cache, table, torch.tensor(length, dtype=torch.int32, device="cuda"), rows, rows, ptr, most,
                               s.st)
        s.ok(s.fva.FVA_DEVERR_BAD_LIST)
        k = s.cache.k.double().cpu().numpy()
        return [bool((k[s.table_np[b, 0], 0] == s.k[b][:64, 0]).all()) for b in range(4)]
    assert go([70, 69, 70, 70]) == [True, False, True, True]
    assert go([70, 70, -1, 70]) == [True, True, False, True]
    bad = s.table.clone()
    bad[1, 0], bad[3, 0] = s.cache.k.shape[0], -1
    assert go([70] * 4, bad) == [True, False, True, False]
    assert go([70] * 4, most=69) == [False] * 4
    assert go([70] * 4, ptr=torch.tensor([0, 70, 140, 210, 281], dtype=torch.int32, device="cuda")) == [True] * 3 + [False]
    assert go([70] * 4, ptr=torch.tensor([-1, 69, 140, 139, 200], dtype=torch.int32, device="cuda"))[0] is False


# ------------------------------------------------------------------------------ routing

@pytest.mark.parametrize("dtype,d,Hkv,G", [("bf16", 128, 2, 4), ("bf16", 64, 1, 1), ("f16", 64, 2, 3), ("f32", 32, 2, 2),
                                           ("f32", 128, 1, 8), ("bf16", 128, 1, 20)])
@pytest.mark.parametrize("p,floor,recent", [(0.9, 2, 1), (0.3, 0, 0), (0.05, 5, 3), (1.0, 0, 0), (0.999, 100, 100)])
def test_route(dtype, d, Hkv, G, p, floor, recent):
    s = Streams([0, 1, 63, 64, 65, 1000, 4097, 2048], Hkv * G, Hkv, d, dtype, scale_k=3.0).fill()
    q = s.query(wide=3)
    kept, n = s.route(q, p, floor, recent)
    s.ok()
    s.check_route(kept, n, s.want_route(p, floor, recent))


def test_route_many_blocks_and_wide_scores():
    """The largest table, and scores so far apart that most shares are 0 (ties by index)."""
    s = Streams([16384 * 64 - 5, 100], 2, 1, 64, "bf16", max_blocks=16384).fill()
    q = s.query()
    kept, n = s.route(q, 0.7, 9, 2)
    s.ok()
    s.check_route(kept, n, s.want_route(0.7, 9, 2))
    s.q = s.q * 512.0
    kept, n = s.route(s.query(s.q), 0.7, 3000, 2)
    s.ok()
    s.check_route(kept, n, s.want_route(0.7, 3000, 2))


def test_route_many_sequences_of_a_wide_table():
    """More units than SMs and a table whose scores do not fit a shared SM's memory."""
    lens = np.random.default_rng(2).integers(0, 700, 100).tolist()
    lens[3] = 64 * 1100 - 3
    s = Streams(lens, 8, 2, 64, "bf16", max_blocks=1200, scale_k=3.0).fill()
    q = s.query()
    kept, n = s.route(q, 0.8, 3, 1)
    s.ok()
    s.check_route(kept, n, s.want_route(0.8, 3, 1))


def test_route_ties_take_the_lowest_blocks():
    s = Streams([64 * 600, 64 * 300 + 5], 2, 2, 64, "bf16")
    for b in range(2):
        s.k[b][:] = 1.0
    s.fill()
    kept, n = s.route(s.query(), 0.25, 0, 2)
    s.ok()
    s.check_route(kept, n, s.want_route(0.25, 0, 2))
    kept, n = s.route(s.query(), 0.01, 40, 0)
    s.check_route(kept, n, s.want_route(0.01, 40, 0))


def test_route_nan_and_bad_pages():
    """A NaN query keeps every block of its group; a table entry that names no page is reported."""
    s = Streams([640, 640], 4, 2, 64, "bf16").fill()
    s.query()
    s.q[0, 1] = np.nan
    kept, n = s.route(s.query(s.q), 0.2, 1, 0)
    s.ok()
    assert n[0].tolist() == [10, int(n[0, 1])] and int(n[0, 1]) < 10 and kept[0, 0, :10].tolist() == list(range(10))
    bad = s.table.clone()
    bad[1, 3] = -1
    s.query(np.ones_like(s.q))
    kept, n = s.route(s.dev(s.q), 0.2, 1, 0, table=bad)
    s.ok(s.fva.FVA_DEVERR_BAD_LIST)
    assert 3 not in kept[1, 0, :int(n[1, 0])].tolist()


# ------------------------------------------------------------------------------ attention

@pytest.mark.parametrize("dtype,d,Hkv,G", [("bf16", 128, 2, 4), ("bf16", 64, 2, 1), ("f16", 128, 1, 2), ("f16", 64, 2, 3),
                                           ("bf16", 128, 1, 16), ("bf16", 64, 1, 20), ("bf16", 128, 1, 40),
                                           ("f32", 32, 2, 2), ("f32", 64, 3, 1), ("f32", 128, 1, 8), ("f32", 128, 1, 17)])
@pytest.mark.parametrize("every", [False, True])
def test_attention(dtype, d, Hkv, G, every):
    """Lengths from none over one to several thousand, routed lists or every block, weights
    added to masses that were there before."""
    s = Streams([0, 1, 63, 64, 65, 700, 4097, 129], Hkv * G, Hkv, d, dtype).fill()
    s.cache.mass.uniform_(0, 3)
    before = s.cache.mass.double().cpu().numpy()
    q = s.query(wide=2)
    if every:
        kept = n = None
        blocks = [[np.arange(-(-m // 64))] * Hkv for m in s.lens]
    else:
        kept, n = s.route(q, 0.6, 2, 1)
        blocks = s.want_route(0.6, 2, 1)
    o, lse = s.attn(q, kept, n, accumulate=True)
    s.ok()
    s.check_attn(o, lse, blocks, before)
    o2, lse2 = s.attn(q, kept, n)
    s.torch.cuda.synchronize()
    assert s.torch.equal(o, o2) and s.torch.equal(lse, lse2)


@pytest.mark.parametrize("B,Hkv,G", [(300, 4, 2), (1, 1, 8), (2000, 1, 1), (3, 1, 128)])
def test_attention_many_and_few_units(B, Hkv, G):
    """More sequences than CTAs and a single long one: shares that hold many units, units that
    cross many shares."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 200, B).tolist() if B > 1 else [50001]
    s = Streams(lens, Hkv * G, Hkv, 64, "bf16").fill()
    before = s.cache.mass.double().cpu().numpy()
    q = s.query()
    o, lse = s.attn(q, None, None, accumulate=True)
    s.ok()
    s.check_attn(o, lse, [[np.arange(-(-m // 64))] * Hkv for m in s.lens], before)


def test_attention_of_empty_streams():
    s = Streams([0, 0, 0], 4, 2, 128, "bf16", spare=1)
    q = s.query()
    kept, n = s.route(q, 0.5, 3, 2)
    assert not n.any() and bool((kept == -1).all())
    o, lse = s.attn(q, kept, n, accumulate=True)
    s.ok()
    assert not o.any() and bool(lse.isneginf().all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_attention_nan_stays_in_its_head(dtype):
    """A NaN in one query head makes that head's output and log-sum-exp NaN, over one share and
    over many, and leaves its neighbours alone."""
    for length in (100, 30000):
        s = Streams([length, 300], 4, 2, 64, dtype).fill()
        s.query()
        clean = s.attn(s.dev(s.q), None, None)
        s.q[0, 1, 5] = np.nan
        o, lse = s.attn(s.dev(s.q), None, None)
        s.ok()
        assert bool(o[0, 1].isnan().all()) and bool(lse[0, 1].isnan())
        rest = [(0, 0), (0, 2), (0, 3), (1, 0), (1, 1), (1, 2), (1, 3)]
        assert all(s.torch.equal(o[i], clean[0][i]) and s.torch.equal(lse[i], clean[1][i]) for i in rest)


def test_attention_without_masses():
    s = Streams([500, 20], 4, 2, 64, "bf16").fill()
    c = s.cache
    s.cache = s.fva.Cache(c.k, c.v, c.key_mean)
    q = s.query()
    o, lse = s.attn(q, None, None)
    s.ok()
    s.cache = c
    s.check_attn(o, lse, [[np.arange(8)] * 2, [np.arange(1)] * 2])
    s.cache = s.fva.Cache(c.k, c.v, c.key_mean)
    with pytest.raises(s.fva.FvaError):
        s.attn(q, None, None, accumulate=True)


def test_attention_large_scores():
    """Scores of some hundreds: the running maximum moves, nothing overflows."""
    s = Streams([3000, 257], 4, 1, 128, "bf16", scale_k=40.0).fill()
    q = s.query()
    o, lse = s.attn(q, None, None)
    s.ok()
    s.check_attn(o, lse, [[np.arange(-(-m // 64))] for m in s.lens])


def test_attention_bad_entries_are_reported_and_skipped():
    s = Streams([640, 640], 4, 2, 64, "bf16").fill()
    q = s.query()
    torch = s.torch
    kept = torch.full((2, 2, s.max_blocks), -1, dtype=torch.int32, device="cuda")
    kept[:, :, :3] = torch.tensor([1, 4, 7], dtype=torch.int32)
    kept[0, 1, 1], kept[1, 0, 2] = 10, -4
    n = torch.full((2, 2), 3, dtype=torch.int32, device="cuda")
    o, lse = s.attn(q, kept, n)
    s.ok(s.fva.FVA_DEVERR_BAD_LIST)
    three, two = np.array([1, 4, 7]), [np.array([1, 7]), np.array([1, 4])]
    s.check_attn(o, lse, [[three, two[0]], [two[1], three]])
    n[0, 0] = 99
    s.attn(q, kept, n)
    s.ok(s.fva.FVA_DEVERR_BAD_LIST)
    n[0, 0] = -1
    o, lse = s.attn(q, kept, n)
    s.ok(s.fva.FVA_DEVERR_BAD_LIST)
    s.check_attn(o, lse, [[np.zeros(0, int), two[0]], [two[1], three]])


def test_attention_rows_that_share_pages():
    """Two query rows over one sequence (the table row twice): both weights are added."""
    s = Streams([500], 4, 2, 64, "bf16").fill()
    s.table_np = np.repeat(s.table_np, 2, 0)
    s.table, s.length = s.table.repeat(2, 1), s.length.repeat(2)
    s.k, s.v, s.B, s.lens = s.k * 2, s.v * 2, 2, s.lens * 2
    q = s.query()
    s.attn(q, None, None, accumulate=True)
    s.ok()
    w = sum(CO.attention(s.q[b, :2], s.k[b][:, 0], s.v[b][:, 0], np.arange(8))[2].sum(0) for b in range(2))
    got = s.cache.mass.double().cpu().numpy()[s.table_np[0, np.arange(500) // 64], 0, np.arange(500) % 64]
    assert np.abs(got - w).max() <= 1e-5 * w.max()


def test_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 and 2^32 bytes of the buffers."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import fva
    s = Streams([200, 70], 4, 2, 128, "bf16")
    n_pages = 140000  # x 2 x 64 x 128 x 2 bytes = 4.6 GB a buffer, 2.3e9 elements
    s.cache = fva.Cache(*(torch.empty((n_pages, 2, 64, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)),
                        torch.empty((n_pages, 2, 128), device="cuda"), torch.zeros((n_pages, 2, 64), device="cuda"))
    s.table_np[0, :4] = [n_pages - 1, n_pages - 9, 132000, 3]
    s.table_np[1, :2] = [n_pages - 3, 131071]
    s.table = torch.from_numpy(s.table_np).cuda()
    s.append(s.lens, s.lens)
    before = np.zeros((n_pages, 2, 64))
    q = s.query()
    kept, n = s.route(q, 0.5, 2, 1)
    s.check_route(kept, n, s.want_route(0.5, 2, 1))
    o, lse = s.attn(q, kept, n, accumulate=True)
    s.ok()
    s.check_attn(o, lse, s.want_route(0.5, 2, 1), before)
    _evict(s, 100, 2, 10, np.array([[n_pages - 20, 139000], [5, n_pages - 30]]))


# ------------------------------------------------------------------------------ eviction

def _evict(s, keep, sink, recent, dst=None, code=0):
    torch = s.torch
    room = -(-keep // 64)
    if dst is None:
        dst = np.array(s.free[:room * s.B]).reshape(s.B, room)
    mass = s.cache.mass.cpu().numpy()
    at = [np.arange(n) for n in s.lens]
    w = [[mass[s.table_np[b, x // 64], g, x % 64] for g in range(s.Hkv)] for b, x in enumerate(at)]
    snap = [x.clone() for x in (s.cache.k, s.cache.v, s.cache.mass)]
    kept = torch.full((s.B, s.Hkv, keep), -7, dtype=torch.int32, device="cuda")
    new_len = torch.full((s.B,), -7, dtype=torch.int32, device="cuda")
    ws = s.ws(s.fva.fva_cache_evict_workspace_bytes(s.cache, s.B, s.max_blocks))
    s.fva.fva_cache_evict(s.cache, s.table, s.length, keep, sink, recent, torch.from_numpy(dst.astype(np.int32)).cuda(), kept,
                          new_len, ws, s.st)
    s.ok(code)
    kept, new_len = kept.cpu().numpy(), new_len.cpu().numpy()
    touched = torch.zeros(s.cache.k.shape[:3:2], dtype=torch.bool, device="cuda")
    for b in range(s.B):
        m = min(keep, s.lens[b])
        assert new_len[b] == m
        for g in range(s.Hkv):
            want = CO.evict(w[b][g], keep, sink, recent)
            assert kept[b, g, :m].tolist() == want.tolist(), (b, g)
            assert (kept[b, g, m:] == -1).all()
            to = np.arange(m)
            page = torch.from_numpy(dst[b, to // 64].astype(np.int64)).cuda()
            slot = torch.from_numpy(to % 64).cuda()
            touched[page, slot] = True
            assert (s.cache.k[page, g, slot].double().cpu().numpy() == s.k[b][want, g]).all()
            assert (s.cache.v[page, g, slot].double().cpu().numpy() == s.v[b][want, g]).all()
            np.testing.assert_array_equal(s.cache.mass[page, g, slot].cpu().numpy(), w[b][g][want])
            means = CO.block_means(s.k[b][want, g])
            got = s.cache.key_mean[torch.from_numpy(dst[b, :len(means)].astype(np.int64)).cuda(), g].cpu().numpy()
            assert (np.abs(got - means) <= (U if s.dt == torch.float32 else 0) * np.abs(means)).all()
    for x, y in zip((s.cache.k, s.cache.v, s.cache.mass), snap):  # nothing else was written
        same = torch.eq(x, y) | (x.isnan() & y.isnan())
        same = same.flatten(3).all(3) if x.dim() == 4 else same
        assert bool((same | touched[:, None]).all())


@pytest.mark.parametrize("dtype,d,Hkv", [("bf16", 128, 2), ("f16", 64, 1), ("f32", 32, 3)])
@pytest.mark.parametrize("keep,sink,recent", [(100, 4, 16), (64, 0, 0), (1, 0, 0), (1, 1, 0), (130, 65, 65), (700, 4, 300),
                                              (5000, 4, 64)])
def test_evict(dtype, d, Hkv, keep, sink, recent):
    s = Streams([0, 1, 64, 65, 701, 3001], Hkv, Hkv, d, dtype, spare=6 * -(-keep // 64)).fill()
    s.cache.mass.copy_(s.torch.from_numpy(np.exp(s.rng.standard_normal(tuple(s.cache.mass.shape)) * 3).astype(np.float32)))
    _evict(s, keep, sink, recent)


@pytest.mark.parametrize("values", [[0.0], [0.0, -0.0], [1.0, 2.0], [0.0, float("nan")], [float("nan")],
                                    [float("inf"), 1e-45, 0.0, -1.0]])
def test_evict_ties_and_odd_weights(values):
    s = Streams([1500, 400], 2, 2, 64, "bf16", spare=14).fill()
    pick = s.rng.choice(np.array(values, dtype=np.float32), tuple(s.cache.mass.shape))
    s.cache.mass.copy_(s.torch.from_numpy(pick))
    _evict(s, 400, 3, 50)


def test_evict_long_stream():
    s = Streams([40001], 2, 2, 64, "bf16", spare=200).fill()
    s.cache.mass.uniform_(0, 1)
    s.cache.mass *= (s.cache.mass > 0.4)
    _evict(s, 12345, 4, 1000)


@pytest.mark.parametrize("lens,max_blocks", [([40001] + [70] * 79, None), ([5000, 64, 3], 16384)])
def test_evict_many_units_and_wide_tables(lens, max_blocks):
    """A long stream in one CTA (more units than SMs), and tokens that are read again in every
    pass (a table too wide for shared memory)."""
    keep = 1234
    s = Streams(lens, 1, 1, 64, "bf16", max_blocks=max_blocks, spare=len(lens) * -(-keep // 64)).fill()
    s.cache.mass.uniform_(0, 1)
    s.cache.mass *= (s.cache.mass > 0.4)
    _evict(s, keep, 4, 100)


def test_evict_reports_destinations_that_cannot_be():
    """A destination that is a source page of its sequence, or no page, is reported and not
    written; nothing else than the good destinations changes."""
    s = Streams([200, 200], 1, 1, 64, "bf16", spare=8).fill()
    before = s.cache.k.clone()
    dst = np.array([[s.free[0], s.table_np[0, 2]], [10 ** 6, s.free[1]]], dtype=np.int32)
    torch = s.torch
    kept = torch.empty((2, 1, 128), dtype=torch.int32, device="cuda")
    s.fva.fva_cache_evict(s.cache, s.table, s.length, 128, 0, 0, torch.from_numpy(dst).cuda(), kept,
                          torch.empty(2, dtype=torch.int32, device="cuda"),
                          s.ws(s.fva.fva_cache_evict_workspace_bytes(s.cache, 2, s.max_blocks)), s.st)
    s.ok(s.fva.FVA_DEVERR_BAD_LIST)
    for page in range(before.shape[0]):
        same = bool((s.cache.k[page].view(torch.int16) == before[page].view(torch.int16)).all())
        assert same == (page not in (s.free[0], s.free[1]))


# ------------------------------------------------------------------------------ together

def test_binding_refuses_mismatched_tensors():
    s = Streams([100], 2, 1, 64, "bf16").fill()
    torch = s.torch
    q = s.query()
    kept, n = s.route(q, 0.5, 1, 1)
    with pytest.raises(ValueError):
        s.attn(q.float(), kept, n)
    with pytest.raises(ValueError):
        s.attn(q, kept.long(), n)
    with pytest.raises(ValueError):
        s.attn(q, kept[:, :, :1], n)
    with pytest.raises(ValueError):
        s.attn(q.cpu(), kept, n)
    with pytest.raises(ValueError):
        s.fva.fva_cache_attn(s.cache, s.table, s.length, q, kept, n, torch.empty_like(q), torch.empty(1 << 24, dtype=torch.uint8))
    with pytest.raises(ValueError):
        s.fva.fva_cache_attn(s.cache, s.table, s.length, q, kept, n, torch.empty_like(q), s.ws(1 << 24),
                             dev_status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(s.fva.FvaError):
        s.fva.fva_cache_attn(s.cache, s.table, s.length, q, kept, None, torch.empty_like(q), s.ws(1 << 24))
    with pytest.raises(ValueError):
        s.fva.Cache(s.cache.k, s.cache.v[:, :, :32], s.cache.key_mean)


def test_route_and_attention_on_another_stream_and_captured():
    """The same calls on a side stream, and captured once and replayed with new queries."""
    import torch
    s = Streams([0, 300, 1000], 4, 2, 128, "bf16").fill()
    a, b = s.query(), s.dev(s.draw(3, 4, 128))
    i32 = dict(dtype=torch.int32, device="cuda")
    kept, n = torch.empty((3, 2, s.max_blocks), **i32), torch.empty((3, 2), **i32)
    o, q = torch.empty_like(a), a.clone()
    rw = s.ws(s.fva.fva_cache_route_workspace_bytes(s.cache, 3, s.max_blocks, 4))
    aw = s.ws(s.fva.fva_cache_attn_workspace_bytes(s.cache, 3, s.max_blocks, 4, False))

    def step():
        s.fva.fva_cache_route(s.cache, s.table, s.length, q, 0.6, 2, 1, kept, n, rw, dev_status=s.st)
        s.fva.fva_cache_attn(s.cache, s.table, s.length, q, kept, n, o, aw, dev_status=s.st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    want = {}
    for name, x in (("a", a), ("b", b)):
        k2, n2 = s.route(x, 0.6, 2, 1)
        want[name] = s.attn(x, k2, n2)[0]
    assert torch.equal(o, want["a"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for name, x in (("b", b), ("a", a), ("b", b)):
        q.copy_(x)
        o.fill_(float("nan"))
        g.replay()
        assert torch.equal(o, want[name])
    s.ok()


def test_streams_served_together():
    """CachedAttention as a program uses it: prompts, decoding steps with attention, an eviction,
    more steps; every step's outputs and choices against the oracle on the host's own copy."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import pipeline
    B, H, Hkv, d, rng = 3, 4, 2, 64, np.random.default_rng(8)
    att = pipeline.CachedAttention(B, H, Hkv, d, n_pages=40, max_blocks=16, p=0.8, k_floor=2, n_recent=1)
    bf = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16()  # noqa: E731
    ks, vs = ([[np.zeros((0, d)) for _ in range(Hkv)] for _ in range(B)] for _ in range(2))
    mass = [[np.zeros(0) for _ in range(Hkv)] for _ in range(B)]

    def add(counts):
        k, v = bf(sum(counts), Hkv, d), bf(sum(counts), Hkv, d)
        att.append(k.cuda(), v.cuda(), counts)
        at = 0
        for b, c in enumerate(counts):
            for g in range(Hkv):
                ks[b][g] = np.concatenate([ks[b][g], k[at:at + c, g].double().numpy()])
                vs[b][g] = np.concatenate([vs[b][g], v[at:at + c, g].double().numpy()])
                mass[b][g] = np.concatenate([mass[b][g], np.zeros(c)])
            at += c

    def step():
        add([1] * B)
        q = bf(B, H, d)
        o = att.attend(q.cuda(), torch.empty((B, H, d), dtype=torch.bfloat16, device="cuda")).double().cpu().numpy()
        kept, n = att.kept.cpu().numpy(), att.n_kept.cpu().numpy()
        for b in range(B):
            for g in range(Hkv):
                qg = q[b, 2 * g:2 * g + 2].double().numpy()
                want = CO.route(qg, CO.block_means(ks[b][g]), 0.8, 2, 1)
                assert kept[b, g, :n[b, g]].tolist() == want.tolist()
                ow, _, w, at = CO.attention(qg, ks[b][g], vs[b][g], want)
                mass[b][g][at] += w.sum(0)
                # eps / 2 of a bf16 output, and 2^-14 of the values for the weights
                assert (np.abs(o[b, 2 * g:2 * g + 2] - ow) <= 2.0 ** -8 * np.abs(ow) + 2.0 ** -14 * (w @ np.abs(vs[b][g][at]))).all()

    add([5, 300, 640])
    for _ in range(3):
        step()
    kept = att.evict(200, 2, 20).cpu().numpy()
    for b in range(B):
        n = min(200, len(ks[b][0]))
        for g in range(Hkv):
            idx = kept[b, g, :n]
            assert (np.diff(idx) > 0).all() and (kept[b, g, n:] == -1).all()
            if len(ks[b][g]) > 200:  # no left-out token weighs more than a kept one, but for rounding
                out = np.setdiff1d(np.arange(len(ks[b][g])), idx)
                middle = idx[(idx >= 2) & (idx < len(ks[b][g]) - 20)]
                assert mass[b][g][out].max() <= mass[b][g][middle].min() + 1e-5
            ks[b][g], vs[b][g], mass[b][g] = ks[b][g][idx], vs[b][g][idx], mass[b][g][idx]
    assert len(att.free) == 40 - sum(len(p) for p in att.pages) and len(set(att.free)) == len(att.free)
    for _ in range(2):
        step()
    assert int(att.dev_status.item()) == 0
    with pytest.raises(RuntimeError):
        add([64 * 15 - 6, 700, 700])
    with pytest.raises(ValueError):
        add([64 * 16, 0, 0])


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("H,Hkv,d,dtype", [(8, 2, 128, "bf16"), (20, 1, 64, "f16"), (3, 3, 32, "f32"), (8, 2, 128, "f32")])
def test_wait_that_runs_out_is_reported(H, Hkv, d, dtype, accumulate):
    """With the loads withheld and a 20 ms limit the attention reports a timeout, ends and leaves
    the device usable; the next call is right."""
    s = Streams([700, 64, 0, 5000], H, Hkv, d, dtype).fill()
    q = s.query()
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


@pytest.mark.parametrize("limit", [1, 2000, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_short_wait_limits_end(dtype, limit):
    """Whatever waits run out, in some of the warps or none, the calls end and the next is right."""
    s = Streams([3000, 1000, 1, 20000], 8, 2, 128, dtype).fill()
    q = s.query()
    want = s.attn(q, None, None)
    s.ok()
    s.fva.fva_set_diagnostics(limit, 0)
    try:
        for _ in range(20):
            s.attn(q, None, None, accumulate=True)
            assert int(s.st.item()) in (0, s.fva.FVA_DEVERR_TIMEOUT)
    finally:
        s.fva.fva_set_diagnostics(0, 0)
    s.st.zero_()
    got = s.attn(q, None, None)
    s.ok()
    assert all(bool((a == b).all()) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[70], [40000]])  # one CTA, and a unit that crosses shares
def test_scores_of_minus_infinity_weigh_nothing(dtype, lens):
    """Heads whose every score is -infinity give 0 and -infinity and add nothing to the masses."""
    import torch
    s = Streams(lens, 2, 1, 64, dtype)
    inf = float("-inf")
    s.k[0][:, 0, 0] = inf
    s.fill()
    q = np.abs(s.draw(1, 2, 64))
    q[:, 0, 0], q[:, 1, 0] = 1.0, 1.0
    o, lse = s.attn(s.query(q), None, None, accumulate=True)
    s.ok()
    pages = torch.from_numpy(s.table_np[0, :-(-lens[0] // 64)].astype(np.int64)).cuda()
    assert bool((o == 0).all()) and bool((lse == inf).all()) and bool((s.cache.mass[pages] == 0).all())


def test_append_refuses_overlapping_rows_and_wrapped_ranges():
    import torch
    s = Streams([100, 80], 2, 1, 64, "bf16")
    one = torch.zeros((1, 1, 64), dtype=s.dt, device="cuda")
    ptr = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    with pytest.raises(s.fva.FvaError):  # an expanded row has stride 0
        s.fva.fva_cache_append(s.cache, s.table, s.length, one.expand(40, 1, 64), one.expand(40, 1, 64), ptr, 20, s.st)
    x = torch.zeros((40, 1, 64), dtype=s.dt, device="cuda")
    for a, b in ((2 ** 31 - 1, -2 ** 31), (30, 10), (-5, 10)):  # differences of 1 (wrapped), -20 and 15
        ptr = torch.tensor([a, b, b], dtype=torch.int32, device="cuda")
        s.fva.fva_cache_append(s.cache, s.table, s.length, x, x, ptr, 20, s.st)
        s.ok(s.fva.FVA_DEVERR_BAD_LIST)
    assert bool(s.cache.k.isnan().all()) and bool(s.cache.key_mean.isnan().all())


def test_refused_calls_leave_the_streams_as_they_were():
    """CachedAttention: a refused append or eviction takes no page and changes no length."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import pipeline
    att = pipeline.CachedAttention(2, 4, 2, 64, n_pages=12, max_blocks=8)
    x = torch.randn(100, 2, 64, device="cuda").bfloat16()
    att.append(x, x, [70, 30])
    state = lambda: (sorted(att.free), [list(p) for p in att.pages], list(att.lengths), att.length.tolist(),  # noqa: E731
                     att.table[0, :2].tolist(), att.table[1, :1].tolist())
    before = state()
    with pytest.raises(ValueError):
        att.append(x.float(), x.float(), [60, 40])
    with pytest.raises(ValueError):
        att.append(x, x[:, :1], [60, 40])
    with pytest.raises(ValueError):
        att.append(x, x, [60, 30])
    wide = torch.randn(100 * 130 + 8, device="cuda").bfloat16()[:100 * 130].view(100, 130)[:, :128].unflatten(1, (2, 64))
    with pytest.raises(RuntimeError):  # rows that start on 4-byte boundaries
        att.append(wide, wide, [60, 40])
    for keep, sink, recent in ((0, 0, 0), (-1, 0, 0), (10, 6, 5), (10, -1, 0), ((1 << 20) + 1, 0, 0)):
        with pytest.raises(ValueError):
            att.evict(keep, sink, recent)
    assert state() == before
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    first = att.attend(q, torch.empty_like(q))
    att.append(x[:0], x[:0], [0, 0])
    assert torch.equal(att.attend(q, torch.empty_like(q)), first)
    assert int(att.dev_status.item()) == 0
    att.evict(1 << 20, 0, 0)  # a budget above every length moves the tokens and keeps them all
    assert att.lengths == before[2] and torch.equal(att.attend(q, torch.empty_like(q)), first)


def test_captured_eviction_and_append_are_replayed():
    """Append and eviction captured into one graph: every replay does what the calls would."""
    import torch
    s = Streams([500, 130], 2, 2, 64, "bf16", spare=12).fill()
    i32 = dict(dtype=torch.int32, device="cuda")
    dst = torch.tensor([s.free[:2], s.free[2:4]], **i32)
    kept, new_len, ws = torch.empty((2, 2, 100), **i32), torch.empty(2, **i32), s.ws(s.fva.fva_cache_evict_workspace_bytes(s.cache, 2, s.max_blocks))
    x = torch.zeros((2, 2, 64), dtype=s.dt, device="cuda")
    ptr = torch.tensor([0, 1, 2], **i32)
    after = torch.tensor([101, 101], **i32)

    def step():
        s.fva.fva_cache_evict(s.cache, s.table, s.length, 100, 2, 10, dst, kept, new_len, ws, dev_status=s.st)
        s.fva.fva_cache_append(s.cache, dst, after, x, x, ptr, 1, s.st)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    pages = torch.from_numpy(s.table_np[0, :8].astype(np.int64)).cuda()
    for seed in range(3):
        torch.manual_seed(seed)
        s.cache.mass[pages] = torch.rand(8, 2, 64, device="cuda")
        x.copy_(torch.randn(2, 2, 64, device="cuda"))
        step()
        want = [t.clone() for t in (kept, new_len, s.cache.k[dst[0].long()], s.cache.key_mean[dst[1].long()])]
        for t in (kept, new_len):
            t.zero_()
        s.cache.k[dst.flatten().long()] = 0
        g.replay()
        got = [kept, new_len, s.cache.k[dst[0].long()], s.cache.key_mean[dst[1].long()]]
        rows = [slice(None), slice(None), slice(None), slice(None)]
        for a, b, r in zip(got, want, rows):
            a, b = a[r].reshape(-1), b[r].reshape(-1)
            if a.dtype.is_floating_point:  # the slots behind the 101 tokens are nobody's
                a, b = a[:64 * 64], b[:64 * 64]
            assert torch.equal(a, b)
    s.ok()


@pytest.mark.parametrize("H,Hkv,d,dtype", [(4, 4, 64, "bf16"), (16, 2, 128, "bf16"), (33, 1, 64, "f16"), (6, 2, 32, "f32"),
                                           (20, 1, 128, "f32"), (2, 2, 64, "f32")])
@pytest.mark.parametrize("lens", [[0], [1], [64, 0, 65], [1023, 200, 1], [1024] * 5, [63 + 64 * i for i in range(16)]])
def test_small_calls_in_one_launch(H, Hkv, d, dtype, lens):
    """Calls that accumulate nothing and whose lists are short: parts of a list may be empty, and a
    sequence longer or shorter than its cluster has CTAs. Also with a kept list, and captured."""
    import torch
    s = Streams(lens, H, Hkv, d, dtype, seed=len(lens)).fill()
    q = s.query()
    o, lse = s.attn(q, None, None)
    s.ok()
    s.check_attn(o, lse, [[np.arange(-(-n // 64))] * Hkv for n in lens])
    kept, n = s.route(q, 0.5, 1, 1)
    o, lse = s.attn(q, kept, n)
    s.ok()
    s.check_attn(o, lse, s.want_route(0.5, 1, 1))
    out = torch.full_like(o, float("nan"))
    ws = s.ws(s.fva.fva_cache_attn_workspace_bytes(s.cache, s.B, s.max_blocks, H, False))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.fva.fva_cache_attn(s.cache, s.table, s.length, q, kept, n, out, ws)
    g.replay()
    assert torch.equal(out, o)


def test_evict_among_very_many_pages():
    """More pages than the destination check holds at a time: a clash among the last ones is
    found, and the rows of far pages (offsets beyond 32 bits) arrive where they should."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import fva
    n_pages, d = 600_000, 64
    cache = fva.Cache.allocate(n_pages, 1, d)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[599_999, 10, 530_000, 524_288]], **i32)
    length, st = torch.tensor([200], **i32), torch.zeros(1, **i32)
    x = torch.randn(200, 1, d, device="cuda").bfloat16()
    y = torch.randn(200, 1, d, device="cuda").bfloat16()
    fva.fva_cache_append(cache, table, length, x, y, torch.tensor([0, 200], **i32), 200, st)
    cache.mass[table[0].long()] = torch.rand(4, 1, 64, device="cuda")
    before = cache.k[524_288].clone()
    kept, new_len = torch.empty((1, 1, 128), **i32), torch.empty(1, **i32)
    ws = torch.empty(fva.fva_cache_evict_workspace_bytes(cache, 1, 4), dtype=torch.uint8, device="cuda")
    for dst, code in (([524_288, 599_998], fva.FVA_DEVERR_BAD_LIST), ([524_287, 599_998], 0)):
        fva.fva_cache_evict(cache, table, length, 128, 2, 8, torch.tensor([dst], **i32), kept, new_len, ws, dev_status=st)
        assert int(st.item()) == code
        st.zero_()
        at = kept[0, 0].long()
        assert torch.equal(cache.k[599_998, 0], x[at[64:], 0]) and torch.equal(cache.v[599_998, 0], y[at[64:], 0])
        assert torch.equal(cache.k[524_288], before)
    assert torch.equal(cache.k[524_287, 0], x[at[:64], 0]) and torch.equal(cache.v[524_287, 0], y[at[:64], 0])
