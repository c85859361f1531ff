"""How exact the fp32 cache attention is: its error against 64 bits, next to that of the same sums in
fp32 in a stated order.

The kernel's own roundings beside the compared sums: exp2f is off by two units in the last place at
most (2^-22 of a weight, independent of its neighbours'), and a division and a few joins add 2^-24 each.

Both errors are samples. A row's squared error is sum_jk w_j w_k e_j e_k (v_j - o)(v_k - o) over its tokens, with
independent e. For normal v its mean is E = d sum w^2 var(e); the terms j = k have the variance
2 E^2 sum w^4 / (sum w^2)^2 at most (normal e), the others 2 E^2 / d. So over rows the sum S of the squared
errors has a relative variance of r = sum E^2 (2 / d + 2 sum w^4 / (sum w^2)^2) / (sum E)^2, and the ratio of two
such errors, square roots of two S, a standard deviation of sqrt(2 r) / 2: four of them are allowed."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _pages(lens):
    import torch
    need = [-(-n // 64) for n in lens]
    ids = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), sum(need)


def _attn(cache, table, length, q):
    import torch
    from adaptive_block_sparse_hilbert_b200 import fva
    B, H, _ = q.shape
    o, st = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(fva.fva_cache_attn_workspace_bytes(cache, B, table.shape[1], H, False), dtype=torch.uint8, device="cuda")
    fva.fva_cache_attn(cache, table, length, q, None, None, o, ws, dev_status=st)
    assert int(st.item()) == 0
    return o.double()


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16, 20])
def test_scores(G, d):
    """Scores some units apart (a part of the blocks lies along the query). Compared sums: a score as
    two halves of the channels, each of two sums over every second channel."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import fva
    lens = [6288, 9001, 19426]
    table, length, n_pages = _pages(lens)
    g = torch.Generator(device="cuda").manual_seed(d + G)
    randn = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    k, v = randn(n_pages, 1, 64, d), randn(n_pages, 1, 64, d)
    way = randn(d)
    way /= way.norm()
    k[torch.rand(n_pages, device="cuda", generator=g) < 0.3] += 4 * way
    q = 2 * math.sqrt(d) * way + randn(3, G, d)
    cache = fva.Cache(k, v, torch.zeros(n_pages, 1, d, device="cuda"))
    o = _attn(cache, table, length, q)
    err, sim, norm, mean, var = 0.0, 0.0, 0.0, 0.0, 0.0
    scale = torch.tensor(1 / math.sqrt(d)).float() * 1.4426950408889634  # of log2 units
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        kd, vd = (x[table[b, at // 64].long(), 0, at % 64].double() for x in (k, v))
        w = torch.softmax(q[b].double() @ kd.T / math.sqrt(d), 1)
        want, w2, w4 = w @ vd, w.square().sum(1), w.pow(4).sum(1)
        mean, var = mean + float(w2.sum()), var + float((w2.square() * (2 / d + 2 * w4 / w2.square())).sum())
        qs = (q[b] * scale.item()).double()
        parts = qs.view(G, 1, 2, d // 4, 2) * kd.view(1, n, 2, d // 4, 2)  # [head, key, half, step, sum]
        acc = torch.zeros(G, n, 2, 2, device="cuda")
        for i in range(d // 4):
            acc = (acc.double() + parts[:, :, :, i]).float()
        s = acc.sum(3).sum(2)
        near = torch.softmax(s.double() * math.log(2), 1) @ vd
        err, sim, norm = err + float((o[b] - want).square().sum()), sim + float((near - want).square().sum()), norm + float(want.square().sum())
    err, sim = math.sqrt(err / norm), math.sqrt(sim / norm)
    factor = 1 + 4 * math.sqrt(2 * var) / mean / 2
    print(f"kernel {err:.2e}, compared sums {sim:.2e}, factor {factor:.2f}")
    assert err <= factor * math.sqrt(sim ** 2 + 2.0 ** -44)


def test_sums_of_values():
    """Long lists inside one share: more units than CTAs, 20 thousand tokens each, all of weight 1 (no
    error in scores or weights). Compared sums: four warps' 16 keys of every block, four at a time. 12,800 independent outputs: four
    standard deviations of the errors' ratio are 4 sqrt(2 / 12800) = 0.05."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import fva
    B, n, d = 400, 20001, 32
    table, length, n_pages = _pages([n] * B)
    g = torch.Generator(device="cuda").manual_seed(5)
    k = torch.zeros(n_pages, 1, 64, d, device="cuda")
    v = torch.randn(n_pages, 1, 64, d, device="cuda", generator=g)
    o = _attn(fva.Cache(k, v, torch.zeros(n_pages, 1, d, device="cuda")), table, length, torch.ones(B, 1, d, device="cuda"))[:, 0]
    nB = table.shape[1]
    valid = (torch.arange(nB * 64, device="cuda") < n).view(nB, 4, 4, 4, 1)
    total, near = torch.zeros(B, d, dtype=torch.float64, device="cuda"), torch.zeros(B, 4, d, device="cuda")
    for i in range(nB):
        x = v[table[:, i].long(), 0].double().view(B, 4, 4, 4, d) * valid[i]  # [sequence, warp, four, key, channel]
        total += x.sum((1, 2, 3))
        for j in range(4):
            near = near + x[:, :, j].sum(2).float()
    want = total / n
    rel = lambda x: float((x - want).norm() / want.norm())  # noqa: E731
    err, sim = rel(o), rel(near.sum(1).double() / n)
    print(f"kernel {err:.2e}, compared sums {sim:.2e}")
    assert err <= 1.05 * math.sqrt(sim ** 2 + 2.0 ** -44)
