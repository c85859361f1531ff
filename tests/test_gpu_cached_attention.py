"""CachedAttention on the device where pages are scarce: its own tables and kernels together."""
import numpy as np
import pytest

from oracle import cache_oracle as CO

pytestmark = pytest.mark.gpu


def test_evict_with_few_pages_left():
    """Streams within the budget stay where they are; the others are cut in turn, each into pages
    that the one before has left; attention over the outcome against the oracle."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import pipeline
    lens, keep, Hkv, d = [700, 90, 1300, 1000, 128], 128, 2, 64
    n_pages = sum(-(-n // 64) for n in lens) + 2
    att = pipeline.CachedAttention(5, 4, Hkv, d, n_pages=n_pages, max_blocks=32, p=1.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(sum(lens), Hkv, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    att.append(k, v, lens)
    att.cache.mass.copy_(torch.rand(att.cache.mass.shape, device="cuda", generator=g))
    mass = att.cache.mass.cpu().numpy()
    start = np.concatenate([[0], np.cumsum(lens)])
    pages = [list(p) for p in att.pages]
    kept = att.evict(keep, 2, 20).cpu().numpy()
    assert att.pages[1] == pages[1] and att.pages[4] == pages[4] and att.lengths == [128, 90, 128, 128, 128]
    assert sorted(att.free + sum(att.pages, [])) == list(range(n_pages)) and att.length.tolist() == att.lengths
    q = torch.randn(5, 4, d, device="cuda", generator=g).bfloat16()
    o = att.attend(q, torch.empty_like(q)).double().cpu().numpy()
    assert int(att.dev_status.item()) == 0
    for b, n in enumerate(lens):
        at = np.arange(n)
        for h in range(Hkv):
            want = CO.evict(mass[np.array(pages[b])[at // 64], h, at % 64], keep, 2, 20)
            assert kept[b, h].tolist() == want.tolist() + [-1] * (keep - len(want))
            kh, vh = (x[start[b]:start[b + 1], h].double().cpu().numpy()[want] for x in (k, v))
            ow, _, w, _ = CO.attention(q[b, 2 * h:2 * h + 2].double().cpu().numpy(), kh, vh, np.arange(-(-len(want) // 64)))
            # eps / 2 of a bf16 output, and 2^-14 of the values for the weights
            assert (np.abs(o[b, 2 * h:2 * h + 2] - ow) <= 2.0 ** -8 * np.abs(ow) + 2.0 ** -14 * (w @ np.abs(vh))).all()


def test_attend_captured_once_and_replayed_between_changes():
    """One captured attend() serves the streams through appends (new pages among them) and evictions,
    the partial kind too: every replay gives what the call would."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import pipeline
    att = pipeline.CachedAttention(3, 8, 2, 128, n_pages=40, max_blocks=16, p=0.7, accumulate=False)
    g = torch.Generator(device="cuda").manual_seed(4)
    rows = lambda n: torch.randn(n, 2, 128, device="cuda", generator=g).bfloat16()  # noqa: E731
    att.append(rows(700), rows(700), [0, 100, 600])
    q = torch.randn(3, 8, 128, device="cuda", generator=g).bfloat16()
    o, want = torch.empty_like(q), torch.empty_like(q)
    att.attend(q, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att.attend(q, o)
    changes = [lambda: att.append(rows(3), rows(3), [1, 1, 1]), lambda: att.append(rows(300), rows(300), [130, 170, 0]),
               lambda: att.evict(200, 4, 20), lambda: att.append(rows(65), rows(65), [64, 0, 1]), lambda: att.evict(64, 4, 20),
               lambda: att.append(rows(3), rows(3), [1, 1, 1])]
    for change in changes:
        change()
        q.copy_(torch.randn(3, 8, 128, device="cuda", generator=g))
        o.fill_(float("nan"))
        graph.replay()
        assert torch.equal(o, att.attend(q, want)) and not bool(o.isnan().any())
    assert att.lengths == [65, 65, 65] and int(att.dev_status.item()) == 0


def test_append_refused_while_a_stream_is_captured():
    """append() reads host memory and may not be captured: it raises, and the streams stay as they were."""
    import torch
    from adaptive_block_sparse_hilbert_b200 import pipeline
    att = pipeline.CachedAttention(1, 2, 1, 64, n_pages=4, max_blocks=4)
    x = torch.ones(70, 1, 64, dtype=torch.bfloat16, device="cuda")
    att.append(x[:60], x[:60], [60])
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(graph):
            att.append(x[:10], x[:10], [10])
    torch.cuda.synchronize()
    assert att.lengths == [60] and att.length.tolist() == [60] and len(att.free) == 3
    att.append(x[:10], x[:10], [10])
    q = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert bool((att.attend(q, torch.empty_like(q)) == 1).all()) and int(att.dev_status.item()) == 0
