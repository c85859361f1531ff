"""CachedAttention's host side: page and length bookkeeping, with the entry points replaced by
host versions over CPU tensors (what they compute is tested on the GPU)."""
import contextlib

import pytest
import torch

from adaptive_block_sparse_hilbert_b200 import fva, pipeline
from oracle import cache_oracle as CO

HKV, D = 2, 64


@pytest.fixture
def streams(monkeypatch):
    """make(B, n_pages, max_blocks) -> a CachedAttention on the CPU; make.calls: its appends."""
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: None)
    calls = []

    def append(cache, table, length, k_new, v_new, new_ptr, max_new, dev_status=None, stream=None):
        calls.append((table.clone(), length.tolist(), new_ptr.tolist(), max_new))
        for b, n in enumerate(length.tolist()):
            lo, hi = new_ptr[b].item(), new_ptr[b + 1].item()
            for t in range(lo, hi):
                at = n - (hi - t)
                page = int(table[b, at // 64])
                cache.k[page, :, at % 64], cache.v[page, :, at % 64] = k_new[t], v_new[t]
                cache.mass[page, :, at % 64] = 0.0
    monkeypatch.setattr(fva, "fva_cache_append", append)

    def evict(cache, table, length, keep, n_sink, n_recent, dst_table, kept, new_len, workspace, dev_status=None,
              stream=None):
        kept.fill_(-1)
        for b, n in enumerate(length.tolist()):
            at, m = torch.arange(n), min(n, keep)
            rows = [x[table[b, at // 64].long(), :, at % 64] for x in (cache.k, cache.v, cache.mass)]
            new_len[b] = m
            to = torch.arange(m)
            for g in range(HKV):
                kept[b, g, :m] = torch.from_numpy(CO.evict(rows[2][:, g].numpy(), keep, n_sink, n_recent))
                for x, r in zip((cache.k, cache.v, cache.mass), rows):
                    x[dst_table[b, to // 64].long(), g, to % 64] = r[kept[b, g, :m].long(), g]
    monkeypatch.setattr(fva, "fva_cache_evict", evict)

    def make(B=2, n_pages=12, max_blocks=8):
        return pipeline.CachedAttention(B, 2 * HKV, HKV, D, n_pages, max_blocks, device="cpu")
    make.calls = calls
    return make


def tokens(n, seed=0):
    return torch.randn(n, HKV, D, generator=torch.Generator().manual_seed(seed)).bfloat16()


def state(att):
    """What a caller can see: free pages, every stream's pages and length, on host and device."""
    used = [att.table[b, :len(p)].tolist() for b, p in enumerate(att.pages)]
    return sorted(att.free), [list(p) for p in att.pages], list(att.lengths), att.length.tolist(), used


def check(att):
    """Every page belongs to one stream or is free, and the device's copies say the same."""
    _, pages, lengths, length, used = state(att)
    assert sorted(att.free + sum(pages, [])) == list(range(att.cache.k.shape[0]))
    assert lengths == length and used == pages
    assert [len(p) for p in pages] == [-(-n // 64) for n in lengths]


def held(att, b):
    """A stream's keys in order, read through the device's table."""
    at = torch.arange(att.lengths[b])
    return att.cache.k[att.table[b, at // 64].long(), :, at % 64]


def test_append_books_pages_and_lengths(streams):
    att = streams()
    x = tokens(300)
    att.append(x[:100], x[:100], [70, 30])
    att.append(x[100:230], x[100:230], [0, 130])
    att.append(x[230:231], x[230:231], [1, 0])
    check(att)
    assert att.lengths == [71, 160] and len(att.free) == 12 - 2 - 3
    assert torch.equal(held(att, 0), torch.cat([x[:70], x[230:231]]))
    assert torch.equal(held(att, 1), torch.cat([x[70:100], x[100:230]]))
    assert streams.calls[1][1:] == ([70, 160], [0, 0, 130], 130)


@pytest.mark.parametrize("where", ["copy", "call"])
@pytest.mark.parametrize("error", [RuntimeError, MemoryError, KeyboardInterrupt])
def test_append_that_fails_changes_nothing(streams, monkeypatch, where, error):
    """An error of any kind, in the copies to the device (memory, a capture in progress) or in the
    call itself, takes no page and counts no token that was not stored."""
    att = streams()
    x = tokens(200)
    att.append(x[:100], x[:100], [70, 30])
    before = state(att)

    def fails(*a, **k):
        raise error("no")
    with monkeypatch.context() as m:
        m.setattr(*((torch.Tensor, "to") if where == "copy" else (fva, "fva_cache_append")), fails)
        for counts in ([60, 40], [1, 1]):  # new pages, and none
            with pytest.raises(error):
                att.append(x[:sum(counts)], x[:sum(counts)], counts)
            assert state(att) == before
    att.append(x[100:], x[100:], [60, 40])
    check(att)
    assert torch.equal(held(att, 0), torch.cat([x[:70], x[100:160]]))


@pytest.mark.parametrize("where", ["copy", "memory", "call"])
@pytest.mark.parametrize("error", [RuntimeError, MemoryError, KeyboardInterrupt])
def test_evict_that_fails_changes_nothing(streams, monkeypatch, where, error):
    """An error of any kind before or in the call loses no page and cuts no stream."""
    att = streams()
    x = tokens(300)
    att.append(x, x, [200, 100])
    before, keys = state(att), held(att, 0)

    def fails(*a, **k):
        raise error("no")
    at = {"copy": (torch.Tensor, "to"), "memory": (torch, "empty"), "call": (fva, "fva_cache_evict")}[where]
    with monkeypatch.context() as m:
        m.setattr(*at, fails)
        for _ in range(3):
            with pytest.raises(error):
                att.evict(128, 2, 8)
            assert state(att) == before
    assert torch.equal(held(att, 0), keys)
    kept = att.evict(128, 2, 8)
    check(att)
    assert att.lengths == [128, 100] and torch.equal(held(att, 0)[:, 1], keys[kept[0, 1].long(), 1])


def evicted(att, keep, sink, recent):
    """Evict with random masses and compare every stream with what it held before."""
    att.cache.mass.uniform_(0, 1)
    pages, lengths = [list(p) for p in att.pages], list(att.lengths)
    read = lambda x, b: x[att.table[b, torch.arange(att.lengths[b]) // 64].long(), :, torch.arange(att.lengths[b]) % 64]  # noqa: E731
    old = [[read(x, b) for x in (att.cache.k, att.cache.v, att.cache.mass)] for b in range(att.B)]
    kept = att.evict(keep, sink, recent)
    check(att)
    for b, n in enumerate(lengths):
        m = min(n, keep)
        assert att.lengths[b] == m and (n > keep or att.pages[b] == pages[b])  # no need to move: not moved
        new = [read(x, b) for x in (att.cache.k, att.cache.v, att.cache.mass)]
        for g in range(HKV):
            want = CO.evict(old[b][2][:, g].numpy(), keep, sink, recent)
            assert kept[b, g].tolist() == want.tolist() + [-1] * (keep - m)
            assert all(torch.equal(x[:, g], y[want, g]) for x, y in zip(new, old[b]))
    return kept


@pytest.mark.parametrize("n_pages,lens,keep", [
    (12, [200, 100, 0, 64], 64),          # room for all that are cut
    (9, [200, 100, 64, 1], 200),          # nothing to cut, and a single page free
    (9, [200, 64, 64, 64], 100),          # one of four, and just the two pages for it
    (15, [200, 130, 190, 140], 70),       # all are cut, in turn: one, two (its four pages are free then), one
    (18, [128, 320, 100, 321], 130),      # two of four, one at a time, out of order with the others
    (9, [65, 129, 63, 65], 64),           # a page is enough
])
def test_evict_needs_pages_only_for_what_it_cuts(streams, n_pages, lens, keep):
    att = streams(B=4, n_pages=n_pages)
    x = tokens(sum(lens))
    att.append(x, x.flip(0), lens)
    evicted(att, keep, 3, 10)
    att.append(x[:4], x[:4], [1] * 4)
    check(att)


def test_evict_without_a_page_is_refused(streams):
    att = streams(B=2, n_pages=6)
    x = tokens(300)
    att.append(x, x, [200, 100])
    before = state(att)
    with pytest.raises(RuntimeError):
        att.evict(64, 2, 8)
    assert state(att) == before
    evicted(att, 200, 2, 8)


@pytest.mark.parametrize("nth,done", [(2, 1), (3, 3)])  # (two pages are free: one stream, two, one)
def test_evict_that_fails_between_groups_keeps_every_stream_whole(streams, monkeypatch, nth, done):
    """Where the streams are cut in turn and the nth call fails, those before it are cut and the others
    as they were: no stream is left with pages that another one has been given."""
    att = streams(B=4, n_pages=15)
    x = tokens(660)
    lens = [200, 130, 190, 140]
    att.append(x, x.flip(0), lens)
    att.cache.mass.uniform_(0, 1)
    keys, masses = [held(att, b) for b in range(4)], []
    for b, n in enumerate(lens):
        at = torch.arange(n)
        masses.append(att.cache.mass[att.table[b, at // 64].long(), :, at % 64])
    evict, calls = fva.fva_cache_evict, []

    def fails(*a, **k):
        calls.append(a)
        if len(calls) == nth:
            raise KeyboardInterrupt
        evict(*a, **k)
    with monkeypatch.context() as m:
        m.setattr(fva, "fva_cache_evict", fails)
        with pytest.raises(KeyboardInterrupt):
            att.evict(70, 2, 8)
    check(att)
    assert att.lengths == [70] * done + lens[done:]
    for b in range(4):
        for g in range(HKV):
            want = CO.evict(masses[b][:, g].numpy(), 70, 2, 8) if b < done else slice(None)
            assert torch.equal(held(att, b)[:, g], keys[b][want, g])
