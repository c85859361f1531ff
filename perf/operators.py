"""Measured cases of the training and serving operators beside the sparse-attention path.

Four kinds of case, each one operator as a program calls it:

  grad    gradient of block-sparse attention (fva_sparse_attn_bwd): dQ, dK, dV from the
          forward's inputs, output and log-sum-exp, for a routed 64 x 64 block mask
  decode  one new token per sequence against a paged key/value cache: every query selects
          its own key blocks by a cheap score (fva_cache_route), then attends over them and
          adds its attention weights to the cache (fva_cache_attn)
  append  new keys and values go into their pages, the block means follow (fva_cache_append)
  evict   each sequence and key head keeps the tokens with the most accumulated attention
          weight, in order, in new pages (fva_cache_evict)

`own` chooses between the plain form (elementary torch) and the framework's calls.
"""
import math

import torch

own = False

BLOCK = 64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest training layer of this repository (4 x 16 x 16 latents, fp32)
        dict(name="grad tiny f32", kind="grad", B=1, T=4, Hg=16, Wg=16, H=2, d=64, dtype="f32", keep=0.4, empty=False),
        # two small clips with an odd block count, a ragged last block and rows that keep nothing
        dict(name="grad ragged", kind="grad", B=2, T=3, Hg=12, Wg=17, H=6, d=128, dtype="bf16", keep=0.5, empty=True),
        # the token grid with uneven heads, at head dim 64
        dict(name="grad hetero d64", kind="grad", B=1, T=13, Hg=30, Wg=45, H=32, d=64, dtype="bf16", keep=0.3, empty=False),
        # a 480p clip, the share of the heads that one of several GPUs holds
        dict(name="grad 480p", kind="grad", B=1, T=21, Hg=30, Wg=52, H=16, d=128, dtype="bf16", keep=0.25, empty=False),
        # one short sequence: what a single call costs
        dict(name="decode one short", kind="decode", B=1, H=8, Hkv=2, d=64, dtype="bf16", len_min=200, len_max=200,
             p=0.9, hot=0.5, k_floor=2, n_recent=1, mass=False),
        # a batch of ordinary sequences, grouped key heads, weights accumulated for eviction
        dict(name="decode batch", kind="decode", B=32, H=32, Hkv=8, d=128, dtype="bf16", len_min=1999, len_max=9001,
             p=0.9, hot=0.2, k_floor=4, n_recent=2, mass=True),
        # two very long streams
        dict(name="decode long", kind="decode", B=2, H=40, Hkv=8, d=128, dtype="bf16", len_min=131077, len_max=250001,
             p=0.9, hot=0.1, k_floor=16, n_recent=4, mass=True),
        # fp32 cache, one key head per query head
        dict(name="decode f32", kind="decode", B=8, H=12, Hkv=12, d=64, dtype="f32", len_min=500, len_max=2900,
             p=0.95, hot=0.3, k_floor=4, n_recent=1, mass=False),
        # prompts of very different lengths behind caches that are empty or end inside a page
        dict(name="append prompts", kind="append", B=16, H=32, Hkv=8, d=128, dtype="bf16", old_min=0, old_max=700,
             new_min=1, new_max=4001),
        # one decoding step of a batch
        dict(name="append tokens", kind="append", B=48, H=16, Hkv=4, d=64, dtype="f16", old_min=100, old_max=8000,
             new_min=1, new_max=1),
        # a batch brought back to its budget
        dict(name="evict batch", kind="evict", B=16, Hkv=8, d=128, dtype="bf16", len_min=3001, len_max=9000, keep=2048,
             n_sink=4, n_recent=256),
        # one long stream cut to a quarter
        dict(name="evict long", kind="evict", B=1, Hkv=8, d=128, dtype="bf16", len_min=250001, len_max=250001,
             keep=62500, n_sink=4, n_recent=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["grad", "decode", "append", "evict"])
    if kind == "grad":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        big = dtype == "bf16"
        T, Hg, Wg = rng.randint(1, 21 if big else 5), _log(rng, 5, 30 if big else 17), _log(rng, 5, 52 if big else 17)
        B, H = rng.choice([1, 1, 2]), rng.randint(1, 8)
        most = 4 * 32760 ** 2 / (B * H * (T * Hg * Wg) ** 2)  # kept pairs of the largest listed layer
        return dict(kind=kind, B=B, T=T, Hg=Hg, Wg=Wg, H=H, d=rng.choice([64, 128] if big else [32, 64, 128]),
                    dtype=dtype, keep=round(min(rng.uniform(0.1, 0.9), most), 3), empty=rng.random() < 0.3)
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind == "decode":
        Hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        top = _log(rng, 1, 100000)
        low = rng.randint(1, top)
        B = max(1, min(64, _log(rng, 1, 64), 1000000 // (top * Hkv)))
        return dict(kind=kind, B=B, H=Hkv * group, Hkv=Hkv, d=d, dtype=dtype, len_min=low, len_max=top,
                    p=round(rng.uniform(0.5, 0.99), 3), hot=round(rng.uniform(0.05, 0.6), 3), k_floor=rng.randint(0, 8),
                    n_recent=rng.randint(0, 4), mass=rng.random() < 0.5)
    if kind == "append":
        new = rng.choice([1, _log(rng, 1, 4000)])
        old = rng.choice([0, _log(rng, 1, 2000)])
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(kind=kind, B=_log(rng, 1, 16), H=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, d=d, dtype=dtype,
                    old_min=rng.randint(0, old), old_max=old, new_min=rng.randint(0, new), new_max=new)
    top = _log(rng, 2, 60000)
    keep = rng.randint(1, top)
    n_sink = rng.randint(0, min(4, keep))
    return dict(kind=kind, B=max(1, min(16, 200000 // top)), Hkv=rng.choice([1, 2, 4, 8]), d=d, dtype=dtype,
                len_min=rng.randint(1, top), len_max=top, keep=keep, n_sink=n_sink,
                n_recent=rng.randint(0, (keep - n_sink) // 2))


# ------------------------------------------------------------------------------ sizes

def _spread(low, high, n, step=5):
    """n whole numbers from low to high, both among them, in no sorted order."""
    at = [low + (high - low) * i // max(1, n - 1) if n > 1 else high for i in range(n)]
    return [at[(i * step + 1) % n] for i in range(n)] if n % step else at


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _grad_counts(case):
    """Kept key blocks of each row, by head: heads differ, as routed heads do."""
    N = case["T"] * case["Hg"] * case["Wg"]
    nB, BH = _blocks(N), case["B"] * case["H"]
    share = [0.4 + 1.2 * i / max(1, BH - 1) if BH > 1 else 1.0 for i in range(BH)]
    return N, nB, [min(nB, max(1, round(case["keep"] * f * nB))) for f in share]


def _decode_kept(case, n):
    """Blocks that a query of a sequence with n tokens keeps: the mass sits in the hot ones."""
    nB = _blocks(n)
    return min(nB, max(math.ceil(case["p"] * max(1, round(case["hot"] * nB))), case["k_floor"]) + case["n_recent"])


def work(case):
    if case["kind"] == "grad":
        N, nB, counts = _grad_counts(case)
        rows = case["B"] * case["H"] * N
        kept = sum(counts) * nB * (0.9 if case["empty"] else 1.0)
        return {"bytes": 8 * rows * case["d"] * ESIZE[case["dtype"]] + 4 * rows + 4 * kept,
                "flops": 5 * 2 * BLOCK * BLOCK * case["d"] * kept}
    d, es, Hkv = case["d"], ESIZE[case["dtype"]], case["Hkv"]
    if case["kind"] == "decode":
        lens = _spread(case["len_min"], case["len_max"], case["B"])
        blocks = sum(_blocks(n) for n in lens)
        kept = sum(min(n, BLOCK * _decode_kept(case, n)) for n in lens)
        mass = 8 * kept * Hkv if case["mass"] else 0
        return {"bytes": Hkv * (blocks * d * 4 + kept * 2 * d * es) + mass + 2 * case["B"] * case["H"] * d * es
                + 4 * blocks * (1 + Hkv), "flops": 2 * case["H"] * d * (blocks + 2 * kept)}
    if case["kind"] == "append":
        old = _spread(case["old_min"], case["old_max"], case["B"], 3)
        new = _spread(case["new_min"], case["new_max"], case["B"])
        pages = sum(_blocks(o + n) - o // BLOCK if n else 0 for o, n in zip(old, new))
        again = sum(o % BLOCK if n else 0 for o, n in zip(old, new))
        return {"bytes": Hkv * d * (4 * es * sum(new) + es * again + 4 * pages), "flops": Hkv * d * (sum(new) + again)}
    lens = _spread(case["len_min"], case["len_max"], case["B"])
    kept = sum(min(n, case["keep"]) for n in lens)
    return {"bytes": Hkv * (4 * sum(lens) + kept * (4 * d * es + 12) + 4 * d * kept // BLOCK), "flops": Hkv * (sum(lens) + kept * d)}


# ------------------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    make = {"grad": _prepare_grad, "decode": _prepare_decode, "append": _prepare_append, "evict": _prepare_evict}
    state = make[case["kind"]](case, g)
    state["case"] = dict(case)
    return state


def _prepare_grad(case, g):
    """Hilbert-ordered Q, K, V, the forward's O and log-sum-exp, dO, and the mask with the tile
    lists that the forward's attention kernel reads (query block pairs over the union of
    their rows). Neighbouring query blocks keep similar key blocks."""
    N, nB, counts = _grad_counts(case)
    BH, d, dt = case["B"] * case["H"], case["d"], DTYPES[case["dtype"]]
    score = _randn(g, BH, (nB + 7) // 8, nB).repeat_interleave(8, 1)[:, :nB] + 0.5 * _randn(g, BH, nB, nB)
    at = torch.arange(nB, device="cuda")
    score = score - 3.0 * ((at[:, None] - at[None, :]).abs() > 1)  # a block and its neighbours come first
    order = score.argsort(dim=-1, descending=True)
    first = at[None, None, :] < torch.tensor(counts, device="cuda")[:, None, None]
    keep = torch.zeros(BH, nB, nB, dtype=torch.bool, device="cuda")
    keep.scatter_(2, order, first.expand(BH, nB, nB))
    if case["empty"]:
        keep &= (torch.rand(BH, nB, 1, generator=g, device="cuda") >= 0.1)
    q, k, v = (_randn(g, BH, N, d).to(dt) for _ in range(3))
    do = (0.02 * _randn(g, BH, N, d)).to(dt)
    o, lse = torch.zeros(BH, N, d, dtype=dt, device="cuda"), torch.empty(BH, N, device="cuda")
    step = max(1, int(1e9) // (N * N))
    for h in range(0, BH, step):
        s = _scores(q[h:h + step].float(), k[h:h + step].float(), keep[h:h + step], N, 1 / math.sqrt(d))
        lse[h:h + step] = torch.logsumexp(s, -1)
        p = (s - lse[h:h + step].nan_to_num(neginf=0.0)[..., None]).exp_()
        o[h:h + step] = (p @ v[h:h + step].float()).to(dt)
    four = (case["B"], case["H"], N, d)
    return dict(q=q.view(four), k=k.view(four), v=v.view(four), o=o.view(four), do=do.view(four),
                lse=lse.view(four[:3]), keep=keep, mask=_mask_lists(keep))


def _mask_lists(keep):
    """CSR rows, tile lists and work list (longest first within a head, heads by load) of a block mask."""
    BH, nB, _ = keep.shape
    i32 = torch.int32
    rows = keep.reshape(BH * nB, nB)
    row_ptr = torch.zeros(BH * nB + 1, dtype=i32, device="cuda")
    row_ptr[1:] = rows.sum(1).cumsum(0)
    col_idx = torch.zeros(BH * nB * nB, dtype=i32, device="cuda")
    cols = rows.nonzero()[:, 1]
    col_idx[:cols.numel()] = cols.to(i32)
    pairs = (nB + 1) // 2
    two = torch.zeros(BH, 2 * pairs, nB, dtype=torch.bool, device="cuda")
    two[:, :nB] = keep
    bits = two.view(BH * pairs, 2, nB)
    bits = bits[:, 0].to(i32) + 2 * bits[:, 1].to(i32)
    cost = (bits > 0).sum(1)
    tile_ptr = torch.zeros(BH * pairs + 1, dtype=i32, device="cuda")
    tile_ptr[1:] = cost.cumsum(0)
    tile_col = torch.zeros(BH * pairs * nB, dtype=i32, device="cuda")
    t, b = bits.nonzero(as_tuple=True)
    tile_col[:t.numel()] = (4 * b).to(i32) + bits[t, b]
    load = cost.view(BH, pairs).sum(1)
    by_cost = cost.view(BH, pairs).argsort(dim=1, descending=True, stable=True)
    by_load = load.argsort(descending=True, stable=True)
    worklist = (by_cost + pairs * torch.arange(BH, device="cuda")[:, None])[by_load].reshape(-1)
    return dict(row_ptr=row_ptr, col_idx=col_idx, head_kept=keep.sum((1, 2)), tile_ptr=tile_ptr, tile_col=tile_col,
                tile_cost=cost.to(i32), worklist=worklist.to(i32))


def _pages(lens, g, spare, extra=0):
    """A page table of shuffled pages, one row of block slots per sequence; unused slots name page 0."""
    need = [_blocks(n) for n in lens]
    n_pages = sum(need) + spare
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(need)) + extra
    at, table = 0, torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, n_pages, ids[at:]


def _cache(g, n_pages, Hkv, d, dt):
    return dict(k=_randn(g, n_pages, Hkv, BLOCK, d).to(dt), v=_randn(g, n_pages, Hkv, BLOCK, d).to(dt),
                key_mean=torch.zeros(n_pages, Hkv, d, device="cuda"))


def _prepare_decode(case, g):
    """A filled cache in which a part of the blocks (the hot ones) lies along the queries' direction."""
    B, H, Hkv, d, dt = case["B"], case["H"], case["Hkv"], case["d"], DTYPES[case["dtype"]]
    lens = _spread(case["len_min"], case["len_max"], B)
    table, n_pages, _ = _pages(lens, g, 3, 2)
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    c = _cache(g, n_pages, Hkv, d, dt)
    way = _randn(g, B, Hkv, d)
    way = way / way.norm(dim=-1, keepdim=True)
    q = (2 * math.sqrt(d) * way[:, :, None] + _randn(g, B, Hkv, H // Hkv, d)).reshape(B, H, d).to(dt)
    for b, n in enumerate(lens):  # sequence by sequence: a long cache is not held twice
        nB = _blocks(n)
        at = torch.rand(nB, generator=g, device="cuda").argsort()[:max(1, round(case["hot"] * nB))]
        page = table[b, :nB].long()
        c["k"][page[at]] = (c["k"][page[at]].float() + 4 * way[b][None, :, None, :]).to(dt)
        valid = (n - BLOCK * torch.arange(nB, device="cuda")).clamp(0, BLOCK)
        rows = c["k"][page].double() * (torch.arange(BLOCK, device="cuda") < valid[:, None])[:, None, :, None]
        c["key_mean"][page] = (rows.sum(2) / valid[:, None, None]).float()
    state = dict(c, table=table, length=length, q=q)
    if case["mass"]:
        state["mass"] = torch.exp(_randn(g, n_pages, Hkv, BLOCK))
    return state


def _prepare_append(case, g):
    """The new tokens' keys and values are slices of a fused projection's rows [q | k | v]."""
    B, H, Hkv, d, dt = case["B"], case["H"], case["Hkv"], case["d"], DTYPES[case["dtype"]]
    old = _spread(case["old_min"], case["old_max"], B, 3)
    new = _spread(case["new_min"], case["new_max"], B)
    table, n_pages, _ = _pages([o + n for o, n in zip(old, new)], g, 2)
    ptr = [0]
    for n in new:
        ptr.append(ptr[-1] + n)
    fused = _randn(g, max(1, ptr[-1]), (H + 2 * Hkv) * d).to(dt)
    c = _cache(g, n_pages, Hkv, d, dt)
    c["mass"] = torch.rand(n_pages, Hkv, BLOCK, generator=g, device="cuda")
    return dict(c, table=table, length=torch.tensor([o + n for o, n in zip(old, new)], dtype=torch.int32, device="cuda"),
                new_ptr=torch.tensor(ptr, dtype=torch.int32, device="cuda"), n_new=ptr[-1], max_new=max(new),
                k_new=fused[:, H * d:(H + Hkv) * d].unflatten(1, (Hkv, d)), v_new=fused[:, (H + Hkv) * d:].unflatten(1, (Hkv, d)))


def _prepare_evict(case, g):
    """Accumulated weights are heavy-tailed, and a third of the tokens has never been attended to."""
    B, Hkv, d, dt = case["B"], case["Hkv"], case["d"], DTYPES[case["dtype"]]
    lens = _spread(case["len_min"], case["len_max"], B)
    room = _blocks(case["keep"])
    table, n_pages, free = _pages(lens, g, room * B)
    c = _cache(g, n_pages, Hkv, d, dt)
    c["mass"] = torch.exp(2 * _randn(g, n_pages, Hkv, BLOCK)) * (torch.rand(n_pages, Hkv, BLOCK, generator=g, device="cuda") > 0.33)
    return dict(c, table=table, length=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                dst_table=free.view(B, room).contiguous())


# ------------------------------------------------------------------------------ plain forms

def run(state):
    if own:
        return _own(state)
    return {"grad": _plain_grad, "decode": _plain_decode, "append": _plain_append, "evict": _plain_evict}[state["case"]["kind"]](state)


def _scores(q, k, keep, N, scale):
    s = (q @ k.transpose(-1, -2)).mul_(scale)
    full = keep.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :N]
    return s.masked_fill_(~full, -math.inf)


def _plain_grad(state):
    """P = exp(scale q k^T - lse) on kept blocks, dP = dO V^T, dS = P (dP - rowsum(P dP));
    dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO; as many heads at a time as fit."""
    q, k, v, do, lse = (state[n].flatten(0, 1) for n in ("q", "k", "v", "do", "lse"))
    keep, (BH, N, d) = state["keep"], q.shape
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    scale, step = 1 / math.sqrt(d), max(1, int(1e9) // (N * N))
    for h in range(0, BH, step):
        at = slice(h, h + step)
        qf, kf, vf, dof = q[at].float(), k[at].float(), v[at].float(), do[at].float()
        p = _scores(qf, kf, keep[at], N, scale)
        p = p.sub_(lse[at].nan_to_num(neginf=0.0)[..., None]).exp_()
        dv[at] = (p.transpose(-1, -2) @ dof).to(q.dtype)
        ds = dof @ vf.transpose(-1, -2)
        ds = ds.sub_((p * ds).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        dq[at] = (ds @ kf).to(q.dtype)
        dk[at] = (ds.transpose(-1, -2) @ qf).to(q.dtype)
    return dict(dq=dq.view(state["q"].shape), dk=dk.view(state["q"].shape), dv=dv.view(state["q"].shape))


def _plain_decode(state):
    """Block scores q . mean(k) in 64 bits (values next to a border decide), each head's softmax
    over its sequence's blocks, the group's mean; blocks in that order until p is reached."""
    case, q, table, length = state["case"], state["q"], state["table"].long(), state["length"]
    B, H, Hkv, d, nB = case["B"], case["H"], case["Hkv"], case["d"], table.shape[1]
    at = torch.arange(nB, device="cuda")
    n_blocks = ((length + BLOCK - 1) // BLOCK)[:, None, None]
    means = state["key_mean"][table].permute(0, 2, 3, 1).double()
    s = (q.view(B, Hkv, H // Hkv, d).double() @ means) / math.sqrt(d)
    s = s.masked_fill(at >= n_blocks[..., None], -math.inf)
    prob = s.softmax(-1).mean(2)
    top, order = prob.sort(dim=-1, descending=True, stable=True)
    enough = ((top.cumsum(-1) < case["p"]).sum(-1, keepdim=True) + 1).clamp(min=case["k_floor"])
    kept = torch.zeros_like(prob, dtype=torch.bool).scatter_(2, order, (at < enough).expand_as(prob))
    kept = (kept | (at >= n_blocks - case["n_recent"])) & (at < n_blocks)
    listed_at = torch.where(kept, at, nB).sort(-1).values
    # attention over the kept blocks, in 32 bits
    n = nB * BLOCK
    kf = state["k"][table].transpose(1, 2).reshape(B, Hkv, n, d).float()
    w = (q.view(B, Hkv, H // Hkv, d).float() @ kf.transpose(-1, -2)) / math.sqrt(d)
    del kf
    hide = ~kept.repeat_interleave(BLOCK, 2) | (torch.arange(n, device="cuda") >= length[:, None, None])
    w = w.masked_fill(hide[:, :, None], -math.inf)
    lse = w.logsumexp(-1)
    w = (w - lse[..., None]).exp().masked_fill(hide[:, :, None], 0)
    o = w @ state["v"][table].transpose(1, 2).reshape(B, Hkv, n, d).float().masked_fill_(hide[..., None], 0)
    out = dict(kept=torch.where(listed_at < nB, listed_at, -1).to(torch.int32), n_kept=kept.sum(-1).to(torch.int32),
               o=o.reshape(B, H, d).to(q.dtype), lse=lse.reshape(B, H))
    if case["mass"]:
        add = w.sum(2).view(B, Hkv, nB, BLOCK).transpose(1, 2)
        state["mass"].index_add_(0, table.flatten(), add.reshape(B * nB, Hkv, BLOCK))
        out["mass"] = state["mass"]
    return out


def _plain_append(state):
    """Token i of sequence b goes to position length[b] - n_new[b] + i; its page's mean follows."""
    table, length, ptr = state["table"].long(), state["length"].long(), state["new_ptr"].long()
    k, v, mean, mass = state["k"], state["v"], state["key_mean"], state["mass"]
    n_new = ptr[1:] - ptr[:-1]
    seq = torch.repeat_interleave(torch.arange(len(n_new), device="cuda"), n_new, output_size=state["n_new"])
    pos = torch.arange(state["n_new"], device="cuda") - ptr[seq] + (length - n_new)[seq]
    page, slot = table[seq, pos // BLOCK], pos % BLOCK
    k[page, :, slot] = state["k_new"][:state["n_new"]]
    v[page, :, slot] = state["v_new"][:state["n_new"]]
    mass[page, :, slot] = 0
    last = ((length + BLOCK - 1) // BLOCK - 1).clamp(min=0)
    block = ((length - n_new) // BLOCK)[:, None] + torch.arange(state["max_new"] // BLOCK + 2, device="cuda")
    block = torch.minimum(block, last[:, None])
    some = (n_new > 0)[:, None].expand_as(block)
    page = table.gather(1, block)[some]
    valid = (length[:, None] - BLOCK * block).clamp(1, BLOCK)[some]
    rows = k[page].double() * (torch.arange(BLOCK, device="cuda") < valid[:, None])[:, None, :, None]
    mean[page] = (rows.sum(2) / valid[:, None, None]).float()
    return dict(k=k, v=v, key_mean=mean, mass=mass)


def _plain_evict(state):
    """The first n_sink and last n_recent tokens stay; of the rest those of the largest weight,
    earlier ones first among equals, until `keep` are kept; they move, in order, to new pages."""
    case, table, length, dst = state["case"], state["table"].long(), state["length"].long(), state["dst_table"].long()
    k, v, mean, mass = state["k"], state["v"], state["key_mean"], state["mass"]
    B, Hkv, d, keep, n = case["B"], case["Hkv"], case["d"], case["keep"], table.shape[1] * BLOCK
    at = torch.arange(n, device="cuda")
    weight = mass[table].transpose(1, 2).reshape(B, Hkv, n)
    stay = (at < case["n_sink"]) | (at >= (length - case["n_recent"])[:, None])
    weight = weight.masked_fill(stay[:, None], math.inf).masked_fill((at >= length[:, None])[:, None], -math.inf)
    order = weight.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    new_len = length.clamp(max=keep)
    held = torch.arange(order.shape[-1], device="cuda") < new_len[:, None, None]
    idx = torch.where(held, order, n).sort(-1).values
    idx = torch.nn.functional.pad(idx, (0, keep - idx.shape[-1]), value=n)
    held = idx < n
    b, h = torch.arange(B, device="cuda")[:, None, None], torch.arange(Hkv, device="cuda")[None, :, None]
    src = idx.clamp(max=n - 1)
    page, slot = table[b, src // BLOCK], src % BLOCK
    to = torch.arange(keep, device="cuda")
    to_page = dst[:, to // BLOCK][:, None].expand_as(idx)[held]
    to_slot, to_head = (to % BLOCK).expand_as(idx)[held], h.expand_as(idx)[held]
    page, slot = page[held], slot[held]
    k[to_page, to_head, to_slot] = k[page, to_head, slot]
    v[to_page, to_head, to_slot] = v[page, to_head, slot]
    mass[to_page, to_head, to_slot] = mass[page, to_head, slot]
    valid = (new_len[:, None] - BLOCK * torch.arange(dst.shape[1], device="cuda")).clamp(0, BLOCK)
    used = valid > 0
    rows = k[dst[used]].double() * (torch.arange(BLOCK, device="cuda") < valid[used][:, None])[:, None, :, None]
    mean[dst[used]] = (rows.sum(2) / valid[used][:, None, None]).float()
    return dict(kept=torch.where(held, idx, -1).to(torch.int32), new_len=new_len.to(torch.int32), k=k, v=v,
                key_mean=mean, mass=mass)


# ------------------------------------------------------------------------------ the framework's calls

def _bytes(n):
    return torch.empty(max(16, n), dtype=torch.uint8, device="cuda")


def _own(state):
    from adaptive_block_sparse_hilbert_b200 import fva

    case, h = state["case"], state.get("handle")
    if h is None:  # what a program sets up once: the handle, its workspaces and its output buffers
        h = state["handle"] = _handle(fva, state)
    if case["kind"] == "grad":
        fva.fva_sparse_attn_bwd(h["shape"], state["q"], state["k"], state["v"], state["o"], state["do"], state["lse"],
                                h["mask"], h["dq"], h["dk"], h["dv"], h["ws"])
        return dict(dq=h["dq"], dk=h["dk"], dv=h["dv"])
    c = h["cache"]
    if case["kind"] == "decode":
        fva.fva_cache_route(c, state["table"], state["length"], state["q"], case["p"], case["k_floor"],
                            case["n_recent"], h["kept"], h["n_kept"], h["route_ws"])
        fva.fva_cache_attn(c, state["table"], state["length"], state["q"], h["kept"], h["n_kept"], h["o"], h["attn_ws"],
                           lse=h["lse"], accumulate=case["mass"])
        out = dict(kept=h["kept"], n_kept=h["n_kept"], o=h["o"], lse=h["lse"])
        return dict(out, mass=state["mass"]) if case["mass"] else out
    if case["kind"] == "append":
        fva.fva_cache_append(c, state["table"], state["length"], state["k_new"], state["v_new"], state["new_ptr"],
                             state["max_new"])
        return dict(k=state["k"], v=state["v"], key_mean=state["key_mean"], mass=state["mass"])
    fva.fva_cache_evict(c, state["table"], state["length"], case["keep"], case["n_sink"], case["n_recent"],
                        state["dst_table"], h["kept"], h["new_len"], h["ws"])
    return dict(kept=h["kept"], new_len=h["new_len"], k=state["k"], v=state["v"], key_mean=state["key_mean"],
                mass=state["mass"])


def _handle(fva, state):
    case = state["case"]
    if case["kind"] == "grad":
        s = fva.make_shape(case["B"], case["H"], case["d"], case["T"], case["Hg"], case["Wg"], case["dtype"])
        return dict(shape=s, mask=fva.Mask(**state["mask"]), ws=_bytes(fva.fva_sparse_attn_bwd_workspace_bytes(s)),
                    **{n: torch.empty_like(state["q"]) for n in ("dq", "dk", "dv")})
    c = fva.Cache(state["k"], state["v"], state["key_mean"], state.get("mass"))
    B, Hkv, width = case["B"], case["Hkv"], state["table"].shape[1]
    i32 = dict(dtype=torch.int32, device="cuda")
    if case["kind"] == "decode":
        H = case["H"]
        return dict(cache=c, kept=torch.empty(B, Hkv, width, **i32), n_kept=torch.empty(B, Hkv, **i32),
                    o=torch.empty_like(state["q"]), lse=torch.empty(B, H, device="cuda"),
                    route_ws=_bytes(fva.fva_cache_route_workspace_bytes(c, B, width, H)),
                    attn_ws=_bytes(fva.fva_cache_attn_workspace_bytes(c, B, width, H, case["mass"])))
    if case["kind"] == "append":
        return dict(cache=c)
    return dict(cache=c, kept=torch.empty(B, Hkv, case["keep"], **i32), new_len=torch.empty(B, **i32),
                ws=_bytes(fva.fva_cache_evict_workspace_bytes(c, B, width)))


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return {"grad": _exact_grad, "decode": _exact_decode, "append": _exact_append, "evict": _exact_evict}[case["kind"]](state)


def _exact_grad(state):
    """The gradient of sum(O dO), head by head, by differentiating the softmax over kept blocks."""
    B, H, N, d = state["q"].shape
    out = {n: torch.zeros(B, H, N, d, dtype=torch.float64, device="cuda") for n in ("dq", "dk", "dv")}
    for b in range(B):
        for h in range(H):
            q, k, v = (state[n][b, h].double().requires_grad_() for n in ("q", "k", "v"))
            block = torch.arange(N, device="cuda") // BLOCK
            seen = state["keep"][b * H + h][block][:, block]
            rows = seen.any(1)
            s = torch.where(seen[rows], q[rows] @ k.T / math.sqrt(d), torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
            o = torch.softmax(s, -1) @ v
            grads = torch.autograd.grad(o, (q, k, v), state["do"][b, h].double()[rows])
            for n, x in zip(("dq", "dk", "dv"), grads):
                out[n][b, h] = x
            del s, o, grads
    return out


def _exact_decode(state):
    """Sequence by sequence and key head by key head, from the definition."""
    case = state["case"]
    B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    G = H // Hkv
    o = torch.zeros(B, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    mass = state["mass"].double() if case["mass"] else None
    for b, n in enumerate(state["length"].tolist()):
        nB = _blocks(n)
        page = state["table"][b, :nB].long()
        for g in range(Hkv):
            q = state["q"][b, g * G:(g + 1) * G].double()
            prob = torch.softmax(q @ state["key_mean"][page, g].double().T / math.sqrt(d), 1).sum(0) / G
            best = sorted(range(nB), key=lambda i, x=prob.tolist(): (-x[i], i))
            total, chosen = 0.0, set(range(max(0, nB - case["n_recent"]), nB))
            for rank, i in enumerate(best):
                if total >= case["p"] and rank >= case["k_floor"]:
                    break
                total += float(prob[i]) if nB <= 64 else 0.0
                chosen.add(i)
                if nB > 64:  # the running mass of a long list, all at once
                    run_mass = torch.cumsum(prob[torch.tensor(best, device="cuda")], 0)
                    count = max(int((run_mass < case["p"]).sum()) + 1, case["k_floor"])
                    chosen.update(best[:count])
                    break
            chosen = torch.tensor(sorted(chosen), device="cuda")
            token = (chosen[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten()
            token = token[token < n]
            k = state["k"][page[token // BLOCK], g, token % BLOCK].double()
            v = state["v"][page[token // BLOCK], g, token % BLOCK].double()
            s = q @ k.T / math.sqrt(d)
            lse[b, g * G:(g + 1) * G] = torch.logsumexp(s, 1)
            w = torch.softmax(s, 1)
            o[b, g * G:(g + 1) * G] = w @ v
            if mass is not None:
                mass[page[token // BLOCK], g, token % BLOCK] += w.sum(0)
    out = dict(kept=None, n_kept=None, o=o, lse=lse)
    return dict(out, mass=mass) if mass is not None else out


def _exact_append(state):
    mean = state["key_mean"].double()
    k, v, mass = state["k"].double(), state["v"].double(), state["mass"].double()
    ptr, lens = state["new_ptr"].tolist(), state["length"].tolist()
    for b, n in enumerate(lens):
        first = n - (ptr[b + 1] - ptr[b])
        if first == n:
            continue
        pos = torch.arange(first, n, device="cuda")
        page = state["table"][b, pos // BLOCK].long()
        k[page, :, pos % BLOCK] = state["k_new"][ptr[b]:ptr[b + 1]].double()
        v[page, :, pos % BLOCK] = state["v_new"][ptr[b]:ptr[b + 1]].double()
        mass[page, :, pos % BLOCK] = 0
        for block in range(first // BLOCK, _blocks(n)):
            at = int(state["table"][b, block])
            mean[at] = k[at, :, :n - block * BLOCK].mean(1)
    return dict(k=k, v=v, key_mean=mean, mass=mass)


def _exact_evict(state):
    case = state["case"]
    k, v, mean, mass = (state[n].double() for n in ("k", "v", "key_mean", "mass"))
    for b, n in enumerate(state["length"].tolist()):
        for g in range(case["Hkv"]):
            at = torch.arange(n, device="cuda")
            page, slot = state["table"][b, at // BLOCK].long(), at % BLOCK
            if n > case["keep"]:
                first, last = min(case["n_sink"], n), max(min(case["n_sink"], n), n - case["n_recent"])
                middle = at[first:last]
                w = state["mass"][page[middle], g, slot[middle]]
                best = middle[torch.argsort(w, descending=True, stable=True)][:case["keep"] - first - (n - last)]
                at = torch.cat([at[:first], best.sort().values, at[last:]])
            to = torch.arange(len(at), device="cuda")
            to_page = state["dst_table"][b, to // BLOCK].long()
            for x in (k, v, mass):
                x[to_page, g, to % BLOCK] = x[page[at], g, slot[at]]
            for j in range(_blocks(len(at))):
                to_at = int(state["dst_table"][b, j])
                mean[to_at, g] = k[to_at, g, :len(at) - j * BLOCK].mean(0)
    return dict(kept=None, new_len=None, k=k, v=v, key_mean=mean, mass=mass)
