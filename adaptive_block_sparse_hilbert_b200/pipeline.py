"""One attention layer through libfva: Hilbert reorder (+ pooling) -> route -> block-sparse
attention -> inverse reorder. Orchestration and buffer ownership only; every step is a
libfva entry point.

    layer = SparseAttentionLayer(shape, p=0.9, k_floor=4)
    layer.forward(q_bnhd, k_bnhd, v_bnhd, o_bnhd)   # torch CUDA tensors, raster order

A layer made with train=True keeps what its gradient needs, and CachedAttention serves streams
token by token from a paged cache:

    layer = SparseAttentionLayer(shape, p=0.9, k_floor=4, train=True)
    layer.forward(q, k, v, o)
    layer.backward(do, dq, dk, dv)                  # raster order, of the last forward()

    att = CachedAttention(B, H, Hkv, d, n_pages, max_blocks)
    att.append(k_prompt, v_prompt, counts)          # [tokens, Hkv, d], tokens per sequence
    att.attend(q, o)                                # [B, H, d]
    att.evict(keep=4096, n_sink=4, n_recent=256)
"""
from __future__ import annotations

import itertools

import torch

from . import fva


class SparseAttentionLayer:
    def __init__(self, shape: fva.fva_shape, p: float, k_floor: int, order: int = fva.FVA_ORDER_HEAD_LPT,
                 device: str = "cuda", v_fp16: bool = True, curve: int = fva.FVA_CURVE_HILBERT,
                 train: bool = False):
        self.shape = shape
        self.p = float(p)
        self.k_floor = int(k_floor)
        self.order = int(order)
        s = shape
        self.N = fva.fva_num_tokens(s)
        self.nB = fva.fva_num_blocks(s)
        dt = torch.bfloat16 if s.dtype == fva.FVA_BF16 else torch.float32
        self.dtype = dt
        bhnd = (s.B, s.H, self.N, s.d)
        self.perm = torch.empty(self.N, dtype=torch.int32, device=device)
        self.inv = torch.empty(self.N, dtype=torch.int32, device=device)
        self.qh = torch.empty(bhnd, dtype=dt, device=device)
        self.kh = torch.empty(bhnd, dtype=dt, device=device)
        # bf16 layers keep the Hilbert-ordered V in fp16 so P.V runs with fp16 P (8x finer
        # rounding of the attention weights than bf16); the conversion is fused into the reorder
        self.v_fp16 = bool(v_fp16) and s.dtype == fva.FVA_BF16
        self.vh = torch.empty(bhnd, dtype=torch.float16 if self.v_fp16 else dt, device=device)
        self.oh = torch.empty(bhnd, dtype=dt, device=device)
        self.pooled_q = torch.empty((s.B, s.H, self.nB, s.d), dtype=torch.float64, device=device)
        self.pooled_k = torch.empty_like(self.pooled_q)
        self.mask = fva.Mask.allocate(s, device)
        ws = fva.fva_route_workspace_bytes(s, False)
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=device)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=device)
        self.curve = int(curve)
        self.train = bool(train)
        if self.train:
            # the gradient's products need V and dO in one 16-bit type, so a layer whose forward
            # reads V as fp16 keeps it as bf16 too
            self.vb = torch.empty(bhnd, dtype=dt, device=device) if self.v_fp16 else self.vh
            self.lse = torch.empty(bhnd[:3], dtype=torch.float32, device=device)
            self.doh, self.dqh, self.dkh, self.dvh = (torch.empty(bhnd, dtype=dt, device=device) for _ in range(4))
            size = fva.fva_sparse_attn_bwd_workspace_bytes(s)
            if size == 0:
                raise ValueError("SparseAttentionLayer: the gradient does not take this shape")
            self.bwd_workspace = torch.empty(size, dtype=torch.uint8, device=device)
            self.scale = None  # of the last attend(): the gradient's
        fva.fva_curve_perm(s, self.curve, self.perm, self.inv, self.dev_status)

    def reorder_inputs(self, q, k, v, stream=None):
        s = self.shape
        fva.fva_reorder(s, q, self.qh, self.pooled_q, self.perm, fva.FVA_FWD, stream)
        fva.fva_reorder(s, k, self.kh, self.pooled_k, self.perm, fva.FVA_FWD, stream)
        fva.fva_reorder(s, v, self.vh, None, self.perm, fva.FVA_FWD_F16 if self.v_fp16 else fva.FVA_FWD, stream)
        if self.train and self.v_fp16:
            fva.fva_reorder(s, v, self.vb, None, self.perm, fva.FVA_FWD, stream)

    def route(self, stream=None):
        fva.fva_route(self.shape, None, None, self.pooled_q, self.pooled_k, self.p, self.k_floor, self.mask,
                      self.workspace, self.order, self.dev_status, stream)

    def attend(self, stream=None, scale: float = 0.0):
        if self.train:
            fva.fva_sparse_attn_lse(self.shape, self.qh, self.kh, self.vh, self.mask, self.oh, self.lse, scale,
                                    self.dev_status, stream)
            self.scale = scale
            return
        fva.fva_sparse_attn(self.shape, self.qh, self.kh, self.vh, self.mask, self.oh, scale, self.dev_status, stream)

    def restore_output(self, o_out, stream=None):
        fva.fva_reorder(self.shape, self.oh, o_out, None, self.perm, fva.FVA_INV, stream)

    def forward(self, q, k, v, o_out, stream=None):
        self.reorder_inputs(q, k, v, stream)
        self.route(stream)
        self.attend(stream)
        self.restore_output(o_out, stream)
        return o_out

    def backward(self, do, dq, dk, dv, stream=None):
        """Gradients of the last forward() (train=True) for the output gradient `do`; all
        [B, N, H, d] in raster order, contiguous. The routed mask is a constant of the gradient."""
        if not self.train:
            raise RuntimeError("SparseAttentionLayer.backward: the layer was made without train=True")
        if self.scale is None:
            raise RuntimeError("SparseAttentionLayer.backward: no forward() to take the gradient of")
        s = self.shape
        for what, t in (("do", do), ("dq", dq), ("dk", dk), ("dv", dv)):
            fva._expect("SparseAttentionLayer.backward", what, t, (s.B, self.N, s.H, s.d), self.dtype, self.perm.device)
        fva.fva_reorder(s, do, self.doh, None, self.perm, fva.FVA_FWD, stream)
        fva.fva_sparse_attn_bwd(s, self.qh, self.kh, self.vb, self.oh, self.doh, self.lse, self.mask, self.dqh, self.dkh,
                                self.dvh, self.bwd_workspace, self.scale, self.dev_status, stream)
        for grad, out in ((self.dqh, dq), (self.dkh, dk), (self.dvh, dv)):
            fva.fva_reorder(s, grad, out, None, self.perm, fva.FVA_INV, stream)
        return dq, dk, dv


class CachedAttention:
    """Attention of B streams over a paged key/value cache, one query token per stream and
    call: append() stores new keys and values, attend() lets every query choose its blocks by
    Top-p with a Top-k floor and attends over them, evict() cuts the streams to a budget of
    tokens by accumulated attention weight. Pages are handed out and taken back on the host;
    every call enqueues on `stream` (default: the current one), so use one stream, or order them.

    append() and evict() change the page table and lengths on the host and copy them to the
    device; attend() touches only device state and may be captured into a CUDA graph and
    replayed between them. An append() that raises leaves the streams as they were, and so does an
    evict(), but for streams it has cut before the failure where it cut them in turn.
    """

    def __init__(self, B: int, H: int, Hkv: int, d: int, n_pages: int, max_blocks: int, dtype=torch.bfloat16,
                 p: float = 0.9, k_floor: int = 4, n_recent: int = 1, accumulate: bool = True, device: str = "cuda"):
        self.B, self.H, self.max_blocks = int(B), int(H), int(max_blocks)
        self.p, self.k_floor, self.n_recent, self.accumulate = float(p), int(k_floor), int(n_recent), bool(accumulate)
        self.cache = fva.Cache.allocate(n_pages, Hkv, d, dtype, device, mass=True)
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.zeros((B, max_blocks), **i32)
        self.length = torch.zeros(B, **i32)
        self.kept = torch.empty((B, Hkv, max_blocks), **i32)
        self.n_kept = torch.empty((B, Hkv), **i32)
        self.lse = torch.empty((B, H), dtype=torch.float32, device=device)
        self.dev_status = torch.zeros(1, **i32)

        def ws(n):
            return torch.empty(max(16, n), dtype=torch.uint8, device=device)
        self.route_ws = ws(fva.fva_cache_route_workspace_bytes(self.cache, B, max_blocks, H))
        self.attn_ws = ws(fva.fva_cache_attn_workspace_bytes(self.cache, B, max_blocks, H, self.accumulate))
        self.evict_ws = ws(fva.fva_cache_evict_workspace_bytes(self.cache, B, max_blocks))
        self.free = list(range(n_pages))[::-1]
        self.pages = [[] for _ in range(B)]   # host copies of the table's rows and the lengths
        self.lengths = [0] * B

    def _stream(self, stream):
        return torch.cuda.current_stream(self.table.device) if stream is None else stream

    def append(self, k_new, v_new, counts, stream=None):
        """k_new, v_new [sum(counts), Hkv, d]: counts[b] new tokens for stream b."""
        st = self._stream(stream)
        counts = [int(n) for n in counts]
        if len(counts) != self.B or min(counts) < 0 or sum(counts) != k_new.shape[0]:
            raise ValueError(f"CachedAttention.append: {counts} does not share out {k_new.shape[0]} tokens")
        need = [-(-(n + c) // fva.BLOCK) - len(p) for n, c, p in zip(self.lengths, counts, self.pages)]
        if any(len(p) + n > self.max_blocks for p, n in zip(self.pages, need)):
            raise ValueError("CachedAttention.append: a stream would outgrow max_blocks")
        if sum(need) > len(self.free):
            raise RuntimeError(f"CachedAttention.append: {sum(need)} pages needed, {len(self.free)} free")
        # What can fail comes before what the streams are known by: a failed call leaves them as
        # they were (table entries behind a stream's last block are not read).
        total = sum(need)
        fresh = self.free[len(self.free) - total:][::-1]
        lengths = [n + c for n, c in zip(self.lengths, counts)]
        ptr = [0, *itertools.accumulate(counts)]
        with torch.cuda.device(self.table.device), torch.cuda.stream(st):
            ints = torch.tensor(lengths + ptr, dtype=torch.int32).to(self.table.device)
            if total:
                at = [b * self.max_blocks + len(p) + i for b, (p, n) in enumerate(zip(self.pages, need)) for i in range(n)]
                both = torch.tensor([at, fresh]).to(self.table.device)
                self.table.view(-1)[both[0]] = both[1].to(torch.int32)
            fva.fva_cache_append(self.cache, self.table, ints[:self.B], k_new, v_new, ints[self.B:], max(counts),
                                 self.dev_status, st)
            self.length.copy_(ints[:self.B])
        self.lengths = lengths
        del self.free[len(self.free) - total:]
        pages = iter(fresh)
        for held, n in zip(self.pages, need):
            held += itertools.islice(pages, n)

    def attend(self, q, o, stream=None, scale: float = 0.0):
        """o [B, H, d] = attention of the query tokens q [B, H, d]; the choice is left in
        kept / n_kept, the softmax's log-sum-exp in lse."""
        fva.fva_cache_route(self.cache, self.table, self.length, q, self.p, self.k_floor, self.n_recent, self.kept,
                            self.n_kept, self.route_ws, scale, self.dev_status, stream)
        fva.fva_cache_attn(self.cache, self.table, self.length, q, self.kept, self.n_kept, o, self.attn_ws, self.lse,
                           scale, self.accumulate, self.dev_status, stream)
        return o

    def evict(self, keep: int, n_sink: int = 4, n_recent: int = 64, stream=None):
        """Cut every stream to at most `keep` tokens; returns the kept tokens' old positions
        (int32 [B, Hkv, keep], -1 behind them). A stream within the budget is left where it is. The
        others move to new pages and give back their old ones, as many at a time as there are
        pages free: those of one (ceil(keep / 64)) are enough."""
        st = self._stream(stream)
        if not 1 <= keep <= 1 << 20 or min(n_sink, n_recent) < 0 or n_sink + n_recent > keep:
            raise ValueError(f"CachedAttention.evict: keep {keep}, first {n_sink}, last {n_recent}: expected 1 <= keep <= "
                             f"2^20 and both ends within it")
        keep, room = int(keep), -(-int(keep) // fva.BLOCK)
        cut = [b for b, n in enumerate(self.lengths) if n > keep]
        if cut and room > len(self.free):
            raise RuntimeError(f"CachedAttention.evict: {room} pages needed, {len(self.free)} free")
        free, fresh, groups = list(self.free), [], []  # (a group: its range of `cut`)
        while len(fresh) < len(cut):
            first = len(fresh)
            end = min(len(cut), first + len(free) // room)
            fresh += [[free.pop() for _ in range(room)] for _ in range(first, end)]
            for b in cut[first:end]:
                free += self.pages[b][::-1]
            groups.append(slice(first, end))
        # As in append(): what can fail comes before what the streams are known by. A group's old pages
        # may be the next one's new ones, so each group is booked when its call is made.
        with torch.cuda.device(self.table.device), torch.cuda.stream(st):
            every = torch.arange(keep, dtype=torch.int32, device=self.table.device)
            kept = torch.empty((self.B, self.cache.k.shape[1], keep), dtype=torch.int32, device=self.table.device)
            some = len(cut) < self.B
            if some:
                kept.copy_(torch.where(every < self.length[:, None], every, -1)[:, None])
            if cut:
                both = torch.tensor([[b, *pages] for b, pages in zip(cut, fresh)]).to(self.table.device)
                at, dst = both[:, 0], both[:, 1:].to(torch.int32)
                # the streams that are cut, side by side
                table, length, out = (x[at] if some else x for x in (self.table, self.length, kept))
                new_len, new_table = torch.empty_like(length), torch.zeros_like(table)
                new_table[:, :room] = dst
                for g in groups:
                    fva.fva_cache_evict(self.cache, table[g], length[g], keep, n_sink, n_recent, dst[g], out[g], new_len[g],
                                        self.evict_ws, self.dev_status, st)
                    self.table[at[g]], self.length[at[g]] = new_table[g], new_len[g]
                    del self.free[len(self.free) - room * (g.stop - g.start):]
                    for b, pages in zip(cut[g], fresh[g]):
                        self.free += self.pages[b][::-1]
                        self.pages[b], self.lengths[b] = pages, keep
                if some:
                    kept[at] = out
        return kept


def ramp_sizes(H: int, steady: int = 4):
    """Head-group sizes for the pipelined layer: groups of 1, 2, 3 heads first (the first
    group's copy-in is the only one nothing overlaps), then `steady`-head groups, and a
    half-size last group (its copy-out is the only one after the compute). Sums to H."""
    sizes, left = [], H
    for n in (1, 2, 3):
        n = min(n, steady, left)
        if n > 0:
            sizes.append(n)
            left -= n
    tail = min(max(1, steady // 2), left)
    left -= tail
    while left > 0:
        n = min(steady, left)
        sizes.append(n)
        left -= n
    if tail > 0:
        sizes.append(tail)
    return sizes


class HostPipelinedLayer:
    """One layer from page-locked host Q, K, V [B, N, H, d] to host O, pipelined over head
    groups: one stream copies group g+1's head slices in while the compute streams run
    groups' reorder -> route -> attention -> inverse reorder and another stream copies group
    g-1's output back. Groups alternate between two compute streams, so a group's launches
    can start on the SMs that the previous group's attention tail leaves idle. Heads are
    independent along the whole path, so every group is an ordinary SparseAttentionLayer on
    a shape with fewer heads, and the output equals the one-shot layer's bit for bit.

    Consecutive forward() calls overlap too: a call's copy-in of a group waits only for the
    previous call's compute of that group (the last reader of the group's input buffers),
    and its compute waits for the previous call's copy-out of that group (the last reader of
    its output buffer). So one layer's copies run during its neighbours' compute. The
    caller's stream is never made to wait: call wait() (or synchronize) before reading
    o_host, and do not overwrite a host input before the call that reads it has finished.

        layer = HostPipelinedLayer(shape, p=0.9, k_floor=4)   # ramp of head groups
        layer.forward(q_host, k_host, v_host, o_host)   # pinned CPU tensors, raster order
        layer.wait()
    """

    def __init__(self, shape: fva.fva_shape, p: float, k_floor: int, groups=None,
                 order: int = fva.FVA_ORDER_HEAD_LPT, device: str = "cuda", v_fp16: bool = True,
                 curve: int = fva.FVA_CURVE_HILBERT, sizes=None, compute_streams: int = 2):
        """groups: None for the ramp schedule (ramp_sizes), or a number of equal groups;
        sizes: explicit head counts per group (overrides groups); compute_streams: streams
        the groups' compute alternates between (1 runs the groups one after another)."""
        s = shape
        H = s.H
        if sizes is None and groups is None:
            sizes = ramp_sizes(H)
        elif sizes is None:
            groups = max(1, min(int(groups), H))
            sizes = [H // groups + (1 if g < H % groups else 0) for g in range(groups)]
        sizes = [int(n) for n in sizes if int(n) > 0]
        if sum(sizes) != H:
            raise ValueError(f"group sizes {sizes} do not add up to {H} heads")
        self.shape = s
        self.heads = []  # (first head, count) per group
        h0 = 0
        for n in sizes:
            self.heads.append((h0, n))
            h0 += n
        self.N = fva.fva_num_tokens(s)
        dt = torch.bfloat16 if s.dtype == fva.FVA_BF16 else torch.float32
        self.esize = 2 if s.dtype == fva.FVA_BF16 else 4
        self.layers, self.q_in, self.k_in, self.v_in, self.o_out = [], [], [], [], []
        for _, n in self.heads:
            gs = fva.make_shape(s.B, n, s.d, s.T, s.Hg, s.Wg, s.dtype)
            self.layers.append(SparseAttentionLayer(gs, p, k_floor, order, device, v_fp16, curve))
            for lst in (self.q_in, self.k_in, self.v_in, self.o_out):
                lst.append(torch.empty((s.B, self.N, n, s.d), dtype=dt, device=device))
        self.s_in = torch.cuda.Stream(device=device)
        self.s_comp = [torch.cuda.Stream(device=device) for _ in range(max(1, int(compute_streams)))]
        self.s_out = torch.cuda.Stream(device=device)
        G = len(self.heads)
        self.in_ready = [torch.cuda.Event() for _ in range(G)]    # group's inputs on the device
        self.comp_done = [torch.cuda.Event() for _ in range(G)]   # group's compute finished
        self.out_done = [torch.cuda.Event() for _ in range(G)]    # group's output in host memory
        self.started = False
        # the buffers (and each group's token order) were made on the current stream
        made = torch.cuda.Event()
        made.record(torch.cuda.current_stream())
        for st in self._streams():
            st.wait_event(made)

    def _streams(self):
        return [self.s_in, *self.s_comp, self.s_out]

    def forward(self, q_host, k_host, v_host, o_host):
        """Enqueue one layer and return the stream that copies its output out (see the
        class notes: nothing is made to wait on it; wait() does that)."""
        s = self.shape
        row = s.H * s.d * self.esize
        rows = s.B * self.N
        for g, ((h0, n), qd, kd, vd) in enumerate(zip(self.heads, self.q_in, self.k_in, self.v_in)):
            if self.started:
                self.s_in.wait_event(self.comp_done[g])
            width = n * s.d * self.esize
            for dst, src in ((qd, q_host), (kd, k_host), (vd, v_host)):
                fva.fva_copy_strided(dst, width, src[:, :, h0:h0 + n, :], row, width, rows, self.s_in)
            self.in_ready[g].record(self.s_in)
        for g, ((h0, n), layer) in enumerate(zip(self.heads, self.layers)):
            st = self.s_comp[g % len(self.s_comp)]
            st.wait_event(self.in_ready[g])
            if self.started:
                st.wait_event(self.out_done[g])
            layer.forward(self.q_in[g], self.k_in[g], self.v_in[g], self.o_out[g], st)
            self.comp_done[g].record(st)
            self.s_out.wait_event(self.comp_done[g])
            width = n * s.d * self.esize
            fva.fva_copy_strided(o_host[:, :, h0:h0 + n, :], row, self.o_out[g], width, width, rows, self.s_out)
            self.out_done[g].record(self.s_out)
        self.started = True
        return self.s_out

    def after(self, stream=None):
        """Make the layer's streams wait for the work already enqueued on `stream` (default:
        the current stream), e.g. a timing event or a producer of the host inputs."""
        st = torch.cuda.current_stream() if stream is None else stream
        for side in self._streams():
            side.wait_stream(st)

    def wait(self, stream=None):
        """Make `stream` (default: the current stream) wait until every enqueued forward()
        has finished, its output copied to host memory."""
        st = torch.cuda.current_stream() if stream is None else stream
        for side in self._streams():
            st.wait_stream(side)

    def dev_status(self):
        """Largest device error code any group reported (0 = none)."""
        return max(int(l.dev_status.item()) for l in self.layers)
