"""One Veda attention layer on the C ABI (veda_core.py, "one layer", attention).

For each group of heads sharing a target tile box: plan (cached), gather Q and K to tile order with
pooling (straight to e4m3 codes and per-tile scales in the FP8 Q/K variant), score, select, gather V,
attend with the scatter fused. In the gather-free mode (``direct``) Q and K are only pooled and the attend
loads every tile as a TMA box of the packed tensors, so no tile-order copy is made. PyTorch only allocates
device buffers and supplies the stream; every step runs in libveda's kernels.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib as L


class VedaLayer:
    """Plans and buffers for one layer geometry.

    seq_len      packed rows S
    ref_spans    [(start, (t, h, w))] reference spans in packed order (tiled at their least-padding box
                 unless the reference budget keeps all)
    target       (start, (t, h, w)) the generated span (last)
    head_shapes  per head: a (t, h, w) box or None for the target's least-padding box
    budgets      (generated, reference), each a (ratio, tiles) pair with exactly one set
    direct       gather-free attend: pool Q and K, then veda_attend_direct on the packed tensors (no
                 tile-order copies). None (default): used when Q/K are bf16 and every group's layout has a
                 box form (veda_layout_export_direct); True: required (raises otherwise); False: the
                 tile-order path (veda_gather + veda_attend), which takes every layout
    logit_bound  the pool/gather of Q also writes ||q||^2 per row and that of K the largest ||k||^2 per
                 head, and the attend takes them as its logit bound (the single bf16 attend may then skip
                 the row max on an item's later tiles; the paired attend takes its softmax reference from
                 it; same softmax). Default True
    paired       with the logit bound: the paired attend (veda_attend_paired / veda_attend_direct_paired,
                 veda_attend_fp8_paired / veda_attend_int8_paired for the 8-bit Q/K), two neighbouring query
                 tiles per work item sharing each kept K/V tile load, the softmax reference fixed by the
                 bound, and an exact redo of any query tile the bound cannot serve. Default True; False
                 keeps the single-tile attend
    """

    # tile-order path: gather q, gather k, the projections' transpose, 2 score GEMMs, select, gather v, attend
    LAUNCHES_PER_GROUP = 8
    LAUNCHES_PER_GROUP_DIRECT = 7  # gather-free path: pool q, pool k, transpose, 2 score GEMMs, select, attend
    LAUNCHES_SCORE = 3  # of these the transpose and the 2 score GEMMs; with a bias veda_score_bias_launches
    EXTRA_LAUNCHES_PAIRED = 2  # the paired attend adds the list merge and the (usually empty) redo pass

    def __init__(self, seq_len, ref_spans, target, head_shapes, budgets, heads, dim, device="cuda", fp8_qk=False,
                 int8_qk=False, direct=None, logit_bound=True, paired=True):
        self.seq_len, self.heads, self.dim = int(seq_len), int(heads), int(dim)
        if fp8_qk and int8_qk:
            raise ValueError("VedaLayer: choose one of fp8_qk and int8_qk")
        if direct and (fp8_qk or int8_qk):
            raise ValueError("VedaLayer: the gather-free attend reads bf16 Q/K")
        self.fp8_qk, self.int8_qk = bool(fp8_qk), bool(int8_qk)
        self.device = torch.device(device)
        lps = L.veda_least_padding_box(target[1])
        groups = {}
        for h, s in enumerate(head_shapes):
            groups.setdefault(tuple(lps if s is None else s), []).append(h)
        spans_ref = [(s, g, None) for s, g in ref_spans]
        layouts = {box: L.veda_plan(spans_ref + [(target[0], target[1], box)], seq_len, budgets[0], budgets[1])
                   for box in sorted(groups)}
        if direct is None:
            direct = not (fp8_qk or int8_qk) and all(L.veda_layout_has_box_form(x) for x in layouts.values())
        elif direct:
            for x in layouts.values():
                if not L.veda_layout_has_box_form(x):
                    L.veda_layout_export_direct(x)  # raises with the reason
        self.direct = bool(direct)
        self.logit_bound = bool(logit_bound)
        self.paired = bool(paired) and self.logit_bound
        # the 8-bit single-tile attend keeps exact per-tile maxima: its norms are needed only when paired
        norms = self.logit_bound and (self.paired or not (self.fp8_qk or self.int8_qk))
        self.groups = []
        for box in sorted(groups):
            lay = layouts[box]
            hs = groups[box]
            n = len(hs)
            dev = self.device
            g = dict(box=box, heads_list=hs, layout=lay,
                     heads=torch.tensor(hs, dtype=torch.int32, device=dev),
                     feats_q=torch.empty(n, lay.n_video, 3 * dim, dtype=torch.float32, device=dev),
                     feats_k=torch.empty(n, lay.n_video, 3 * dim, dtype=torch.float32, device=dev),
                     workspace=torch.empty(L.veda_score_workspace_bytes(lay, n, dim) // 4, dtype=torch.float32,
                                           device=dev),
                     scores=torch.empty(n, lay.n_video, lay.n_video, dtype=torch.float32, device=dev),
                     kept_idx=torch.empty(n, lay.n_video, lay.max_kept, dtype=torch.int32, device=dev),
                     kept_cnt=torch.empty(n, lay.n_video, dtype=torch.int32, device=dev))
            if self.fp8_qk or self.int8_qk:  # Q and K are gathered straight to 8-bit codes with per-tile scales
                code_t = torch.int8 if self.int8_qk else torch.uint8
                g.update(q8=torch.empty(n, lay.n_slots, dim, dtype=code_t, device=dev),
                         k8=torch.empty(n, lay.n_slots, dim, dtype=code_t, device=dev),
                         sq=torch.empty(n, lay.n_tiles, dtype=torch.float32, device=dev),
                         sk=torch.empty(n, lay.n_tiles, dtype=torch.float32, device=dev))
            elif not self.direct:
                g.update(q_t=torch.empty(n, lay.n_slots, dim, dtype=torch.bfloat16, device=dev),
                         k_t=torch.empty(n, lay.n_slots, dim, dtype=torch.bfloat16, device=dev))
            if not self.direct:
                g.update(v_t=torch.empty(n, lay.n_slots, dim, dtype=torch.bfloat16, device=dev))
            if norms:
                g.update(q_row_sq=torch.empty(n, self.seq_len, dtype=torch.float32, device=dev),
                         k_max_sq=torch.empty(n, dtype=torch.float32, device=dev))
            else:
                g.update(q_row_sq=None, k_max_sq=None)
            g.update(pair_ws=L.paired_workspace(lay, n, dev) if self.paired else None)
            self.groups.append(g)
        self._launches_plain = ((self.LAUNCHES_PER_GROUP_DIRECT if self.direct else self.LAUNCHES_PER_GROUP) +
                                (self.EXTRA_LAUNCHES_PAIRED if self.paired else 0)) * len(self.groups)
        self.launches = self._launches_plain  # kernels one forward launches
        self.bias_spec = None  # (reach, far) of set_bias
        # streams that have read the parameters, by handle; of foreign streams the last reads' events
        self._readers, self._foreign_reads = {}, {}
        self._changed, self._behind = None, set()  # the parameters' last change, and the streams that have waited for it
        self._side = torch.cuda.Stream(self.device)  # the V gathers

    def set_projections(self, proj_q, proj_k):
        """proj_q, proj_k: fp32 [H, 3D, D] (any device); each group keeps its heads' slices on device. As with set_bias,
        the values change on the current stream: behind the calls made so far, on whatever stream, that read the old
        ones, and before every later one. Where shapes stay, so do addresses: a captured forward replays with new values."""
        with self._changing():
            for g in self.groups:
                for key, proj in (("proj_q", proj_q), ("proj_k", proj_k)):
                    idx = torch.tensor(g["heads_list"], dtype=torch.long, device=proj.device)
                    self._put(g, key, proj.detach().index_select(0, idx).to(self.device, torch.float32).contiguous())

    @contextlib.contextmanager
    def _changing(self):
        """Around a change of the parameters on the current stream."""
        here = torch.cuda.current_stream(self.device)
        for s in self._readers.values():
            here.wait_stream(s)
        for read in self._foreign_reads.values():
            here.wait_event(read)
        try:
            yield
        finally:
            self._changed = torch.cuda.Event()
            self._changed.record(here)
            self._behind = {here.cuda_stream} if self._lasting(here) else set()

    @staticmethod
    def _lasting(stream):
        """torch's own streams live as long as the process; a foreign one's id is its handle."""
        return stream.cuda_stream == 0 or stream.cuda_stream != stream.stream_id

    @staticmethod
    def _capturing(stream):
        with torch.cuda.stream(stream):
            return torch.cuda.is_current_stream_capturing()

    def _before_read(self, stream):
        """Before work on `stream` that reads the parameters: waits for their last change. Returns what _after_read takes.
        (A capturing stream cannot wait for work outside its graph, nor that for it: whoever replays the graph orders it.)"""
        s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(stream, device=self.device)
        if self._changed is not None and s.cuda_stream not in self._behind and not self._capturing(s):
            s.wait_event(self._changed)
            if self._lasting(s):
                self._behind.add(s.cuda_stream)
        return s

    def _after_read(self, s):
        """Behind that work: the parameters' next change waits for it."""
        if self._lasting(s):
            self._readers[s.cuda_stream] = s
        elif not self._capturing(s):  # it may be gone by then
            read = self._foreign_reads.setdefault(s.cuda_stream, torch.cuda.Event())
            read.record(s)

    def _put(self, g, key, value):
        """A group's tensor, in place where its shape stays, else (or with value None) in the old one's stead, whose memory
        is free for other use once the current stream, which waits for the readers, has come to here."""
        old = g.get(key)
        if old is not None and value is not None and old.shape == value.shape:
            old.copy_(value)
            return
        if old is not None:
            old.record_stream(torch.cuda.current_stream(self.device))
            del g[key]
        if value is not None:
            g[key] = value

    def set_bias(self, reach=None, far=None, bias=None):
        """A learned relative position bias of the tile scores (veda_score_bias): per-axis (t, h, w) reaches and far
        distances in tiles, and bias fp32 [H, buckets] (any device; veda_bias_buckets gives the number). Selection then
        ranks score + bias. No arguments: no bias, the scores of veda_score. Streams as in set_projections."""
        if bias is None and (reach is not None or far is not None):
            raise ValueError("VedaLayer.set_bias: reach and far come with a bias")
        buckets = None if bias is None else L.veda_bias_buckets(reach, far)
        if bias is not None and tuple(bias.shape) != (self.heads, buckets):
            raise ValueError(f"VedaLayer.set_bias: bias must be [{self.heads}, {buckets}], not {tuple(bias.shape)}")
        with self._changing():
            for g in self.groups:
                if bias is None:
                    for key in ("bias", "hats", "bias_ws"):
                        self._put(g, key, None)
                    continue
                n, lay = len(g["heads_list"]), g["layout"]
                idx = torch.tensor(g["heads_list"], dtype=torch.long, device=bias.device)
                self._put(g, "bias", bias.detach().index_select(0, idx).to(self.device, torch.float32).contiguous())
                if "hats" not in g:
                    g["hats"] = torch.empty(2, n, lay.n_video, self.dim, dtype=torch.float32, device=self.device)
                    g["bias_ws"] = torch.empty(L.veda_score_bias_workspace_bytes(lay, n, self.dim), dtype=torch.uint8,
                                               device=self.device)
        self.bias_spec = None if bias is None else (tuple(reach), tuple(far))
        self.launches = self._launches_plain
        if bias is not None:
            with torch.cuda.device(self.device):
                self.launches += sum(L.veda_score_bias_launches(g["layout"], len(g["heads_list"]), self.dim) -
                                     self.LAUNCHES_SCORE for g in self.groups)

    def _score(self, g, stream):
        lay = g["layout"]
        reading = self._before_read(stream)
        if self.bias_spec is None:
            L.veda_score(lay, g["feats_q"], g["feats_k"], g["proj_q"], g["proj_k"], g["workspace"], g["scores"], stream)
        else:
            L.veda_score_bias(lay, g["feats_q"], g["feats_k"], g["proj_q"], g["proj_k"], *self.bias_spec, g["bias"],
                              g["hats"], g["bias_ws"], g["scores"], stream)
        self._after_read(reading)

    def kept_tiles(self):
        """Total kept (video query tile, key tile) pairs of the last forward, per the page's ``kept``."""
        return sum(int(g["kept_cnt"].sum()) - g["layout"].n_global_ok * g["kept_cnt"].numel() for g in self.groups)

    def work_tiles(self):
        """The page's ``work`` counter (kept video pairs + dense global rows and columns), all groups."""
        total = 0
        for g in self.groups:
            lay = g["layout"]
            n = len(g["heads_list"])
            kept_video = int(g["kept_cnt"].sum()) - lay.n_global_ok * n * lay.n_video
            total += kept_video + n * lay.n_global * (lay.n_tiles + lay.n_video)
        return total

    def attended_tile_pairs(self):
        """Tile pairs the attend kernels process: kept lists of video rows + dense lists of global rows."""
        total = 0
        for g in self.groups:
            lay = g["layout"]
            total += int(g["kept_cnt"].sum()) + len(g["heads_list"]) * lay.n_global * lay.n_kv_ok
        return total

    def forward(self, q, k, v, out, stream=None, events=None):
        """q, k, v: bf16 [S, H, D] cuda (any strides the ABI accepts); out: bf16 [S, H, D], overwritten.

        ``events``: optional dict; CUDA event pairs recorded around each stage are appended under the stage
        names (the page's PhaseTimer): gather_qk, score, select, gather_v and attend on the tile-order path
        (gather_v runs on a second stream, concurrently with score and select; the others on ``stream``),
        pool_qk, score, select and attend on the gather-free path (all on ``stream``). The layer's buffers are shared
        by its calls: whoever makes them on several streams orders them."""
        st = stream if stream is not None else torch.cuda.current_stream()

        def mark(name, on):
            if events is None:
                return None
            e = torch.cuda.Event(enable_timing=True)
            e.record(on)
            events.setdefault(name, []).append([e, None])
            return name

        def done(name, on):
            if name is not None:
                e = torch.cuda.Event(enable_timing=True)
                e.record(on)
                events[name][-1][1] = e

        # V needs neither scores nor lists: its gather runs on a second stream while this stream scores and
        # selects (work bound by latency and arithmetic, not by HBM); it starts after the Q/K gathers, which
        # would otherwise share the HBM bandwidth with it, and each group's attend waits for its V
        side = self._side
        for g in self.groups:
            lay = g["layout"]
            if self.direct:
                m = mark("pool_qk", st)
                L.veda_pool(lay, q, g["heads"], g["feats_q"], st, row_sq=g["q_row_sq"])
                L.veda_pool(lay, k, g["heads"], g["feats_k"], st, max_sq=g["k_max_sq"])
                done(m, st)
                m = mark("score", st)
                self._score(g, st)
                done(m, st)
                m = mark("select", st)
                L.veda_select(lay, g["scores"], g["kept_idx"], g["kept_cnt"], st)
                done(m, st)
                m = mark("attend", st)
                if self.paired:
                    L.veda_attend_direct_paired(lay, q, k, v, g["kept_idx"], g["kept_cnt"], out, g["heads"],
                                                g["q_row_sq"], g["k_max_sq"], g["pair_ws"], st)
                else:
                    L.veda_attend_direct(lay, q, k, v, g["kept_idx"], g["kept_cnt"], out, g["heads"], st,
                                         q_row_sq=g["q_row_sq"], k_max_sq=g["k_max_sq"])
                done(m, st)
                continue
            m = mark("gather_qk", st)
            if self.fp8_qk or self.int8_qk:
                gather = L.veda_gather_int8 if self.int8_qk else L.veda_gather_fp8
                gather(lay, q, g["heads"], g["q8"], g["sq"], g["feats_q"], st, row_sq=g["q_row_sq"])
                gather(lay, k, g["heads"], g["k8"], g["sk"], g["feats_k"], st, max_sq=g["k_max_sq"])
            else:
                L.veda_gather(lay, q, g["heads"], g["q_t"], g["feats_q"], st, row_sq=g["q_row_sq"])
                L.veda_gather(lay, k, g["heads"], g["k_t"], g["feats_k"], st, max_sq=g["k_max_sq"])
            done(m, st)
            qk_done = torch.cuda.Event()
            qk_done.record(st)
            side.wait_event(qk_done)
            m = mark("gather_v", side)
            L.veda_gather(lay, v, g["heads"], g["v_t"], None, side)
            done(m, side)
            v_done = torch.cuda.Event()
            v_done.record(side)
            m = mark("score", st)
            self._score(g, st)
            done(m, st)
            m = mark("select", st)
            L.veda_select(lay, g["scores"], g["kept_idx"], g["kept_cnt"], st)
            done(m, st)
            st.wait_event(v_done)
            m = mark("attend", st)
            if (self.fp8_qk or self.int8_qk) and self.paired:
                attend = L.veda_attend_int8_paired if self.int8_qk else L.veda_attend_fp8_paired
                attend(lay, g["q8"], g["k8"], g["sq"], g["sk"], g["v_t"], g["kept_idx"], g["kept_cnt"], out, g["heads"],
                       g["q_row_sq"], g["k_max_sq"], g["pair_ws"], st)
            elif self.fp8_qk or self.int8_qk:
                attend = L.veda_attend_int8 if self.int8_qk else L.veda_attend_fp8
                attend(lay, g["q8"], g["k8"], g["sq"], g["sk"], g["v_t"], g["kept_idx"], g["kept_cnt"], out, g["heads"], st)
            elif self.paired:
                L.veda_attend_paired(lay, g["q_t"], g["k_t"], g["v_t"], g["kept_idx"], g["kept_cnt"], out, g["heads"],
                                     g["q_row_sq"], g["k_max_sq"], g["pair_ws"], st)
            else:
                L.veda_attend(lay, g["q_t"], g["k_t"], g["v_t"], g["kept_idx"], g["kept_cnt"], out, g["heads"], st,
                              q_row_sq=g["q_row_sq"], k_max_sq=g["k_max_sq"])
            done(m, st)
        return out
