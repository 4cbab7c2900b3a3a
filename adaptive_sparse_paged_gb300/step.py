"""One decode step, or one chunk of new tokens, over L layers, optionally captured into a CUDA graph.

Per layer: asp_coverage_select (one cluster kernel, or score + select kernels) then asp_sparse_decode
(self-planning attention), and optionally asp_page_summarize in APPEND mode
first. The layers share one workspace; stream order serialises them. Nothing
returns to the host between layers, which is what lets the whole step live
inside one CUDA graph (MOIRA abstract, page "Adaptive DHiSparse: Speculative
Decoding over a Load-Adaptive KV Hierarchy").
"""

from __future__ import annotations

import math

import torch

from . import binding as B


def _check_shape(name, t, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


class DecodeStep:
    def __init__(self, kvs, q, gamma: float, budget: int = 0, sm_scale: float | None = None,
                 append=None, weights=None, decay: float = 1.0):
        """kvs: list of PagedKV (one per layer, same shape); q: fp32 [L, B, Hq, d].

        append: optional (k_new, v_new), bf16 [L, B, Hkv, d] each, written with
        APPEND before each layer's selection.
        weights: optional fp32 [L, B, Hkv, max_pages * P], the attention weight every
        cached token has received so far: after each layer's attention it becomes
        decay * weights + what this step gave (asp_decode_weights, in place; a
        replay adds again).
        """
        self.kvs = list(kvs)
        if not self.kvs:
            raise ValueError("kvs must hold at least one layer")
        kv0 = self.kvs[0]
        L = len(self.kvs)
        dev = kv0.device
        _check_shape("q", q, (L, kv0.batch, kv0.num_q_heads, kv0.head_dim))
        if append is not None:
            shp = (L, kv0.batch, kv0.num_kv_heads, kv0.head_dim)
            _check_shape("append[0]", append[0], shp)
            _check_shape("append[1]", append[1], shp)
        self.q = q
        self.gamma, self.budget = float(gamma), int(budget)
        self.sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(kv0.head_dim)
        self.append = append
        if weights is not None:
            _check_shape("weights", weights, (L,) + tuple(B.weights_shape(kv0)))
        self.weights, self.decay = weights, float(decay)
        self.lists = torch.zeros((L, kv0.batch, kv0.num_kv_heads, kv0.max_pages), dtype=torch.int32,
                                 device=dev)
        self.lens = torch.zeros((L, kv0.batch, kv0.num_kv_heads), dtype=torch.int32, device=dev)
        self.out = torch.zeros((L, kv0.batch, kv0.num_q_heads, kv0.head_dim), dtype=torch.float32,
                               device=dev)
        self.lse = torch.zeros((L, kv0.batch, kv0.num_q_heads), dtype=torch.float32, device=dev)
        self.ws = B.new_workspace(kv0)
        self.graph = None

    # kernel launches of one step, per layer: the selection's (one cluster
    # kernel, or a score pass and a select kernel; select alone at gamma = 1),
    # the decode, the append kernel when enabled, and the two of the weights
    @property
    def launches_per_step(self) -> int:
        per, _ = B.asp_select_plan(self.kvs[0], self.gamma, self.budget)
        return len(self.kvs) * (per + 1 + (1 if self.append is not None else 0) +
                                (2 if self.weights is not None else 0))

    def run_layer(self, l: int, stream=None, events=None, w_out=None):
        """w_out: where layer l's weights go instead of back to where they come from."""
        kv = self.kvs[l]
        if self.append is not None:
            B.asp_page_summarize(kv, B.ASP_SUMMARIZE_APPEND, self.append[0][l], self.append[1][l],
                                 self.ws, stream)
        if events is not None:
            events[0].record(stream)
        B.asp_coverage_select(kv, self.q[l], self.gamma, self.budget, self.lists[l],
                              self.lens[l], self.ws, stream)
        if events is not None:
            events[1].record(stream)
        B.asp_sparse_decode(kv, self.q[l], self.lists[l], self.lens[l], self.sm_scale,
                            self.out[l], self.lse[l], self.ws, stream)
        if events is not None:
            events[2].record(stream)
        if self.weights is not None:
            B.asp_decode_weights(kv, self.q[l], self.lists[l], self.lens[l], self.lse[l],
                                 self.sm_scale, self.decay, self.weights[l],
                                 self.weights[l] if w_out is None else w_out, self.ws, stream)

    def run(self, stream=None):
        for l in range(len(self.kvs)):
            self.run_layer(l, stream)

    def capture(self):
        """Captures one full step into a CUDA graph, after a warm-up step of its own that leaves
        `weights` as they are."""
        s = torch.cuda.Stream(device=self.kvs[0].device)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            # warm-up outside capture: sets kernel attributes, loads modules. A step adds to its
            # weights, so this one's go into a layer's worth of scratch.
            scratch = None if self.weights is None else torch.empty_like(self.weights[0])
            for l in range(len(self.kvs)):
                self.run_layer(l, w_out=scratch)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        self.graph = g
        return g

    def replay(self):
        self.graph.replay()


class DecodeLoop:
    """n consecutive decode steps over L layers, captured into one CUDA graph.

    Step i appends one token per request at position T0_b + i (APPEND: its K
    and V rows, folded into its page's summary), then runs every layer's
    coverage selection and attention with that step's queries; the page lists
    change from step to step as the queries and the newest pages do (MOIRA
    abstract: lists per request, layer, KV head and step). Each step has its own
    length buffer (T0 + i + 1) and its own outputs, so the steps are unrolled
    in the graph rather than indexed by a device counter.

    The block tables must already map the pages of T0 + n tokens, and the
    summaries must describe the first T0 tokens when the loop first runs.
    Replaying the graph re-times the same work: the appends are idempotent,
    but a replayed step's last-page summary then already holds the later
    steps' tokens, so only the first run's lists are those of fresh steps.
    """

    def __init__(self, kvs, seq_lens0, q, k_new, v_new, gamma: float, budget: int = 0,
                 sm_scale: float | None = None, fused_append: bool = True):
        """kvs: PagedKV per layer; seq_lens0: int32 [B] (T0); q: fp32 [n, L, B, Hq, d];
        k_new, v_new: bf16 [n, L, B, Hkv, d]. fused_append: append inside the score
        pass (asp_coverage_select_append) instead of a separate APPEND launch."""
        if not kvs:
            raise ValueError("kvs must hold at least one layer")
        kv0 = kvs[0]
        n, L = q.shape[0], len(kvs)
        _check_shape("q", q, (n, L, kv0.batch, kv0.num_q_heads, kv0.head_dim))
        _check_shape("k_new", k_new, (n, L, kv0.batch, kv0.num_kv_heads, kv0.head_dim))
        _check_shape("v_new", v_new, tuple(k_new.shape))
        _check_shape("seq_lens0", seq_lens0, (kv0.batch,))
        dev = kv0.device
        self.n, self.L = n, L
        self.q, self.k_new, self.v_new = q, k_new, v_new
        self.gamma, self.budget = float(gamma), int(budget)
        self.sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(kv0.head_dim)
        self.seq_lens = [(seq_lens0 + (i + 1)).to(torch.int32).contiguous() for i in range(n)]
        self.kvs = [[B.PagedKV(kv.k_cache, kv.v_cache, kv.summaries, kv.block_table,
                               self.seq_lens[i], kv.num_q_heads) for kv in kvs] for i in range(n)]
        self.lists = torch.zeros((n, L, kv0.batch, kv0.num_kv_heads, kv0.max_pages),
                                 dtype=torch.int32, device=dev)
        self.lens = torch.zeros((n, L, kv0.batch, kv0.num_kv_heads), dtype=torch.int32, device=dev)
        self.out = torch.zeros((n, L, kv0.batch, kv0.num_q_heads, kv0.head_dim),
                               dtype=torch.float32, device=dev)
        self.lse = torch.zeros((n, L, kv0.batch, kv0.num_q_heads), dtype=torch.float32,
                               device=dev)
        self.fused_append = bool(fused_append)
        self.ws = B.new_workspace(kv0)
        self.graph = None

    @property
    def launches(self) -> int:
        """Kernel launches of the whole loop: [append,] the selection's, the decode."""
        per, _ = B.asp_select_plan(self.kvs[0][0], self.gamma, self.budget,
                                   append=self.fused_append)
        return self.n * self.L * ((0 if self.fused_append else 1) + per + 1)

    def run(self, stream=None):
        for i in range(self.n):
            for l in range(self.L):
                kv = self.kvs[i][l]
                if self.fused_append:
                    B.asp_coverage_select_append(kv, self.k_new[i, l], self.v_new[i, l],
                                                 self.q[i, l], self.gamma, self.budget,
                                                 self.lists[i, l], self.lens[i, l], self.ws,
                                                 stream)
                else:
                    B.asp_page_summarize(kv, B.ASP_SUMMARIZE_APPEND, self.k_new[i, l],
                                         self.v_new[i, l], self.ws, stream)
                    B.asp_coverage_select(kv, self.q[i, l], self.gamma, self.budget,
                                          self.lists[i, l], self.lens[i, l], self.ws, stream)
                B.asp_sparse_decode(kv, self.q[i, l], self.lists[i, l], self.lens[i, l],
                                    self.sm_scale, self.out[i, l], self.lse[i, l], self.ws,
                                    stream)

    def capture(self):
        """Captures the loop into one CUDA graph. The capture itself launches
        nothing, so the first replay is the loop's first (fresh) run."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        self.graph = g
        return g

    def replay(self):
        self.graph.replay()


class ChunkStep:
    """One chunk of new tokens (whole prompts, parts of them, drafted tokens) over L layers.

    Per layer: the norms, the rotation and the write of the chunk's projected rows into
    the cache and its summaries (asp_norm_rotate_append), causal attention over the whole
    cache (asp_chunk_attention) and, on request, the attention weight that every cached
    token received (asp_chunk_weights), which `evict` goes by. The layers share one
    workspace; nothing returns to the host, so a step can be captured and replayed with
    other rows, offsets and lengths in the same buffers. Nothing of it knows those on the
    host: q_offsets and the caches' seq_lens (which count the new tokens) say what is new.
    """

    def __init__(self, kvs, qkv, q_offsets, inv_freq=None, q_weight=None, k_weight=None,
                 positions=None, eps: float = 1e-6, interleaved: bool = False,
                 sm_scale: float | None = None, weights=None, decay: float = 1.0):
        """kvs: list of PagedKV (one per layer, same shape); qkv: bf16 [L, N, Hq + 2 Hkv, d];
        q_offsets: int32 [B + 1]; inv_freq: fp32 [rotary_dim / 2] or None; q_weight, k_weight:
        bf16 [L, d] or None; positions: int32 [N] or None (the slots); weights: fp32
        [L, B, Hkv, max_pages * P] or None, becomes decay * weights + what the chunk gave."""
        self.kvs = list(kvs)
        if not self.kvs:
            raise ValueError("kvs must hold at least one layer")
        kv0 = self.kvs[0]
        L = len(self.kvs)
        n = int(qkv.shape[1]) if qkv.dim() == 4 else -1
        _check_shape("qkv", qkv, (L, n, kv0.num_q_heads + 2 * kv0.num_kv_heads, kv0.head_dim))
        _check_shape("q_offsets", q_offsets, (kv0.batch + 1,))
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                _check_shape(name, w, (L, kv0.head_dim))
        if weights is not None:
            _check_shape("weights", weights, (L,) + tuple(B.weights_shape(kv0)))
        self.qkv, self.q_offsets, self.inv_freq = qkv, q_offsets, inv_freq
        self.q_weight, self.k_weight, self.positions = q_weight, k_weight, positions
        self.eps, self.interleaved = float(eps), bool(interleaved)
        self.sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(kv0.head_dim)
        self.weights, self.decay = weights, float(decay)
        shape = (L, n, kv0.num_q_heads, kv0.head_dim)
        self.q = torch.zeros(shape, dtype=torch.bfloat16, device=kv0.device)
        self.out = torch.zeros(shape, dtype=torch.bfloat16, device=kv0.device)
        self.lse = torch.zeros(shape[:3], dtype=torch.float32, device=kv0.device)
        self.ws = B.new_workspace(kv0)
        self.graph = None

    def run_layer(self, l: int, stream=None):
        kv = self.kvs[l]
        B.asp_norm_rotate_append(kv, self.qkv[l], self.q_offsets, self.positions,
                                 None if self.q_weight is None else self.q_weight[l],
                                 None if self.k_weight is None else self.k_weight[l], self.eps,
                                 self.inv_freq, self.interleaved, self.q[l], self.ws, stream)
        B.asp_chunk_attention(kv, self.q[l], self.q_offsets, self.sm_scale, self.out[l],
                              self.lse[l], self.ws, stream)
        if self.weights is not None:
            B.asp_chunk_weights(kv, self.q[l], self.q_offsets, self.lse[l], self.sm_scale,
                                self.decay, self.weights[l], self.weights[l], self.ws, stream)

    def run(self, stream=None):
        for l in range(len(self.kvs)):
            self.run_layer(l, stream)

    def capture(self):
        """Captures the step into a CUDA graph (call `run` once before: it loads the kernels).
        That run is a step like any other: it adds the chunk's part to `weights`, and a replay
        adds again."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        self.graph = g
        return g

    def replay(self):
        self.graph.replay()


def evict(kvs, weights, keep: int, recent: int, ws, dst_table=None, stream=None):
    """Cuts every layer's cache back to `keep` tokens a request (asp_weight_evict).

    weights: fp32 [L, B, Hkv, max_pages * P], moved along in place; dst_table: int32
    [B, max_pages] of pages that the caches' table does not use, or None: in place. Returns
    (kept int32 [L, B, Hkv, keep], new_lens int32 [B]): the caller then goes on with
    new_lens as seq_lens and, where one was given, dst_table as the block table. A request
    for which dst_table names pages of its own stays as it is: its kept is -1, new_lens has
    its old length, and the workspace's error word says so."""
    kvs = list(kvs)
    if not kvs:
        raise ValueError("kvs must hold at least one layer")
    kv0 = kvs[0]
    _check_shape("weights", weights, (len(kvs),) + tuple(B.weights_shape(kv0)))
    kept = torch.full((len(kvs), kv0.batch, kv0.num_kv_heads, int(keep)), -1, dtype=torch.int32,
                      device=kv0.device)
    new_lens = torch.zeros(kv0.batch, dtype=torch.int32, device=kv0.device)
    for l, kv in enumerate(kvs):
        B.asp_weight_evict(kv, weights[l], keep, recent,
                           kv.block_table if dst_table is None else dst_table, weights[l], kept[l],
                           new_lens, ws, stream)
    return kept, new_lens
