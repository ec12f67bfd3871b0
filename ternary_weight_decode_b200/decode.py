"""Batch-1 (and skinny multi-slot) decode step over a 27B-shaped ternary
layer stack, run through the C ABI and replayed as one CUDA graph.

The weight path of one decoder layer (Bonsai page, "Decode 为什么只能算一般":
per layer the Q/K/V/O projections, then the Hadamard-rotated FFN input shared
by the fused gate/up + SwiGLU kernel, then down; CUDA Graph replay).  Each
projection quantises its own fp32 input inside the kernel, from the block
statistics its producer wrote (4 launches per layer, 1 per step for the
statistics of the step input):

  1. tern_gemv_fused(Wqkv, x)                   -> qkv   (N = 7168 = q 5120 + k 1024 + v 1024)
  2. tern_gemv_fused(Wo, qkv[:, :5120], +x)     -> x     (attention stand-in: the q output)
  3. tern_gateup_swiglu_fused(Wg, Wu, H x)      -> h     (N = 17408, Hadamard-rotated input)
  4. tern_gemv_fused(Wd, h, +x)                 -> x     (K = 17408)

By default (M = 1 or 2) the projections run as the streamed kernels, which
need no statistics (each CTA quantises the input itself) and split every
matrix evenly over the SMs.  The fused form with statistics ("fused") and
the unfused form with separate act_quant_fwht launches ("unfused", 8 per
layer) are kept for comparison and for M > 2.

By default attention is not on this path (the pages give no detail) and its
output is stood in by the q projection.  With ``attention=PagedAttention(...)``
it is: the M token rows are the next tokens of M sequences with an 8-bit paged
KV cache, and between steps 1 and 2 come

  1a. tern_kv_append_paged(q, k, v of qkv)  -> q rotated, K and V into the cache
  1b. tern_attention_paged(q)               -> the input of Wo

Norms are not on this path; a weightless RMSNorm before each block is folded
into s_x only (TERN_QUANT_RMSNORM), which leaves every int8 code unchanged and
keeps the residual stream bounded over 64 layers.  Every step above runs in
libtern's kernels; with attention, two torch additions a decode step advance
the lengths and positions on the device.
"""
from __future__ import annotations

from dataclasses import dataclass, field

import torch

from . import synth, tern

HIDDEN = 5120
QKV = 7168
FFN = 17408


def layer_bytes(fmt: int, hidden: int = HIDDEN, qkv: int = QKV, ffn: int = FFN) -> int:
    """Algorithmic bytes of one layer: packed codes (canonical bytes per row)
    plus fp16 group scales, for the four projections."""
    def mat(N, K):
        return N * tern.tern_canonical_row_bytes(fmt, K) + 2 * N * ((K + 127) // 128)
    return mat(qkv, hidden) + mat(hidden, hidden) + 2 * mat(ffn, hidden) + mat(hidden, ffn)


@dataclass
class Layer:
    wqkv: tern.TernMatrix
    wo: tern.TernMatrix
    wg: tern.TernMatrix
    wu: tern.TernMatrix
    wd: tern.TernMatrix


def make_matrix(fmt: int, N: int, K: int, seed: int, stream: int, scratch: torch.Tensor):
    """Generates trits and scales on the device and packs them with tern_pack."""
    W = tern.TernMatrix.empty(fmt, N, K)
    trits = scratch[: N * K].view(N, K)
    synth.device_trits(seed, stream, N, K, out=trits)
    tern.tern_pack(fmt, trits, W)
    synth.device_scales(seed, stream + 1, N, (K + 127) // 128, out=W.scales)
    return W


@dataclass
class PagedAttention:
    """Attention of the decode step over an 8-bit paged KV cache: its settings,
    and (after ``build``) the caches, page table and lengths of M sequences.

    ``ctx`` and ``pos`` live on the device and a step advances them, so that one
    captured graph decodes token after token; ``max_ctx`` tokens of pages are
    set aside for each sequence."""
    max_ctx: int
    kind: int = tern.TERN_KV_INT8
    page_size: int = 64
    window: int = 0
    sinks: int = 0
    theta: float = 1e6
    head_dim: int = 128

    def build(self, n_layers: int, M: int, hidden: int, qkv: int) -> "PagedAttention":
        self.Hq = hidden // self.head_dim
        self.Hkv = (qkv - hidden) // (2 * self.head_dim)
        assert self.Hq * self.head_dim == hidden and (self.Hq + 2 * self.Hkv) * self.head_dim == qkv
        per = -(-self.max_ctx // self.page_size)
        pages = torch.arange(M * per, dtype=torch.int32, device="cuda").view(M, per)
        self.ctx = torch.zeros(M, dtype=torch.int32, device="cuda")   # tokens of each sequence so far
        self.pos = torch.full((1, M), -1, dtype=torch.int32, device="cuda")
        rows = torch.arange(M + 1, dtype=torch.int32, device="cuda")
        self.batch = tern.PagedBatch(rows, self.ctx, pages, M, 1, self.max_ctx)
        self.rope = tern.RopePlan.build(self.theta, self.head_dim, self.max_ctx)
        self.caches = [tern.PagedCache.empty(self.kind, self.Hkv, self.head_dim, self.page_size, M * per)
                       for _ in range(n_layers)]
        self.ws = tern.attention_paged_workspace(self.Hq, self.caches[0])
        self.q = torch.zeros((M, self.Hq, self.head_dim), dtype=torch.float32, device="cuda")
        self.out = torch.zeros((M, hidden), dtype=torch.float32, device="cuda")
        self.refused = torch.zeros(1, dtype=torch.int32, device="cuda")  # tokens past max_ctx (not appended, or as 0)
        return self

    def set_ctx(self, ctx) -> None:
        """Sets the tokens that each sequence has (the next step appends behind them)."""
        self.ctx.copy_(torch.as_tensor(ctx, dtype=torch.int32))
        self.pos[0].copy_(self.ctx - 1)

    def advance(self) -> None:
        self.ctx.add_(1)
        self.pos.add_(1)

    def layer(self, l: int, qkv_out: torch.Tensor) -> torch.Tensor:
        """The attention of layer l on the rows of its QKV projection -> [M, hidden]."""
        M, D, q, kv = qkv_out.shape[0], self.head_dim, self.Hq * self.head_dim, self.Hkv * self.head_dim
        parts = (qkv_out[:, :q].view(M, self.Hq, D), qkv_out[:, q:q + kv].view(M, self.Hkv, D),
                 qkv_out[:, q + kv:q + 2 * kv].view(M, self.Hkv, D))
        tern.tern_kv_append_paged(*parts, self.pos, self.rope, self.batch, self.caches[l], self.q,
                                  d_invalid=self.refused)
        tern.tern_attention_paged(self.q, self.batch, self.caches[l], self.out.view(M, self.Hq, D), self.ws,
                                  window=self.window, sinks=self.sinks)
        return self.out


@dataclass
class DecodeModel:
    fmt: int
    n_layers: int
    M: int = 1
    hidden: int = HIDDEN
    qkv: int = QKV
    ffn: int = FFN
    mode: str = "streamed"  # "streamed" (M <= 2), "fused" or "unfused"
    attention: PagedAttention | None = None  # None: stood in by the q projection
    layers: list = field(default_factory=list)

    @property
    def fused(self) -> bool:
        return self.mode != "unfused"

    def build(self, seed_base: int = 0):
        scratch = torch.empty(max(self.qkv, self.ffn) * max(self.hidden, self.ffn),
                              dtype=torch.int8, device="cuda")
        for l in range(self.n_layers):
            s = seed_base + l
            self.layers.append(Layer(
                make_matrix(self.fmt, self.qkv, self.hidden, s, synth.stream_id(l, synth.PROJ_QKV), scratch),
                make_matrix(self.fmt, self.hidden, self.hidden, s, synth.stream_id(l, synth.PROJ_O), scratch),
                make_matrix(self.fmt, self.ffn, self.hidden, s, synth.stream_id(l, synth.PROJ_GATE), scratch),
                make_matrix(self.fmt, self.ffn, self.hidden, s, synth.stream_id(l, synth.PROJ_UP), scratch),
                make_matrix(self.fmt, self.hidden, self.ffn, s, synth.stream_id(l, synth.PROJ_DOWN), scratch),
            ))
        del scratch
        if self.mode == "streamed":
            assert self.M <= 2, "the streamed kernels take M = 1 or 2"
            for L in self.layers:
                for W in (L.wqkv, L.wo, L.wg, L.wu, L.wd):
                    W.retile_scales()
            self.ws = tern.stream_workspace(self.fmt, max(self.qkv, self.ffn, self.hidden), self.M, True)
        torch.cuda.synchronize()
        M = self.M
        ld_h = ((self.hidden + 15) // 16) * 16
        ld_f = ((self.ffn + 15) // 16) * 16
        self.x = torch.zeros((M, self.hidden), dtype=torch.float32, device="cuda")
        self.qkv_out = torch.zeros((M, self.qkv), dtype=torch.float32, device="cuda")
        self.h = torch.zeros((M, self.ffn), dtype=torch.float32, device="cuda")
        self.q_h = torch.zeros((M, ld_h), dtype=torch.int8, device="cuda")
        self.q_f = torch.zeros((M, ld_f), dtype=torch.int8, device="cuda")
        self.s = torch.zeros((4, M), dtype=torch.float32, device="cuda")
        self.st_x = tern.stats_buffer(M, self.hidden)
        self.st_qkv = tern.stats_buffer(M, self.qkv)
        self.st_x1 = tern.stats_buffer(M, self.hidden)
        self.st_h = tern.stats_buffer(M, self.ffn)
        if self.attention is not None:
            self.attention.build(self.n_layers, M, self.hidden, self.qkv)
            self.st_attn = tern.stats_buffer(M, self.hidden)
        return self

    def bytes_per_step(self) -> int:
        return self.n_layers * layer_bytes(self.fmt, self.hidden, self.qkv, self.ffn)

    def launches_per_step(self) -> int:
        """libtern's launches (with attention, PagedAttention.advance adds two of torch's)."""
        n = {"streamed": 4 * self.n_layers, "fused": 4 * self.n_layers + 1, "unfused": 8 * self.n_layers}[self.mode]
        if self.attention is not None:  # append and attention; the fused form also needs the output's statistics
            n += (3 if self.mode == "fused" else 2) * self.n_layers
        return n

    def attend(self, l: int) -> torch.Tensor:
        """The input of layer l's O projection, behind its QKV projection."""
        return self.qkv_out[:, : self.hidden] if self.attention is None else self.attention.layer(l, self.qkv_out)

    def layer_step_streamed(self, L: Layer, keep=None, l: int = 0):
        M = self.M
        rms, rot = tern.TERN_QUANT_RMSNORM, tern.TERN_QUANT_FWHT128
        if keep is not None:
            keep.append(("qkv_in", self.x.clone()))
        tern.tern_gemv_streamed(L.wqkv, self.x, self.qkv_out, self.ws, qflags=rms, M=M)
        if keep is not None:
            keep.append(("o_in", self.qkv_out.clone(), self.x.clone()))
        o_in = self.attend(l)
        if keep is not None and self.attention is not None:
            keep.append(("attention", o_in.clone()))
        tern.tern_gemv_streamed(L.wo, o_in, self.x, self.ws, qflags=rms, residual=self.x, M=M)
        if keep is not None:
            keep.append(("ffn_in", self.x.clone()))
        tern.tern_gateup_swiglu_streamed(L.wg, L.wu, self.x, self.h, self.ws, qflags=rms | rot, M=M)
        if keep is not None:
            keep.append(("down_in", self.h.clone(), self.x.clone()))
        tern.tern_gemv_streamed(L.wd, self.h, self.x, self.ws, qflags=rms, residual=self.x, M=M)

    def layer_step_fused(self, L: Layer, keep=None, l: int = 0):
        M = self.M
        rms, rot = tern.TERN_QUANT_RMSNORM, tern.TERN_QUANT_FWHT128
        if keep is not None:
            keep.append(("qkv_in", self.x.clone()))
        tern.tern_gemv_fused(L.wqkv, self.x, self.st_x, self.qkv_out, qflags=rms,
                             y_stats=self.st_qkv, M=M)
        if keep is not None:
            keep.append(("o_in", self.qkv_out.clone(), self.x.clone()))
        o_in, o_stats = self.attend(l), self.st_qkv
        if self.attention is not None:
            o_stats = self.st_attn
            tern.tern_act_stats(o_in, o_stats)
        if keep is not None and self.attention is not None:
            keep.append(("attention", o_in.clone()))
        tern.tern_gemv_fused(L.wo, o_in, o_stats, self.x, qflags=rms, residual=self.x, y_stats=self.st_x1, M=M)
        if keep is not None:
            keep.append(("ffn_in", self.x.clone()))
        tern.tern_gateup_swiglu_fused(L.wg, L.wu, self.x, self.st_x1, self.h, qflags=rms | rot,
                                      h_stats=self.st_h, M=M)
        if keep is not None:
            keep.append(("down_in", self.h.clone(), self.x.clone()))
        tern.tern_gemv_fused(L.wd, self.h, self.st_h, self.x, qflags=rms, residual=self.x,
                             y_stats=self.st_x, M=M)

    def layer_step(self, L: Layer, keep=None, l: int = 0):
        M = self.M
        norm = tern.TERN_QUANT_RMSNORM
        tern.act_quant_fwht(self.x, self.q_h, self.s[0], 0, flags=norm)
        tern.tern_gemv(L.wqkv, self.q_h, self.s[0], self.qkv_out, M=M)
        o_in = self.qkv_out if self.attention is None else self.attend(l)
        if keep is not None and self.attention is not None:
            keep.append(("attention", self.qkv_out.clone(), o_in.clone()))
        tern.act_quant_fwht(o_in, self.q_h, self.s[1], 0, K=self.hidden, flags=norm)
        if keep is not None:
            keep.append(("o_in", self.q_h.clone(), self.s[1].clone(), self.x.clone()))
        tern.tern_gemv(L.wo, self.q_h, self.s[1], self.x, residual=self.x, M=M)
        tern.act_quant_fwht(self.x, self.q_h, self.s[2], 128, flags=norm)
        if keep is not None:
            keep.append(("ffn_in", self.q_h.clone(), self.s[2].clone()))
        tern.tern_gateup_swiglu(L.wg, L.wu, self.q_h, self.s[2], self.h, M=M)
        tern.act_quant_fwht(self.h, self.q_f, self.s[3], 0, flags=norm)
        if keep is not None:
            keep.append(("down_in", self.q_f.clone(), self.s[3].clone(), self.x.clone(), self.h.clone()))
        tern.tern_gemv(L.wd, self.q_f, self.s[3], self.x, residual=self.x, M=M)

    def step(self, keep=None):
        if self.attention is not None:
            self.attention.advance()
        if self.mode == "fused":
            tern.tern_act_stats(self.x, self.st_x)
        layer_step = {"streamed": self.layer_step_streamed, "fused": self.layer_step_fused,
                      "unfused": self.layer_step}[self.mode]
        for l, L in enumerate(self.layers):
            layer_step(L, keep, l)

    def capture(self) -> torch.cuda.CUDAGraph:
        """One CUDA graph holding the whole step (the warming step here counts as one: with paged
        attention set the lengths after it)."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.step()  # warm: sets kernel attributes outside capture
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.step()
        return g
