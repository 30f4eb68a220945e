"""The ends of a mixture-of-experts block, around dispatch and combine.

    router = Router(T, E, k, balance_coef=0.01, train=True)
    r = router.route(logits)                       # r.topk_idx, r.topk_w for dispatch and combine
    d_logits = router.backward(logits, d_topk_w, d_losses)
    w = W4Weights(codes, scales, group=128, paired=True)
    y = expert_w4(recv, w, layout.counts, layout.offsets, x_scales=recv_scales)
    norm = BlockNorm(T, H, gate="channel", scaled=True, train=True)
    h, n = norm.forward(h, y, w_post, w_pre, gate, res_scale)

As elsewhere in this package, objects allocate their outputs and workspace
once, and calls only launch kernels on the given (or current) stream: a
second call overwrites what the first returned.  (expert_w4 is a function: it
allocates its result where no `out` is given.)
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from ._lib import (CAPACITY, GATE_CHANNEL, GATE_NONE, GATE_TOKEN, PACKED, PAYLOAD_BF16, PAYLOAD_FP8_E4M3,
                   PAYLOAD_FP8_E4M3_UE8M0, TYPE_BF16, TYPE_F32, W4, Norm, Route, check, load)
from ._tensors import _empty, _ptr, _rows_ptr, _shaped_ptr, _stream

_TYPES = {torch.bfloat16: TYPE_BF16, torch.float32: TYPE_F32}
_E4M3_ROWS = (torch.float8_e4m3fn, torch.uint8)
_GATES = {None: GATE_NONE, "channel": GATE_CHANNEL, "token": GATE_TOKEN}


@dataclass
class Routing:
    topk_idx: torch.Tensor              # i32 [T, k]
    topk_w: torch.Tensor                # f32 [T, k]
    lse: torch.Tensor | None            # f32 [T]; with train=True, as the rest
    counts: torch.Tensor | None         # i32 [num_seqs, E]
    prob_sums: torch.Tensor | None      # f32 [num_seqs, E]
    seq_tokens: torch.Tensor | None     # i32 [num_seqs + 2]
    losses: torch.Tensor | None         # f32 [2]: balance, z
    err_flags: torch.Tensor             # u32 word as i32 [1], OR-ed into; the caller clears it


class Router:
    """The choice of each token's experts from router logits (ep_route): top k,
    limited to the best topk_groups of `groups` groups where given, weighted by
    the softmax over the chosen logits (or, with full_softmax, over all).  With
    train=True also per-expert counts, the balance and z losses and backward().

    dtype: type of the logits and their gradient, f32 or bf16.  num_seqs: the
    balance loss is taken over each of so many sequences (seq_offsets) and
    averaged.
    """

    def __init__(self, T: int, E: int, k: int, groups: int = 1, topk_groups: int = 1, full_softmax: bool = False,
                 dtype: torch.dtype = torch.float32, num_seqs: int = 1, balance_coef: float = 0.0, z_coef: float = 0.0,
                 train: bool = False, device: str | torch.device = "cuda"):
        lib = load()
        if dtype not in _TYPES:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
        self.desc = Route(T, E, k, groups, topk_groups, int(full_softmax), _TYPES[dtype], num_seqs, balance_coef, z_coef)
        self._ref = ctypes.byref(self.desc)
        nbytes = lib.ep_route_workspace_bytes(self._ref)
        if nbytes == ctypes.c_size_t(-1).value:
            check(1, "ep_route_workspace_bytes")
        self.T, self.E, self.k, self.dtype, self.num_seqs, self.train = T, E, k, dtype, num_seqs, train
        dev = torch.device(device)
        i32, f32 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.float32, device=dev)
        self.out = Routing(
            topk_idx=torch.empty((T, k), **i32), topk_w=torch.empty((T, k), **f32),
            lse=torch.empty(T, **f32) if train else None, counts=torch.empty((num_seqs, E), **i32) if train else None,
            prob_sums=torch.empty((num_seqs, E), **f32) if train else None,
            seq_tokens=torch.empty(num_seqs + 2, **i32) if train else None,
            losses=torch.empty(2, **f32) if train else None, err_flags=torch.zeros(1, **i32))
        self.workspace_bytes = int(nbytes) if train else 0
        self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=dev) if train else None
        self.d_logits = torch.empty((T, E), dtype=dtype, device=dev) if train else None
        o = self.out
        self._lib, self._shape = lib, (T, E)
        self._outputs = (_ptr(o.topk_idx), _ptr(o.topk_w), _ptr(o.lse), _ptr(o.counts), _ptr(o.prob_sums), _ptr(o.seq_tokens),
                         _ptr(o.losses), _ptr(self.workspace), self.workspace_bytes, _ptr(o.err_flags))
        self._saved = (_ptr(o.topk_idx), _ptr(o.topk_w), _ptr(o.lse), _ptr(o.counts), _ptr(o.seq_tokens))
        self._d_logits = _ptr(self.d_logits)

    def _seqs(self, seq_offsets):
        if seq_offsets is None:
            if self.train and self.num_seqs != 1:
                raise ValueError(f"{self.num_seqs} sequences need seq_offsets")
            return None
        return _shaped_ptr(seq_offsets, torch.int32, "seq_offsets", (self.num_seqs + 1,))

    def route(self, logits: torch.Tensor, select_bias: torch.Tensor | None = None, token_mask: torch.Tensor | None = None,
              seq_offsets: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> Routing:
        """logits [T, E]; select_bias f32 [E] shifts the choice alone;
        token_mask u8 or bool [T] leaves tokens out; seq_offsets i32
        [num_seqs + 1]."""
        lp, ld = _rows_ptr(logits, self.dtype, "logits", self._shape)
        if token_mask is not None and token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        st = self._lib.ep_route(
            self._ref, lp, ld, _shaped_ptr(select_bias, torch.float32, "select_bias", (self.E,)),
            _shaped_ptr(token_mask, torch.uint8, "token_mask", (self.T,)), self._seqs(seq_offsets), *self._outputs, _stream(stream))
        if st:
            check(st, "ep_route")
        return self.out

    def backward(self, logits: torch.Tensor, d_topk_w: torch.Tensor | None, d_losses: torch.Tensor | None,
                 seq_offsets: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
        """d_logits, from the logits and outputs of the last route() and the
        gradients of topk_w f32 [T, k] and of the losses f32 [2] (each None for
        zero)."""
        if not self.train:
            raise ValueError("this router was made without train=True")
        lp, ld = _rows_ptr(logits, self.dtype, "logits", self._shape)
        st = self._lib.ep_route_backward(
            self._ref, lp, ld, self._seqs(seq_offsets), *self._saved,
            _shaped_ptr(d_topk_w, torch.float32, "d_topk_w", (self.T, self.k)),
            _shaped_ptr(d_losses, torch.float32, "d_losses", (2,)), self._d_logits, _stream(stream))
        if st:
            check(st, "ep_route_backward")
        return self.d_logits


class W4Weights:
    """4-bit weights with group scales, laid out for expert_w4 (ep_w4_pack).

    codes u8 [E, rows, K/2]: input channel 2i in the low half of byte i; code c
    stands for (c - 8) * scale.  scales bf16 [E, rows, ceil(K / group)].
    paired: rows are N gate rows and then N up rows of a SwiGLU.  They are
    packed on `stream`, whose memory they are: wait for it before products on
    another one, and before codes and scales are overwritten.  Codes and scales
    are not needed afterwards and may be dropped at once.
    """

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, group: int = 128, paired: bool = False,
                 stream: torch.cuda.Stream | None = None):
        lib = load()
        if codes.dim() != 3:
            raise ValueError(f"codes must be [E, rows, K/2], got {tuple(codes.shape)}")
        E, rows, half = codes.shape
        if paired and rows % 2:
            raise ValueError(f"paired weights have an even number of rows, got {rows}")
        self.E, self.N, self.K, self.group, self.paired = E, rows // 2 if paired else rows, 2 * half, group, paired
        self.desc = W4(E, self.N, self.K, group, int(paired))
        self._ref = ctypes.byref(self.desc)
        nbytes = lib.ep_w4_bytes(self._ref)
        if nbytes == ctypes.c_size_t(-1).value:
            check(1, "ep_w4_bytes")
        cp = _ptr(codes, torch.uint8, "codes")
        sp = _shaped_ptr(scales, torch.bfloat16, "scales", (E, rows, -(-self.K // group)))
        self.packed = _empty(int(nbytes), torch.uint8, codes.device, stream)
        if stream is not None:
            for t in (codes, scales):
                t.record_stream(stream)         # the allocator does not hand them out again before they are packed
        self._lib, self._packed = lib, _ptr(self.packed)
        check(lib.ep_w4_pack(self._ref, cp, sp, self._packed, _stream(stream)), "ep_w4_pack")


def expert_w4(x: torch.Tensor, weights: W4Weights, counts: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
              capacity: int | None = None, x_scales: torch.Tensor | None = None, max_rows: int | None = None,
              out: torch.Tensor | None = None, err_flags: torch.Tensor | None = None,
              stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Every expert's product over its rows of the receive buffer (ep_expert_w4).

    x bf16 [R, K], or one-byte e4m3 with x_scales [R, K/128] (float32, or uint8
    UE8M0 exponents), as dispatch leaves it; counts / offsets from the layout
    (neither for a single matrix over all rows); capacity as in Plan.  max_rows:
    rows in use at most (T * k), all of x if not given.  Returns bf16 [R, N];
    rows without a copy are left as they were (without `out`, undefined).
    Without `out` the result is allocated by this call, as memory of `stream`
    where one is given (as under `with torch.cuda.stream(stream)`).
    """
    w = weights
    if x.dim() != 2 or x.shape[1] != w.K:
        raise ValueError(f"x must be [R, {w.K}], got {tuple(x.shape)}")
    R = x.shape[0]
    if x_scales is None:
        payload, xp, sp = PAYLOAD_BF16, _shaped_ptr(x, torch.bfloat16, "x", (R, w.K)), None
    else:
        if x.dtype not in _E4M3_ROWS:
            raise TypeError(f"x_scales go with rows of e4m3 (torch.float8_e4m3fn, or torch.uint8 holding its codes), got {x.dtype}")
        if x_scales.dtype not in (torch.float32, torch.uint8):
            raise TypeError("x_scales must be float32 or uint8 (UE8M0)")
        payload = PAYLOAD_FP8_E4M3_UE8M0 if x_scales.dtype == torch.uint8 else PAYLOAD_FP8_E4M3
        xp, sp = _ptr(x, None, "x"), _shaped_ptr(x_scales, x_scales.dtype, "x_scales", (R, w.K // 128))
    if counts is None and offsets is None and w.E != 1:
        raise ValueError("several experts need the layout's counts and offsets")
    if out is None:
        out = _empty((R, w.N), torch.bfloat16, x.device, stream)
    st = w._lib.ep_expert_w4(
        w._ref, w._packed, PACKED if capacity is None else CAPACITY, capacity or 0, R, R if max_rows is None else max_rows,
        _shaped_ptr(counts, torch.int32, "counts", (w.E,)), _shaped_ptr(offsets, torch.int32, "offsets", (w.E + 1,)), xp, sp, payload,
        _shaped_ptr(out, torch.bfloat16, "out", (R, w.N)), _shaped_ptr(err_flags, torch.int32, "err_flags", (1,)), _stream(stream))
    if st:
        check(st, "ep_expert_w4")
    return out


@dataclass
class BlockNormGrads:
    d_h: torch.Tensor                   # stream type [T, H]
    d_y: torch.Tensor | None            # bf16 [T, H]
    d_w_post: torch.Tensor | None       # f32 [H]
    d_w_pre: torch.Tensor | None        # f32 [H]
    d_gate: torch.Tensor | None         # f32 [H] or [T]
    d_res_scale: torch.Tensor | None    # f32 [1]


class BlockNorm:
    """The norm after a block, its gate and residual scale, and the norm before
    the next block (ep_block_norm), with gradients when train is set.

    dtype: type of the residual stream (h, h_out and their gradients), bf16 or
    f32; the block's output y and the normed n are bf16.  gate: None, "channel"
    (f32 [H]) or "token" (f32 [T]).  post / pre: whether there is a norm after
    / before; scaled: whether the residual is scaled by a device scalar;
    block: False for the first norm of a network (no y).
    """

    def __init__(self, T: int, H: int, dtype: torch.dtype = torch.bfloat16, gate: str | None = None, post: bool = True,
                 pre: bool = True, scaled: bool = False, block: bool = True, eps: float = 1e-6, train: bool = False,
                 device: str | torch.device = "cuda"):
        lib = load()
        if dtype not in _TYPES:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
        if gate not in _GATES:
            raise ValueError(f"gate must be None, 'channel' or 'token', got {gate!r}")
        if not block and (post or gate is not None):
            raise ValueError("post and gate need the block's output: pass post=False and gate=None with block=False")
        self.norm = Norm(T, H, _TYPES[dtype], _GATES[gate], eps)
        self._ref = ctypes.byref(self.norm)
        nbytes = lib.ep_block_norm_workspace_bytes(self._ref)
        if nbytes == ctypes.c_size_t(-1).value:
            check(1, "ep_block_norm_workspace_bytes")
        self.T, self.H, self.dtype, self.gate, self.post, self.pre = T, H, dtype, gate, bool(post), bool(pre)
        self.scaled, self.block, self.train = bool(scaled), bool(block), bool(train)
        dev = torch.device(device)
        f32 = dict(dtype=torch.float32, device=dev)
        self.h_out = torch.empty((T, H), dtype=dtype, device=dev)
        self._lib, self._shape, self._row = lib, (T, H), (H,)
        self._gate_shape = (H if gate == "channel" else T,)
        self.n = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if pre else None
        self.rstd = torch.empty((2, T), **f32) if train else None
        self.grads = None
        self.workspace = None
        self.err_flags = torch.zeros(1, dtype=torch.int32, device=dev) if train else None    # OR-ed into; the caller clears it
        if train:
            self.workspace = torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=dev)
            self.workspace_bytes = int(nbytes)
            self.grads = BlockNormGrads(
                d_h=torch.empty((T, H), dtype=dtype, device=dev),
                d_y=torch.empty((T, H), dtype=torch.bfloat16, device=dev) if block else None,
                d_w_post=torch.empty(H, **f32) if post else None, d_w_pre=torch.empty(H, **f32) if pre else None,
                d_gate=None if gate is None else torch.empty(H if gate == "channel" else T, **f32),
                d_res_scale=torch.empty(1, **f32) if scaled else None)
            g = self.grads
            self._outputs = (_ptr(g.d_h), _ptr(g.d_y), _ptr(g.d_w_post), _ptr(g.d_gate), _ptr(g.d_res_scale), _ptr(g.d_w_pre),
                             _ptr(self.workspace), self.workspace_bytes, _ptr(self.err_flags))
        self._n, self._rstd = _ptr(self.n), _ptr(self.rstd)

    def _inputs(self, h, y, w_post, w_pre, gate, res_scale):
        if ((y is None) is self.block or (w_post is None) is self.post or (w_pre is None) is self.pre or
                (gate is None) is not (self.gate is None) or (res_scale is None) is self.scaled):
            for t, wanted, name in ((y, self.block, "y"), (w_post, self.post, "w_post"), (w_pre, self.pre, "w_pre"),
                                    (gate, self.gate is not None, "gate"), (res_scale, self.scaled, "res_scale")):
                if (t is not None) != wanted:
                    raise ValueError(f"{name} is {'missing' if wanted else 'not part of this norm'}")
        f32 = torch.float32
        hp, ldh = _rows_ptr(h, self.dtype, "h", self._shape)
        yp, ldy = _rows_ptr(y, torch.bfloat16, "y", self._shape)
        return (hp, ldh, yp, ldy, _shaped_ptr(w_post, f32, "w_post", self._row), _shaped_ptr(gate, f32, "gate", self._gate_shape),
                _shaped_ptr(res_scale, f32, "res_scale", (1,)), _shaped_ptr(w_pre, f32, "w_pre", self._row))

    def forward(self, h: torch.Tensor, y: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                w_pre: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                res_scale: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
        """Returns (h_out, n); n is None without a norm before the next block."""
        st = self._lib.ep_block_norm(self._ref, *self._inputs(h, y, w_post, w_pre, gate, res_scale), self.h_out.data_ptr() or None,
                                     self._n, self._rstd, _stream(stream))
        if st:
            check(st, "ep_block_norm")
        return self.h_out, self.n

    def backward(self, h: torch.Tensor, y: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                 w_pre: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                 res_scale: torch.Tensor | None = None, d_h_out: torch.Tensor | None = None,
                 d_n: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> BlockNormGrads:
        """Gradients, from the inputs of the last forward() and the gradients
        of its outputs (d_h_out may be None: zero)."""
        if not self.train:
            raise ValueError("this norm was made without train=True")
        st = self._lib.ep_block_norm_backward(
            self._ref, *self._inputs(h, y, w_post, w_pre, gate, res_scale), self._rstd,
            _shaped_ptr(d_h_out, self.dtype, "d_h_out", self._shape), _shaped_ptr(d_n, torch.bfloat16, "d_n", self._shape),
            *self._outputs, _stream(stream))
        if st:
            check(st, "ep_block_norm_backward")
        return self.grads
