"""The ends of a layer-normed block, and expert products in 8-bit integers.

    rng = torch.tensor([seed, 0], device="cuda")        # seed, step
    norm = LayerNorm(T, H, p=0.1, site=3, train=True)
    h, n = norm.forward(h, y, w, b, rng)                # h + dropout(y), and its layer norm
    d = norm.backward(h, w, d_n, d_h, rng)              # d.d_h, d.d_y, d.d_w, d.d_b
    x = dropout(x, 0.1, rng, site=4)
    rng[1] += 5                                         # the next step: by more than the largest site
    w = I8Weights(codes, scales, paired=True)
    q, q_scales = quant_i8(recv, layout.counts, layout.offsets)
    y = expert_i8(q, q_scales, w, layout.counts, layout.offsets)

Dropout keeps no mask: which elements are dropped follows from the seed, the
step, the site and the element's place, so a backward pass is given the same.
The seed and the step stay on the device, so that a captured step can be
replayed with the step counted up inside it.

Step and site are added: the masks of a step are its own only if the step goes
up by more than the largest site each time (sites 0..n-1: by n), or if the sites
lie further apart than the steps reach (site=i << 32, steps below 2**32 counted
by 1).  Counted by 1 with sites 3 and 4, one layer would get the mask that the
other had a step before.

LayerNorm allocates its outputs and workspace once, as BlockNorm does; the
functions allocate their results where no `out` is given.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from ._lib import CAPACITY, I8, PACKED, TYPE_BF16, TYPE_F32, LayerNormDesc, check, load
from ._tensors import _empty, _int32, _on_current, _ptr, _rows_ptr, _shaped_ptr, _stream

_TYPES = {torch.bfloat16: TYPE_BF16, torch.float32: TYPE_F32}
_MASK64 = 2 ** 64 - 1
_PAIR = torch.Size((2,))


def dropout(x: torch.Tensor, p: float, rng: torch.Tensor | None, site: int = 0, residual: torch.Tensor | None = None,
            out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """residual + dropout(x), or dropout(x) alone (ep_dropout).

    x [T, H] bf16 or f32, and residual and out like it; their rows may lie
    further apart than their length.  rng i64 [2] on the device (seed, step);
    None: nothing is dropped.  site tells the dropouts of one step apart, and
    the step goes up by more than the largest of them.  out may be x or
    residual.  The gradient with respect to x is dropout(d_out, p, rng, site)."""
    lib, shape, dtype = load(), x.shape, x.dtype
    if len(shape) != 2:
        raise ValueError(f"x must be [T, H], got {tuple(shape)}")
    kind = _TYPES.get(dtype)
    if kind is None:
        raise TypeError(f"x must be torch.bfloat16 or torch.float32, got {dtype}")
    T, H = shape
    if H == 0:
        raise ValueError("x has no columns")
    xp, ld_x = _rows_ptr(x, dtype, "x", shape)
    rp, ld_res = (None, 0) if residual is None else _rows_ptr(residual, dtype, "residual", shape)
    if out is None:
        out = _empty(shape, dtype, x.device, stream)
    op, ld_out = _rows_ptr(out, dtype, "out", shape)
    st = lib.ep_dropout(T, H, kind, xp, ld_x, rp, ld_res, p, _shaped_ptr(rng, torch.int64, "rng", _PAIR), site & _MASK64, op, ld_out,
                        _stream(stream))
    if st:
        check(st, "ep_dropout")
    return out


@dataclass
class LayerNormGrads:
    d_h: torch.Tensor                   # stream type [T, H]
    d_y: torch.Tensor | None            # bf16 [T, H]; d_h itself where the two are the same
    d_w: torch.Tensor | None            # f32 [H]
    d_b: torch.Tensor | None            # f32 [H]


class LayerNorm:
    """The residual sum of a block's output after dropout, and the layer norm
    before the next block (ep_layer_norm), with gradients when train is set.

    dtype: type of the residual stream (h, h_out and their gradients), bf16 or
    f32; the block's output y and the normed n are bf16.  p, site: dropout of
    y, and which dropout of the network it is (the step goes up by more than the
    largest site each time).  weight / bias: whether the norm
    has them; block: False for the first norm of a network (no y, h_out is h).
    """

    def __init__(self, T: int, H: int, dtype: torch.dtype = torch.bfloat16, p: float = 0.0, site: int = 0, weight: bool = True,
                 bias: bool = True, block: bool = True, eps: float = 1e-5, train: bool = False, device: str | torch.device = "cuda"):
        lib = load()
        if dtype not in _TYPES:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
        if p and not block:
            raise ValueError("dropout needs the block's output: pass p=0 with block=False")
        self.desc = LayerNormDesc(_int32(T, "T"), _int32(H, "H"), _TYPES[dtype], eps, p, site & _MASK64)
        self._ref = ctypes.byref(self.desc)
        nbytes = lib.ep_layer_norm_workspace_bytes(self._ref)
        if nbytes == ctypes.c_size_t(-1).value:
            check(1, "ep_layer_norm_workspace_bytes")
        self.T, self.H, self.dtype, self.p, self.site = T, H, dtype, p, site
        self.weight, self.bias, self.block, self.train = bool(weight), bool(bias), bool(block), bool(train)
        dev = torch.device(device)
        f32 = dict(dtype=torch.float32, device=dev)
        self.h_out = torch.empty((T, H), dtype=dtype, device=dev) if block else None
        self.n = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.stats = torch.empty((2, T), **f32) if train else None
        self.err_flags = torch.zeros(1, dtype=torch.int32, device=dev)      # OR-ed into; the caller clears it
        self.workspace = self.grads = None
        self._lib, self._shape, self._row = lib, torch.Size((T, H)), torch.Size((H,))
        self._n, self._stats, self._flags = _ptr(self.n), _ptr(self.stats), _ptr(self.err_flags)
        if train:
            self.workspace = torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=dev)
            self.workspace_bytes = int(nbytes)
            d_h = torch.empty((T, H), dtype=dtype, device=dev)
            own = block and (p > 0 or dtype != torch.bfloat16)
            d_y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if own else None
            g = self.grads = LayerNormGrads(d_h=d_h, d_y=d_y if own else d_h if block else None,
                                            d_w=torch.empty(H, **f32) if weight else None, d_b=torch.empty(H, **f32) if bias else None)
            self._outputs = (_ptr(d_h), _ptr(d_y), _ptr(g.d_w), _ptr(g.d_b), _ptr(self.workspace), self.workspace_bytes, self._flags)

    def forward(self, h: torch.Tensor, y: torch.Tensor | None = None, w: torch.Tensor | None = None, b: torch.Tensor | None = None,
                rng: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
        """Returns (h_out, n).  rng i64 [2] on the device (seed, step); None:
        nothing is dropped."""
        if (y is None) is self.block or (w is None) is self.weight or (b is None) is self.bias:
            for t, wanted, name in ((y, self.block, "y"), (w, self.weight, "w"), (b, self.bias, "b")):
                if (t is not None) != wanted:
                    raise ValueError(f"{name} is {'missing' if wanted else 'not part of this norm'}")
        _on_current(self.n, "the norm")
        f32 = torch.float32
        hp, ld_h = _rows_ptr(h, self.dtype, "h", self._shape)
        yp, ld_y = _rows_ptr(y, torch.bfloat16, "y", self._shape)
        st = self._lib.ep_layer_norm(
            self._ref, hp, ld_h, yp, ld_y, _shaped_ptr(w, f32, "w", self._row), _shaped_ptr(b, f32, "b", self._row),
            _shaped_ptr(rng, torch.int64, "rng", _PAIR), None if self.h_out is None else self.h_out.data_ptr() or None, self._n,
            self._stats, self._flags, _stream(stream))
        if st:
            check(st, "ep_layer_norm")
        return (self.h_out if self.block else h), self.n

    def backward(self, h_out: torch.Tensor, w: torch.Tensor | None, d_n: torch.Tensor, d_h_out: torch.Tensor | None = None,
                 rng: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> LayerNormGrads:
        """Gradients of the last forward(), from its h_out (h where the norm has
        no block), the same w and rng, and the gradients of its outputs (d_h_out
        may be None: zero).  The rows' statistics are those that the last
        forward() left in `stats`: two forward() calls before their backward()
        calls need a LayerNorm each, a copy of h_out is not enough."""
        if not self.train:
            raise ValueError("this norm was made without train=True")
        if (w is None) is self.weight:
            raise ValueError(f"w is {'missing' if self.weight else 'not part of this norm'}")
        _on_current(self.n, "the norm")
        hp, ld_h = _rows_ptr(h_out, self.dtype, "h_out", self._shape)
        st = self._lib.ep_layer_norm_backward(
            self._ref, hp, ld_h, _shaped_ptr(w, torch.float32, "w", self._row), _shaped_ptr(rng, torch.int64, "rng", _PAIR), self._stats,
            _shaped_ptr(d_h_out, self.dtype, "d_h_out", self._shape), _shaped_ptr(d_n, torch.bfloat16, "d_n", self._shape),
            *self._outputs, _stream(stream))
        if st:
            check(st, "ep_layer_norm_backward")
        return self.grads


def _held(E: int, counts, offsets):
    return _shaped_ptr(counts, torch.int32, "counts", (E,)), _shaped_ptr(offsets, torch.int32, "offsets", (E + 1,))


def quant_i8(x: torch.Tensor, counts: torch.Tensor | None = None, offsets: torch.Tensor | None = None, capacity: int | None = None,
             out: torch.Tensor | None = None, scales: torch.Tensor | None = None, err_flags: torch.Tensor | None = None,
             stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Rows of the receive buffer to 8-bit integers with a scale each
    (ep_quant_i8): x bf16 [R, K] -> (codes i8 [R, K], scales f32 [R]).

    counts / offsets from the layout, capacity as in Plan; neither: all rows.
    Rows without a copy are left as they were (without `out`, undefined)."""
    lib = load()
    if x.dim() != 2:
        raise ValueError(f"x must be [R, K], got {tuple(x.shape)}")
    R, K = x.shape
    if capacity is not None and counts is None:
        raise ValueError("a capacity buffer needs the layout's counts")
    if capacity is None and offsets is None and counts is not None:
        raise ValueError("packed rows need the layout's offsets")
    E = _int32(counts.numel() if counts is not None else offsets.numel() - 1 if offsets is not None else 1, "E")
    mode, capacity = (PACKED, 0) if capacity is None else (CAPACITY, _int32(capacity, "capacity"))
    _int32(K, "K")
    xp, ld = _rows_ptr(x, torch.bfloat16, "x", (R, K))
    held = _held(E, counts, offsets)
    if out is None:
        out = _empty((R, K), torch.int8, x.device, stream)
    if scales is None:
        scales = _empty((R,), torch.float32, x.device, stream)
    st = lib.ep_quant_i8(E, K, mode, capacity, R, *held, xp, ld,
                         _shaped_ptr(out, torch.int8, "out", (R, K)), _shaped_ptr(scales, torch.float32, "scales", (R,)),
                         _shaped_ptr(err_flags, torch.int32, "err_flags", (1,)), _stream(stream))
    if st:
        check(st, "ep_quant_i8")
    return out, scales


class I8Weights:
    """8-bit weights with a scale for each output channel, laid out for
    expert_i8 (ep_i8_pack).

    codes i8 [E, rows, K]; scales f32 [E, rows].  paired: rows are N gate rows
    and then N up rows of a SwiGLU.  They take the codes' bytes with K, and rows
    (N of a pair), made up to multiples of 128 (64).  They are packed on `stream`, whose memory
    they are: wait for it before products on another one, and before codes and
    scales are overwritten.  Codes and scales are not needed afterwards and may
    be dropped at once.
    """

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, paired: bool = False, stream: torch.cuda.Stream | None = None):
        lib = load()
        if codes.dim() != 3:
            raise ValueError(f"codes must be [E, rows, K], got {tuple(codes.shape)}")
        E, rows, K = codes.shape
        if paired and rows % 2:
            raise ValueError(f"paired weights have an even number of rows, got {rows}")
        self.E, self.N, self.K, self.paired = E, rows // 2 if paired else rows, K, paired
        self.desc = I8(_int32(E, "E"), _int32(self.N, "N"), _int32(K, "K"), int(paired))
        self._ref = ctypes.byref(self.desc)
        nbytes = lib.ep_i8_bytes(self._ref)
        if nbytes == ctypes.c_size_t(-1).value:
            check(1, "ep_i8_bytes")
        cp = _shaped_ptr(codes, torch.int8, "codes", (E, rows, K))
        sp = _shaped_ptr(scales, torch.float32, "scales", (E, rows))
        self.packed = _empty(int(nbytes), torch.uint8, codes.device, stream)
        if stream is not None:
            for t in (codes, scales):
                t.record_stream(stream)         # the allocator does not hand them out again before they are packed
        self._lib, self._packed = lib, _ptr(self.packed)
        check(lib.ep_i8_pack(self._ref, cp, sp, self._packed, _stream(stream)), "ep_i8_pack")


def expert_i8(x: torch.Tensor, x_scales: torch.Tensor, weights: I8Weights, counts: torch.Tensor | None = None,
              offsets: torch.Tensor | None = None, capacity: int | None = None, max_rows: int | None = None,
              out: torch.Tensor | None = None, err_flags: torch.Tensor | None = None,
              stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Every expert's product over its rows of the receive buffer in 8-bit
    integers (ep_expert_i8).

    x i8 [R, K] and x_scales f32 [R], as quant_i8 gives them; the rest as in
    expert_w4.  Returns bf16 [R, N]; rows without a copy are left as they were
    (without `out`, undefined)."""
    w = weights
    if x.dim() != 2 or x.shape[1] != w.K:
        raise ValueError(f"x must be [R, {w.K}], got {tuple(x.shape)}")
    if w.E == 1 and capacity is None and offsets is None and counts is not None:
        raise ValueError("packed rows need the layout's offsets")
    R = x.shape[0]
    mode, capacity = (PACKED, 0) if capacity is None else (CAPACITY, _int32(capacity, "capacity"))
    _on_current(w.packed, "weights")
    xp, sp = _shaped_ptr(x, torch.int8, "x", (R, w.K)), _shaped_ptr(x_scales, torch.float32, "x_scales", (R,))
    if counts is None and offsets is None and w.E != 1:
        raise ValueError("several experts need the layout's counts and offsets")
    held = _held(w.E, counts, offsets)
    if out is None:
        out = _empty((R, w.N), torch.bfloat16, x.device, stream)
    st = w._lib.ep_expert_i8(
        w._ref, w._packed, mode, capacity, R, R if max_rows is None else max_rows,
        *held, xp, sp, _shaped_ptr(out, torch.bfloat16, "out", (R, w.N)),
        _shaped_ptr(err_flags, torch.int32, "err_flags", (1,)), _stream(stream))
    if st:
        check(st, "ep_expert_i8")
    return out
