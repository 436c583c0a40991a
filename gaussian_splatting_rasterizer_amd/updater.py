"""Building blocks of the learned updater that consumes the score tokens: a gated
feed-forward block, a gated linear recurrence (the hidden state carried from
update to update) and the orthogonalisation of a weight's update.

Each class checks its tensors, owns the workspace its calls need (grown when a
call needs more) and runs on the current stream or the one given; like a
Rasterizer, an object is used from one thread and one stream at a time.  With a
stream given, the caller orders it with the current one (wait_stream, both
ways); tensors of either may be dropped as soon as the call has returned.  The
backward passes are explicit calls, as in Rasterizer.backward.
"""
from __future__ import annotations

from . import binding as b

_ACTIVATIONS = {"silu": b.GS_ACT_SILU, "gelu": b.GS_ACT_GELU}


def _dtype_code(dtype, allowed=("float32", "bfloat16", "float16")):
    name = str(dtype).replace("torch.", "")
    if name not in allowed:
        raise ValueError(f"dtype {dtype} is not supported (one of {', '.join(allowed)})")
    return {"float32": b.GS_F32, "bfloat16": b.GS_BF16, "float16": b.GS_F16}[name]


def _matrix(t, name, rows, cols, dtype, device):
    """Checks a [rows, cols] device tensor whose rows are contiguous and do not overlap; returns its row stride."""
    if t.dim() != 2 or tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{rows}, {cols}]")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    step, along = t.stride()
    if (cols > 1 and along != 1) or (rows > 1 and step < cols):
        raise ValueError(f"{name} needs contiguous rows that do not overlap (strides {t.stride()})")
    return step if rows > 1 else cols


def _exact(t, name, shape, dtype, device):
    """Checks a contiguous device tensor of one shape."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


class _Op:
    """A device, and scratch memory that grows when a call needs more (released in the order of the streams that used
    it).  A captured graph goes on using the scratch memory it was captured with: the object keeps that memory as long
    as it lives, so it has to outlive the graph."""

    _captured = False  # a captured graph uses the workspace
    _kept = ()         # earlier workspaces that captured graphs use
    _held = ()         # tensors that every call uses beside its arguments

    def __init__(self, device):
        import torch
        b.load_library()
        self.torch = torch
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"the tensors must be on a GPU, got {self.device}")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.workspace = None
        self._home = None  # the stream the workspace was allocated on

    def _scratch(self, nbytes, stream):
        if self.workspace is None or self.workspace.numel() < nbytes:
            if self._captured:
                self._kept = (*self._kept, self.workspace)
                self._captured = False
            self.workspace = self.torch.empty(max(int(nbytes), 256), dtype=self.torch.uint8, device=self.device)
            self._home = stream.cuda_stream
        elif stream.cuda_stream != self._home:
            self.workspace.record_stream(stream)
        if self.torch.cuda.is_current_stream_capturing():
            self._captured = True
        return self.workspace

    def _on(self, stream, call, *args):
        """call(stream, *args) with the stream and its device current, for allocations and the launch."""
        t = self.torch
        current = t.cuda.current_stream(self.device)
        if (stream is None or stream == current) and t.cuda.current_device() == self.device.index:
            return call(current, *args)
        if stream is None or stream == current:
            with t.cuda.stream(current), t.cuda.device(self.device):
                return call(current, *args)
        with t.cuda.stream(stream), t.cuda.device(self.device):
            out = call(stream, *args)
        # the allocator reuses a tensor in the order of its own stream: tell it of the other one
        for v in self._tensors(args, self._held):
            v.record_stream(stream)
        for v in self._tensors(out):
            v.record_stream(current)
        return out

    def _tensors(self, *values):
        for v in values:
            if isinstance(v, self.torch.Tensor):
                yield v
            elif isinstance(v, (tuple, list)):
                yield from self._tensors(*v)
            elif isinstance(v, dict):
                yield from self._tensors(*v.values())


class GatedFFN(_Op):
    """y = (act(x w_gate^T) * (x w_up^T)) w_down^T.

    w_gate, w_up [d_hidden, d_in] and w_down [d_out, d_hidden], contiguous, one type (float32, bfloat16 or float16);
    they are borrowed, not copied: updating them in place is seen by the next call.
    """

    def __init__(self, w_gate, w_up, w_down, activation="silu"):
        super().__init__(w_gate.device)
        if activation not in _ACTIVATIONS:
            raise ValueError(f"activation {activation!r} is not one of {', '.join(_ACTIVATIONS)}")
        if w_gate.dim() != 2 or w_down.dim() != 2:
            raise ValueError("weights must be matrices")
        self.dtype = w_gate.dtype
        self.code = _dtype_code(self.dtype)
        self.activation = _ACTIVATIONS[activation]
        self.d_hidden, self.d_in = (int(v) for v in w_gate.shape)
        self.d_out = int(w_down.shape[0])
        self.w_gate = _exact(w_gate, "w_gate", (self.d_hidden, self.d_in), self.dtype, self.device)
        self.w_up = _exact(w_up, "w_up", (self.d_hidden, self.d_in), self.dtype, self.device)
        self.w_down = _exact(w_down, "w_down", (self.d_out, self.d_hidden), self.dtype, self.device)
        self._held = (self.w_gate, self.w_up, self.w_down)
        self._sizes = {}

    @property
    def _weights(self):
        return b.gs_ffn_weights(self.w_gate.data_ptr(), self.w_up.data_ptr(), self.w_down.data_ptr())

    def _dims(self, rows):
        """(dims, sizes) for a number of rows."""
        if rows not in self._sizes:
            if len(self._sizes) > 64:
                self._sizes.clear()
            d = b.gs_ffn_dims(rows, self.d_in, self.d_hidden, self.d_out, self.code, self.activation)
            self._sizes[rows] = (d, b.gs_ffn_sizes(d))
        return self._sizes[rows]

    def forward(self, x, y=None, save=False, stream=None):
        """x [rows, d_in] -> y [rows, d_out]; with save, (y, saved) for backward."""
        return self._on(stream, self._forward, x, y, save)

    def _forward(self, stream, x, y, save):
        rows = int(x.shape[0])
        ldx = _matrix(x, "x", rows, self.d_in, self.dtype, self.device)
        dims, (n_saved, n_ws, _) = self._dims(rows)
        empty = self.torch.empty
        if y is None:
            y = empty((rows, self.d_out), dtype=self.dtype, device=self.device)
            ldy = self.d_out
        else:
            ldy = _matrix(y, "y", rows, self.d_out, self.dtype, self.device)
        saved = empty(max(n_saved, 256), dtype=self.torch.uint8, device=self.device) if save else None
        b.gs_ffn_forward(dims, x, ldx, self._weights, y, ldy, saved, self._scratch(n_ws, stream), stream)
        return (y, saved) if save else y

    def new_grads(self, rows):
        """Gradient tensors of a backward pass over `rows` rows."""
        like = dict(dtype=self.dtype, device=self.device)
        return {"x": self.torch.empty((rows, self.d_in), **like),
                "w_gate": self.torch.empty_like(self.w_gate), "w_up": self.torch.empty_like(self.w_up),
                "w_down": self.torch.empty_like(self.w_down)}

    def backward(self, x, saved, dy, grads=None, stream=None):
        """Gradients for dL/dy = dy [rows, d_out]: a dict of x, w_gate, w_up, w_down (written; with a given dict, only
        the tensors it holds)."""
        return self._on(stream, self._backward, x, saved, dy, grads)

    def _backward(self, stream, x, saved, dy, grads):
        rows = int(x.shape[0])
        ldx = _matrix(x, "x", rows, self.d_in, self.dtype, self.device)
        lddy = _matrix(dy, "dy", rows, self.d_out, self.dtype, self.device)
        dims, (n_saved, _, n_ws) = self._dims(rows)
        if saved is None or saved.numel() < n_saved or saved.device != self.device:
            raise ValueError("saved is not what forward(x, save=True) returned for these rows")
        ld_gx = self.d_in
        if grads is None:
            grads = self.new_grads(rows)
        else:
            if grads.get("x") is not None:
                ld_gx = _matrix(grads["x"], "grads['x']", rows, self.d_in, self.dtype, self.device)
            for name in ("w_gate", "w_up", "w_down"):
                if grads.get(name) is not None:
                    _exact(grads[name], f"grads[{name!r}]", getattr(self, name).shape, self.dtype, self.device)
        ptr = {k: grads[k].data_ptr() if grads.get(k) is not None else None for k in ("x", "w_gate", "w_up", "w_down")}
        out = b.gs_ffn_grads(ptr["x"], ld_gx, ptr["w_gate"], ptr["w_up"], ptr["w_down"])
        b.gs_ffn_backward(dims, x, ldx, self._weights, saved, dy, lddy, out, self._scratch(n_ws, stream), stream)
        return grads


class GatedScan(_Op):
    """h_t = sigma(gate_t) h_{t-1} + (1 - sigma(gate_t)) x_t per channel, over sequences that lie one after another.

    gate, x, y [rows, channels] in dtype (float32, bfloat16 or float16), rows contiguous; states float32
    [n_seq, channels].  offsets: int64 [n_seq + 1] on the GPU (first row of each sequence, then rows), or None for
    sequences of equal length, as many as h0 has rows (one without h0).
    """

    def __init__(self, channels, dtype, device="cuda"):
        super().__init__(device)
        self.channels = int(channels)
        self.dtype = dtype
        self.code = _dtype_code(dtype)
        self._sizes = {}

    def _setup(self, gate, x, h0, offsets):
        t = self.torch
        rows, c = int(gate.shape[0]), self.channels
        ldz = _matrix(gate, "gate", rows, c, self.dtype, self.device)
        ldx = _matrix(x, "x", rows, c, self.dtype, self.device)
        if offsets is not None:
            if offsets.dim() != 1 or offsets.shape[0] < 1:
                raise ValueError("offsets must have n_seq + 1 entries")
            n_seq = int(offsets.shape[0]) - 1
            _exact(offsets, "offsets", (n_seq + 1,), t.int64, self.device)
        else:
            n_seq = int(h0.shape[0]) if h0 is not None else 1
        if h0 is not None:
            _exact(h0, "h0", (n_seq, c), t.float32, self.device)
        key = (rows, n_seq)
        if key not in self._sizes:
            if len(self._sizes) > 64:
                self._sizes.clear()
            d = b.gs_scan_dims(rows, n_seq, c, self.code)
            self._sizes[key] = (d, b.gs_scan_sizes(d))
        dims, sizes = self._sizes[key]
        inputs = b.gs_scan_inputs(gate.data_ptr(), x.data_ptr(), h0.data_ptr() if h0 is not None else None, ldz, ldx)
        return rows, n_seq, dims, sizes, inputs

    def forward(self, gate, x, h0=None, offsets=None, y=None, h_last=None, save=False, stream=None):
        """-> (y, h_last); with save, (y, h_last, saved) for backward.  h_last may be h0 (updated in place;
        backward needs the h0 from before)."""
        return self._on(stream, self._forward, gate, x, h0, offsets, y, h_last, save)

    def _forward(self, stream, gate, x, h0, offsets, y, h_last, save):
        rows, n_seq, dims, (n_saved, n_ws), inputs = self._setup(gate, x, h0, offsets)
        t, c = self.torch, self.channels
        if y is None:
            y = t.empty((rows, c), dtype=self.dtype, device=self.device)
            ldy = c
        else:
            ldy = _matrix(y, "y", rows, c, self.dtype, self.device)
        if h_last is None:
            h_last = t.empty((n_seq, c), dtype=t.float32, device=self.device)
        else:
            _exact(h_last, "h_last", (n_seq, c), t.float32, self.device)
        saved = t.empty(max(n_saved, 256), dtype=t.uint8, device=self.device) if save else None
        b.gs_scan_forward(dims, offsets, inputs, y, ldy, h_last, saved, self._scratch(n_ws, stream), stream)
        return (y, h_last, saved) if save else (y, h_last)

    def backward(self, gate, x, saved, dy, dh_last=None, h0=None, offsets=None, grads=None, stream=None):
        """Gradients for dy [rows, channels] and dh_last [n_seq, channels]: a dict of gate, x, h0 (written; with a
        given dict, only the tensors it holds; its h0 may be dh_last)."""
        return self._on(stream, self._backward, gate, x, saved, dy, dh_last, h0, offsets, grads)

    def _backward(self, stream, gate, x, saved, dy, dh_last, h0, offsets, grads):
        rows, n_seq, dims, (n_saved, n_ws), inputs = self._setup(gate, x, h0, offsets)
        t, c = self.torch, self.channels
        lddy = _matrix(dy, "dy", rows, c, self.dtype, self.device)
        if saved is None or saved.numel() < n_saved or saved.device != self.device:
            raise ValueError("saved is not what forward(..., save=True) returned for these rows")
        if dh_last is not None:
            _exact(dh_last, "dh_last", (n_seq, c), t.float32, self.device)
        ld = {"gate": c, "x": c}
        if grads is None:
            like = dict(dtype=self.dtype, device=self.device)
            grads = {"gate": t.empty((rows, c), **like), "x": t.empty((rows, c), **like),
                     "h0": t.empty((n_seq, c), dtype=t.float32, device=self.device)}
        else:
            for name in ("gate", "x"):
                if grads.get(name) is not None:
                    ld[name] = _matrix(grads[name], f"grads[{name!r}]", rows, c, self.dtype, self.device)
            if grads.get("h0") is not None:
                _exact(grads["h0"], "grads['h0']", (n_seq, c), t.float32, self.device)
        ptr = {k: grads[k].data_ptr() if grads.get(k) is not None else None for k in ("gate", "x", "h0")}
        out = b.gs_scan_grads(ptr["gate"], ptr["x"], ptr["h0"], ld["gate"], ld["x"])
        b.gs_scan_backward(dims, offsets, inputs, saved, dy, lddy, dh_last, out, self._scratch(n_ws, stream), stream)
        return grads


class Orthogonalizer(_Op):
    """Newton-Schulz orthogonalisation of `batch` matrices [rows, cols]: run(g) -> out.

    dtype and out_dtype: float32 or bfloat16.
    """

    def __init__(self, batch, rows, cols, dtype, out_dtype=None, steps=5, coefficients=None, eps=None,
                 device="cuda"):
        super().__init__(device)
        allowed = ("float32", "bfloat16")
        self.dtype, self.out_dtype = dtype, out_dtype if out_dtype is not None else dtype
        self.shape = (int(batch), int(rows), int(cols))
        d = b.gs_default_ortho_dims()
        d.batch, d.rows, d.cols = self.shape
        d.dtype, d.out_dtype = _dtype_code(self.dtype, allowed), _dtype_code(self.out_dtype, allowed)
        d.steps = int(steps)
        if coefficients is not None:
            d.a, d.b, d.c = (float(v) for v in coefficients)
        if eps is not None:
            d.eps = float(eps)
        self.dims = d
        self.nbytes = b.gs_ortho_size(d)

    def run(self, g, out=None, stream=None):
        """g [batch, rows, cols] (or [rows, cols] when batch is 1), contiguous."""
        return self._on(stream, self._run, g, out)

    def _run(self, stream, g, out):
        shape = self.shape if g.dim() != 2 or self.shape[0] != 1 else self.shape[1:]
        _exact(g, "g", shape, self.dtype, self.device)
        if out is None:
            out = self.torch.empty(shape, dtype=self.out_dtype, device=self.device)
        else:
            _exact(out, "out", shape, self.out_dtype, self.device)
        b.gs_orthogonalize(self.dims, g, out, self._scratch(self.nbytes, stream), stream)
        return out
