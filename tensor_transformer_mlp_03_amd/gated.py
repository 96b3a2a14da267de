"""A gated feed-forward block in training and in serving, as objects that a program keeps: the
gated MLP, dropout in front of the residual's addition, and products with 4-bit weights (the
edge that feeds these in 8 bits is ``block.Edge.forward_fp8``).

Each holds its weights, which are read where they lie, and its workspace; every call takes the
caller's inputs and outputs, enqueues kernels on a stream (the current one by default) and
returns.  No arithmetic happens here.  A workspace is made by the first call of a size on the
stream of that call and belongs to one stream at a time, as block.py's buffers do: a program
that uses an object on two streams orders them itself, and two threads do not call one object
at once.  Dropout.forward and Fp4Linear use none.
"""
from __future__ import annotations

from . import _lib as L
from .block import _capturing, _on


class _Workspace:
    """Device memory that calls on one stream after another write to.  What a captured graph writes
    to stays allocated as long as this object does."""

    def __init__(self):
        self._ws, self._captured = None, {}
        self._stream, self._several = None, False  # of the last call; whether there were several

    def get(self, n, device, stream):
        if stream is None:
            return self._get(n, device)
        with _on(stream, device):
            return self._get(n, device)

    def _get(self, n, device):
        import torch
        if self._ws is None or self._ws.numel() < n or self._ws.device != device:
            self._ws = torch.empty(max(n, 16), dtype=torch.uint8, device=device)
        if self._ws.is_cuda:
            if L._current_stream() != self._stream:
                self._several, self._stream = self._stream is not None, L._current_stream()
            if self._several:
                self._ws.record_stream(torch.cuda.current_stream())
            if _capturing():
                self._captured[id(self._ws)] = self._ws
        return self._ws


def _used(stream, *tensors):
    """Marks tensors as used on the stream that a call was given: one that is freed goes back to the
    stream that it was made on when what the other does by now is done."""
    import torch
    with _on(stream, tensors[0].device):
        for t in (t for t in tensors if t.is_cuda):
            t.record_stream(torch.cuda.current_stream())


class GatedMLP:
    """One rank's gated MLP:  [P_g | P_u] = X A,  Z = (act(P_g) * P_u) B.

    ``A`` [H, 2F] bf16: the gate weight's and the up weight's columns side by side; ``B`` [F, H]
    bf16.  ``act``: "silu", "gelu", "relu" or "sigmoid".
    """

    def __init__(self, A, B, act="silu"):
        self.H, self.F = L._glu_sizes(A, B)
        if act not in L.ACTS or act == "none":
            raise ValueError(f"no gate {act!r}")
        self.A, self.B, self.act = A, B, act
        self._sizes = {}
        self._ws = _Workspace()

    def forward(self, X, Z, P=None, stream=None):
        """Z [M,H] (float32 or bf16) from X [M,H] bf16; P [M,2F] bf16 receives the pre-activations
        for a backward that keeps them."""
        M = X.shape[0]
        ws = self._ws.get(self._bytes(M, None), X.device, stream)
        L.tpmlp_glu_fwd(X, self.A, self.B, Z, P, self.act, ws, stream)

    def backward(self, dZ, X, P, dX, dA, dB, stream=None):
        """dX [M,H] and the weights' gradients dA, dB (each float32 or bf16) from dZ [M,H] bf16; P
        as the forward left it, or None to make it again, in float32."""
        M = X.shape[0]
        ws = self._ws.get(self._bytes(M, P is None), X.device, stream)
        L.tpmlp_glu_bwd(dZ, X, self.A, self.B, P, dX, dA, dB, self.act, ws, stream)

    def _bytes(self, M, recompute):
        n = self._sizes.get((M, recompute))
        if n is None:
            if recompute is None:
                n = L.tpmlp_glu_fwd_workspace_bytes(M, self.H, self.F)
            else:
                n = L.tpmlp_glu_bwd_workspace_bytes(M, self.H, self.F, recompute)
            if len(self._sizes) > 4096:
                self._sizes.clear()
            self._sizes[(M, recompute)] = n
        return n


class Dropout:
    """Dropout with a bias, added to the residual stream:  out = r + mask * (y + bias) / (1 - p).

    ``state``: two int64 values on the GPU, the seed and the step, which the kernels read: a
    program advances the step in place between steps, inside a captured graph too, and leaves it
    as it was between a forward and its backward.  ``site`` tells several dropouts of one step
    apart.  A rank that holds rows ``first_row`` onward drops what one that holds all rows does.
    """

    def __init__(self, p, state, site=0, bias=None):
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be from 0 to 1")
        self.p, self.state, self.site, self.bias = p, state, site, bias
        self._ws = _Workspace()

    def forward(self, y, r, out, first_row=0, stream=None):
        """out [M,H] (may be r, or y) from y [M,H] and r [M,H] (None: nothing is added), float32 or bf16."""
        L.tpmlp_dropout_fwd(y, self.bias, r, out, self.p, self.state, self.site, first_row, stream)

    def backward(self, dout, dy, db=None, first_row=0, stream=None):
        """dy [M,H] (may be dout) and, if given, the bias's gradient db [H] float32.  The gradient of
        r is dout itself."""
        ws = None
        if db is not None:
            ws = self._ws.get(L.tpmlp_dropout_bwd_workspace_bytes(*dout.shape), dout.device, stream)
        L.tpmlp_dropout_bwd(dout, dy, db, self.p, self.state, self.site, first_row, ws, stream)


class Fp4Linear:
    """A product with 4-bit weights:  Y = act(X W^T), or gated  Y = act(X W_g^T) * (X W_u^T).

    ``codes`` [N, K / 2] uint8 (or float4_e2m1fn_x2), two E2M1 values a byte, the lower k in the low half;
    ``scales`` [N, K / 32] uint8 (or float8_e8m0fnu), 2^(e - 127) for every 32 values; gated: W_g's rows,
    then W_u's.  They are copied into the order that the kernels read, on ``stream``, and not kept: their
    memory is not used anew before that is done.
    """

    def __init__(self, codes, scales, act="none", gated=False, stream=None):
        import torch
        rows, k2 = codes.shape
        self.K, self.N = 2 * k2, rows // 2 if gated else rows
        if self.K % 32 or (gated and rows % 2):
            raise ValueError(f"no 4-bit weight of {rows} rows of {self.K}")
        if tuple(scales.shape) != (rows, self.K // 32):
            raise ValueError(f"scales has shape {tuple(scales.shape)}, expected {(rows, self.K // 32)}")
        if act not in L.ACTS:
            raise ValueError(f"no activation {act!r}")
        self.act, self.gated = act, gated
        n = L.tpmlp_fp4_packed_bytes(self.N, self.K, gated)
        if stream is None:
            self.packed = torch.empty(n, dtype=torch.uint8, device=codes.device)
        else:
            with _on(stream, codes.device):
                self.packed = torch.empty(n, dtype=torch.uint8, device=codes.device)
        L.tpmlp_fp4_pack(codes, scales, self.packed, gated, stream)
        if self.packed.is_cuda:
            self._made = L._stream(stream)
            self._pinned = None if scales.is_cuda else scales  # in host memory that no stream keeps
            if stream is not None:
                _used(stream, codes, scales)

    _made = None  # the stream that ``packed`` was made on

    @classmethod
    def from_weight(cls, W, act="none", gated=False, stream=None):
        """From a bf16 weight [K, N] as the MLP's lie: A [H, F] or A [H, 2F] (gated), B [F, H]."""
        import torch
        K, N = W.shape
        if K % 32:
            raise ValueError(f"a weight of {K} rows has no blocks of 32")
        if stream is not None:
            with _on(stream, W.device):
                made = cls.from_weight(W, act, gated)
            if W.is_cuda:
                _used(stream, W)
            return made
        codes = torch.empty(N, K // 2, dtype=torch.uint8, device=W.device)
        scales = torch.empty(N, K // 32, dtype=torch.uint8, device=W.device)
        L.tpmlp_fp4_quantize(W, codes, scales)
        return cls(codes, scales, act, gated)

    def forward(self, X, Y, x_scales=None, stream=None):
        """Y [M,N] (float32 or bf16) from X [M,K]: bf16, or E4M3 codes with x_scales as
        ``block.Edge.forward_fp8`` writes them."""
        if X.shape[1] != self.K or Y.shape[1] != self.N:
            raise ValueError(f"X {tuple(X.shape)} and Y {tuple(Y.shape)} do not fit a weight of {self.N} by {self.K}")
        L.tpmlp_fp4_fwd(X, x_scales, self.packed, Y, self.act, self.gated, stream)
        if self.packed.is_cuda and L._stream(stream) != self._made:
            import torch
            _used(torch.cuda.current_stream() if stream is None else stream, self.packed)
