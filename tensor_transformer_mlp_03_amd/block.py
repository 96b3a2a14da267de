"""What stands around one MLP in a training or serving step, as objects that a program
keeps between steps: the edge between two blocks (norms, gate, residual scale), the route of
tokens to experts and back, and the global gradient norm with clipping.

Each holds its parameters, index buffers and workspace; every call takes the caller's inputs
and outputs, enqueues kernels on a stream (the current one by default) and returns.  No
arithmetic happens here.  Buffers and workspaces belong to one stream at a time: a program
that uses an object on two streams orders them itself, and two threads do not call one
object at once, but for Edge.forward, which holds no buffer.  Route and GradClip make theirs
when they are made, on the current stream, as torch does any tensor's: a program that uses
them on another one makes them under it, or orders the two.  Edge makes its backward's with
the first call of a size, on the stream of that call.
"""
from __future__ import annotations

from . import _lib as L


def _capturing():
    import torch
    return torch.cuda.is_current_stream_capturing()


def _on(stream, device):
    """Makes the stream that a call is given the current one: what is allocated then is that stream's."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = L._stream(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


class Edge:
    """The edge between two blocks:  r' = alpha r + gate * N_post(y),  x = N_pre(r').

    ``post`` and ``pre``: "none", "rms" or "layer".  The norms' vectors and the gate are all
    float32 or all bf16 tensors and are read where they lie, so an optimizer's update in place
    is seen by the next call.  ``gate``: [H], or [G, H] with one row for each ``gate_rows``
    consecutive tokens.
    """

    def __init__(self, H, post="none", pre="none", w_post=None, b_post=None, w_pre=None, b_pre=None, gate=None,
                 gate_rows=0, alpha=1.0, eps=1e-5):
        self.params = {k: t for k, t in (("w_post", w_post), ("b_post", b_post), ("w_pre", w_pre), ("b_pre", b_pre),
                                         ("gate", gate)) if t is not None}
        self.desc = L.edge_desc(H, post, pre, w_post, b_post, w_pre, b_pre, gate, gate_rows, alpha, eps)
        self.grads, self._grad_args, self._ws, self._M = {}, {}, None, -1
        self._captured = {}  # buffers that graphs write to, which another M replaces, each once, by identity
        self._stream, self._several = None, False  # of the last backward; whether there were several

    def forward(self, y, r, r_out, x, stream=None):
        """y [M,H] float32 or bf16 (None: no block before); r, r_out [M,H] (r_out may be r);
        x [M,H] bf16 (None without a norm before the next block)."""
        L.tpmlp_edge_fwd(self.desc, y, r, r_out, x, stream)

    def backward(self, y, r_out, dr_out, dx, dr, dy, stream=None):
        """Gradients from r_out as the forward wrote it, dr_out (None: zeros) and dx [M,H]
        float32 or bf16.  Writes dr (may be dr_out) and dy (bf16) and returns the parameters'
        float32 gradients by name, which the next backward overwrites.  What a backward that
        is captured into a graph writes to stays allocated as long as this object does."""
        if stream is None:
            self._ready(dr)
        else:
            with _on(stream, dr.device):
                self._ready(dr)
        L.tpmlp_edge_bwd(self.desc, y, r_out, dr_out, dx, dr, dy, ws=self._ws, stream=stream, **self._grad_args)
        return self.grads

    def _ready(self, dr):
        """Buffers for dr's rows.  The current stream is the call's: another M's buffers go back to the stream that
        they were made on, where they are free once what ran before is done, and are marked as used on others."""
        M = dr.shape[0]
        if M != self._M:
            self._place(M, dr.device)
        if dr.is_cuda and L._current_stream() != self._stream:
            self._several, self._stream = self._stream is not None, L._current_stream()
        if self._several:
            import torch
            stream = torch.cuda.current_stream()
            for t in (self._ws, *self.grads.values()):
                t.record_stream(stream)
        if _capturing():
            self._captured.update((id(t), t) for t in (self._ws, *self.grads.values()))

    def _place(self, M, device):
        import torch
        d = self.desc
        f32 = dict(dtype=torch.float32, device=device)
        self.grads = dict(self.grads)  # the last one's holder keeps its tensors
        for k in self.params:
            shape = (-(-M // d.gate_rows), d.H) if k == "gate" else (d.H,)
            if k not in self.grads or self.grads[k].shape != shape:
                self.grads[k] = torch.empty(shape, **f32)
        self._grad_args = {"d" + k: t for k, t in self.grads.items()}
        n = L.tpmlp_edge_bwd_workspace_bytes(d, M)
        if self._ws is None or self._ws.numel() < n:
            self._ws = torch.empty(max(n, 16), dtype=torch.uint8, device=device)
        self._M = M


class Route:
    """T tokens' K choices among E experts: the pairs sorted by expert into segments of a
    multiple of ``align`` rows, and the moves there and back.

    ``rows``: rows of the sorted buffers.  After ``sort``, expert e's rows are ``offsets[e]``
    onward, ``counts[e]`` of them tokens and the rest of its segment zeros; with a ``capacity``
    the segments start at multiples of it, and an expert's later pairs are dropped.
    """

    def __init__(self, T, K, E, align=8, capacity=0, device="cuda"):
        import torch
        self.T, self.K, self.E, self.align, self.capacity = T, K, E, align, capacity
        self.rows = L.tpmlp_route_rows(T, K, E, align, capacity)
        if self.rows < 0:
            raise ValueError(f"no route of T={T} K={K} E={E} align={align} capacity={capacity}")
        i32 = dict(dtype=torch.int32, device=device)
        self.counts, self.offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        self.row_of, self.src_of = torch.empty((T, K), **i32), torch.empty(self.rows, **i32)
        n = L.tpmlp_route_workspace_bytes(T, K, E)
        self.ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None

    def sort(self, ids, stream=None):
        """ids [T,K] int32 or int64; an id outside 0 .. E-1 drops the pair."""
        if tuple(ids.shape) != (self.T, self.K):
            raise ValueError(f"ids has shape {tuple(ids.shape)}, expected {(self.T, self.K)}")
        L.tpmlp_route_sort(ids, self.E, self.align, self.capacity, self.counts, self.offsets, self.row_of, self.src_of,
                           self.ws, stream)

    def dispatch(self, X, Xs, stream=None):
        """Xs [rows,H] = X [T,H] in the sorted order (bf16), zeros on padding."""
        L.tpmlp_route_dispatch(X, self.row_of, self.src_of, Xs, stream)

    def dispatch_backward(self, dXs, dX, stream=None):
        """dX [T,H] = sum of dXs over each token's rows."""
        L.tpmlp_route_combine(dXs, self.row_of, None, dX, stream)

    def combine(self, Zs, w, Y, stream=None):
        """Y [T,H] = sum over k of w[t,k] Zs[row of (t,k)]; w [T,K] float32."""
        L.tpmlp_route_combine(Zs, self.row_of, w, Y, stream)

    def combine_backward(self, dY, Zs, w, dZs, dw, stream=None):
        """dZs [rows,H] (bf16, the experts' dZ) and dw [T,K] from dY [T,H]."""
        L.tpmlp_route_combine_bwd(dY, Zs, self.row_of, self.src_of, w, dZs, dw, stream)


class GradClip:
    """The global norm of a list of gradients and their clipping, in place or into ``outs``.

    One rank that holds all of them calls ``clip``.  Ranks that hold different parameters call
    ``sumsq``, add the one float64 over the ranks (an all-reduce), and call ``scale``.
    """

    def __init__(self, grads, outs=None):
        import torch
        self.table = L.GradTable(grads, outs)
        device = self.table.grads[0].device if self.table.n else "cuda"
        self.norm = torch.empty((), dtype=torch.float32, device=device)
        self.total = torch.empty((), dtype=torch.float64, device=device)
        self.ws = torch.empty(L.tpmlp_grad_workspace_bytes(self.table), dtype=torch.uint8, device=device)

    def clip(self, max_norm, scale=1.0, stream=None):
        """Scales by ``scale`` and so that the norm is at most ``max_norm``; returns the norm
        before clipping (a float32 tensor, overwritten by the next call)."""
        L.tpmlp_clip_grad_norm(self.table, max_norm, self.norm, self.ws, scale, stream)
        return self.norm

    def sumsq(self, stream=None):
        """The sum of squares of this rank's gradients (a float64 tensor)."""
        L.tpmlp_grad_sumsq(self.table, self.total, self.ws, stream)
        return self.total

    def scale(self, max_norm, scale=1.0, stream=None):
        """Clips by the norm that ``sumsq``'s tensor gives; returns that norm."""
        L.tpmlp_grad_clip(self.table, self.total, max_norm, self.norm, scale, stream)
        return self.norm
