"""The user-facing objects around the C ABI.

MixedPrecisionLinear owns the packed weight blob (torch device memory), sizes the
workspace, and runs one forward pass with mx_linear (quantize activations,
mixed-precision GEMM) on the current CUDA stream.  MicroscaledLinear is its
counterpart with both operands in microscaled 4-bit floating point, and
MicroscaledExperts a layer of such experts with its routing.  All arithmetic
happens in libmx.so's kernels.
"""
from __future__ import annotations

import torch

from . import binding as mx


class MixedPrecisionLinear:
    """Y = X W^T with W split into 8-bit symmetric / 4-bit asymmetric rows (MixLLM)."""

    def __init__(self, W: torch.Tensor, is8: torch.Tensor, group: int = 128, n8: int | None = None):
        if not W.is_cuda:
            raise ValueError("W must be a CUDA tensor")
        N, K = W.shape
        if n8 is None:
            n8 = int(is8.count_nonzero().item())
        self.layout = mx.mx_layout_init(N, K, group, n8)
        self.blob = torch.empty(self.layout.total_bytes, dtype=torch.uint8, device=W.device)
        self._status = torch.zeros(1, dtype=torch.int32, device=W.device)
        mx.mx_pack_weights(self.layout, W, is8.to(W.device, torch.uint8), self.blob, status=self._status)
        self._ws = {}

    @classmethod
    def from_blob(cls, blob: torch.Tensor) -> "MixedPrecisionLinear":
        """Re-open a packed blob (for example one saved with torch.save)."""
        self = cls.__new__(cls)
        self.layout = mx.mx_layout_from_header(blob[:mx.HEADER_BYTES].cpu())
        if blob.numel() < self.layout.total_bytes:
            raise ValueError("blob shorter than its header says")
        self.blob = blob
        self._status = torch.zeros(1, dtype=torch.int32, device=blob.device)
        self._ws = {}
        return self

    @property
    def N(self) -> int:
        return self.layout.N

    @property
    def K(self) -> int:
        return self.layout.K

    def check_pack_status(self) -> None:
        """Raise if the packer reported an error (mask count mismatch)."""
        st = int(self._status.item())
        if st != 0:
            raise mx.MXError(st, "mx_pack_weights", "device-side error while packing")

    def workspace(self, M: int, xdtype=torch.float16, path: int = 0, act_group: int = 0) -> torch.Tensor | None:
        """Device scratch for mx_linear at M tokens (None when it needs none); cached."""
        key = (M, xdtype, path, act_group)
        if key not in self._ws:
            n = mx.mx_linear_workspace_size(self.layout, M, xdtype, path=path, act_group=act_group)
            self._ws[key] = torch.empty(n, dtype=torch.uint8, device=self.blob.device) if n else None
        return self._ws[key]

    def forward(self, X: torch.Tensor, out: torch.Tensor | None = None, path: int = 0,
                act_group: int = 0) -> torch.Tensor:
        """act_group: 0 -- one activation scale per token; the weight group -- group-wise."""
        M, K = X.shape
        if K != self.K:
            raise ValueError(f"X has K={K}, layer expects {self.K}")
        Y = out if out is not None else torch.empty((M, self.N), dtype=torch.float16, device=self.blob.device)
        mx.mx_linear(self.layout, self.blob, X, Y, workspace=self.workspace(M, X.dtype, path, act_group),
                     path=path, act_group=act_group)
        return Y

    __call__ = forward

    def graphed(self, x_host: torch.Tensor, y_host: torch.Tensor | None = None, path: int = 0,
                act_group: int = 0) -> "GraphedLinear":
        """Capture host-in / host-out calls for this input buffer (see GraphedLinear)."""
        return GraphedLinear(self, x_host, y_host, path, act_group)


class GraphedLinear:
    """A MixedPrecisionLinear call captured once as a CUDA graph for a fixed M.

    The graph copies the pinned host input into the device, runs mx_linear
    (quantize + GEMM, one kernel for decode-sized M) and copies Y back into the
    pinned host output, so one `replay()` per
    step is the whole host-to-host pass with a single launch from the host.
    The copies are kernels that read and write the mapped host buffers
    (mx_copy_mapped), so the graph holds kernels only and mx_linear's weight
    stream starts while the input crosses the bus.
    The caller rewrites `x_host` between replays and reads `y_host` after the
    stream is synchronised (or after an event recorded after `replay()`).
    """

    def __init__(self, layer: MixedPrecisionLinear, x_host: torch.Tensor, y_host: torch.Tensor | None = None,
                 path: int = 0, act_group: int = 0):
        if not x_host.is_pinned():
            raise ValueError("x_host must be pinned host memory")
        if y_host is not None and not y_host.is_pinned():
            raise ValueError("y_host must be pinned host memory")
        M, K = x_host.shape
        dev = layer.blob.device
        self.layer = layer
        self.x_host = x_host
        self.y_host = y_host if y_host is not None else torch.empty((M, layer.N), dtype=torch.float16).pin_memory()
        self.x_dev = torch.empty((M, K), dtype=x_host.dtype, device=dev)
        self.y_dev = torch.empty((M, layer.N), dtype=torch.float16, device=dev)
        ws = layer.workspace(M, x_host.dtype, path, act_group)
        self.stream = torch.cuda.Stream(dev)

        def body():
            mx.mx_copy_mapped(self.x_dev, self.x_host)
            mx.mx_linear(layer.layout, layer.blob, self.x_dev, self.y_dev, workspace=ws, path=path,
                         act_group=act_group)
            mx.mx_copy_mapped(self.y_host, self.y_dev)

        with torch.cuda.stream(self.stream):        # configure kernels outside capture
            body()
        self.stream.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=self.stream):
            body()

    def replay(self) -> None:
        """Launch the captured pass on `self.stream` (a graph replays on the current stream)."""
        with torch.cuda.stream(self.stream):
            self.graph.replay()


KEPT_SIZES = 1024                                # sizes of calls whose host geometry a layer keeps


class _Microscaled:
    """What the microscaled layers hold: the weights, the activations' scale, host geometry by the size of a
    call, and the word in which the kernels report a wait that ran out."""

    def _hold(self, blob: torch.Tensor, act_scale: torch.Tensor | None) -> None:
        self.blob, self.act_scale, self._sizes = blob, act_scale, {}
        self._status = torch.zeros(1, dtype=torch.int32, device=blob.device)

    def _keep(self, key, sizes):
        """Host geometry of a call's size, worked out once; of so many sizes at most."""
        if len(self._sizes) >= KEPT_SIZES:
            self._sizes.clear()
        self._sizes[key] = sizes
        return sizes

    def check_status(self) -> None:
        """Wait for the device and raise if a wait inside a kernel of this layer ran out since the last
        check: an output of that time is then incomplete.  Graphs captured from the layer report here too."""
        if self._status.is_cuda:
            torch.cuda.synchronize(self._status.device)
        st = int(self._status.item())
        if st != 0:
            self._status.zero_()
            raise mx.MXError(st, type(self).__name__, "a wait inside a kernel ran out: an output is incomplete")


class MicroscaledLinear(_Microscaled):
    """Y = X W^T with W and X in microscaled 4-bit floating point (see mx_fp4.h).

    format: mx.FP4_E4M3_16 (blocks of 16, E4M3 scales, one fp32 scale per matrix) or
    mx.FP4_E8M0_32 (blocks of 32, power-of-two scales).  For the first, weight_scale is
    the weights' fp32 scale (device fp32 [1]; None takes it from W with mx_fp4_gscale) and
    act_scale the activations' (device fp32 [1], from calibration).  None is 1: blocks of
    activations below 6 * 2^-6 = 0.094 in size then get fewer bits of scale, and below
    6 * 2^-10 = 0.006 they become zero.  Scratch comes
    from torch's allocator in each call, so calls on several streams, and graphs captured from
    them, share none.  Waits inside the kernels are bounded: a call whose wait ran out leaves parts of
    its output unwritten, which check_status reports.
    """

    def __init__(self, W: torch.Tensor, format: int = mx.FP4_E4M3_16, act_scale: torch.Tensor | None = None,
                 weight_scale: torch.Tensor | None = None):
        if not W.is_cuda:
            raise ValueError("W must be a CUDA tensor")
        if W.dim() != 2:
            raise ValueError(f"W has shape {tuple(W.shape)}, expected [N, K]")
        self.layout = mx.mx_fp4_layout_init(W.shape[0], W.shape[1], format)
        self._hold(_microscaled_weights(self.layout, W, weight_scale), act_scale)

    @classmethod
    def from_blob(cls, blob: torch.Tensor, act_scale: torch.Tensor | None = None) -> "MicroscaledLinear":
        """Re-open a packed blob (for example one saved with torch.save)."""
        self = cls.__new__(cls)
        self.layout = _reopen(blob)
        self._hold(blob, act_scale)
        if self.layout.groups != 1:
            raise ValueError(f"blob holds {self.layout.groups} experts: open it with MicroscaledExperts")
        return self

    @property
    def N(self) -> int:
        return self.layout.rows

    @property
    def K(self) -> int:
        return self.layout.K

    def forward(self, X: torch.Tensor, out: torch.Tensor | None = None, out_dtype=None, path: int = 0) -> torch.Tensor:
        """X [M, K] float32, float16 or bfloat16; the result has out_dtype, or X's dtype."""
        L, blob = self.layout, self.blob
        if X.dim() != 2 or X.shape[1] != L.K:
            raise ValueError(f"X has shape {tuple(X.shape)}, expected [M, {L.K}]")
        M = X.shape[0]
        if out is None:
            out = blob.new_empty((M, L.rows), dtype=out_dtype or X.dtype)
        if M == 0:
            return out
        n = self._sizes.get((M, path))
        if n is None:
            n = self._keep((M, path), mx.mx_fp4_linear_workspace_size(L, M, path))
        ws = blob.new_empty(n) if n else None
        mx.mx_fp4_linear(L, blob, X, out, ws, gscale=self.act_scale, path=path, status=self._status)
        return out

    __call__ = forward


class MicroscaledExperts(_Microscaled):
    """A layer of E experts, each one microscaled 4-bit projection, with its routing.

    W [E, N, K]; weight_scale fp32 [E], else as MicroscaledLinear.  forward(X, ids, weights)
    runs sort, projection and weighted sum in one call; sort, project and combine are its steps,
    for callers that put something between them (an activation function, a second layer of experts
    over the same plan: project with sorted=True) or need the plan for the gradients of the routing
    (mx_experts_combine_bwd, mx_experts_gather_bwd; the product has none).
    """

    def __init__(self, W: torch.Tensor, format: int = mx.FP4_E4M3_16, act_scale: torch.Tensor | None = None,
                 weight_scale: torch.Tensor | None = None):
        if not W.is_cuda:
            raise ValueError("W must be a CUDA tensor")
        if W.dim() != 3:
            raise ValueError(f"W has shape {tuple(W.shape)}, expected [E, N, K]")
        self.layout = mx.mx_fp4_layout_init(W.shape[1], W.shape[2], format, groups=W.shape[0])
        self._hold(_microscaled_weights(self.layout, W, weight_scale), act_scale)

    @classmethod
    def from_blob(cls, blob: torch.Tensor, act_scale: torch.Tensor | None = None) -> "MicroscaledExperts":
        self = cls.__new__(cls)
        self.layout = _reopen(blob)
        self._hold(blob, act_scale)
        return self

    @property
    def E(self) -> int:
        return self.layout.groups

    @property
    def N(self) -> int:
        return self.layout.rows

    @property
    def K(self) -> int:
        return self.layout.K

    def sort(self, ids: torch.Tensor) -> mx.ExpertsPlan:
        """ids int32 [T, k]: each token's experts; ids outside 0 .. E-1 drop the slot."""
        if ids.dim() != 2:
            raise ValueError(f"ids has shape {tuple(ids.shape)}, expected [T, k]")
        P = mx.mx_experts_layout_init(ids.shape[0], ids.shape[1], self.E)
        plan = mx.ExpertsPlan(P, buffer=self.blob.new_empty(P.total_bytes))
        mx.mx_experts_sort(plan, ids)
        return plan

    def project(self, X: torch.Tensor, plan: mx.ExpertsPlan, sorted: bool = False, out: torch.Tensor | None = None,
                out_dtype=torch.float32, path: int = 0) -> torch.Tensor:
        """Each expert's product over its sorted rows, [n, N].  X: token rows [T, K], or with
        sorted=True rows in sorted order [n, K].  Rows behind the kept ones are not written."""
        L, blob, P = self.layout, self.blob, plan.P
        if out is None:
            out = blob.new_empty((P.n, L.rows), dtype=out_dtype)
        if P.n == 0:
            return out
        n = mx.mx_fp4_linear_sorted_workspace_size(L, P, path)
        ws = blob.new_empty(n) if n else None
        mx.mx_fp4_linear_sorted(L, blob, plan, X, out, ws, sorted=sorted, gscale=self.act_scale, path=path,
                                status=self._status)
        return out

    def combine(self, Ys: torch.Tensor, plan: mx.ExpertsPlan, weights: torch.Tensor, out: torch.Tensor | None = None,
                out_dtype=None) -> torch.Tensor:
        """Per token the sum of its rows of Ys times weights (fp32 [T, k])."""
        return mx.mx_experts_combine(plan, Ys, weights, Y=out, out_dtype=out_dtype)

    def forward(self, X: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, out: torch.Tensor | None = None,
                out_dtype=None) -> torch.Tensor:
        """Y [T, N], in one call.  The experts' outputs are held in fp32 between the product and
        the sum, so Y is rounded once."""
        L, blob = self.layout, self.blob
        if ids.dim() != 2:
            raise ValueError(f"ids has shape {tuple(ids.shape)}, expected [T, k]")
        T, k = ids.shape
        if out is None:
            out = blob.new_empty((T, L.rows), dtype=out_dtype or X.dtype)
        if T == 0:
            return out
        sizes = self._sizes.get((T, k))
        if sizes is None:
            P = mx.mx_experts_layout_init(T, k, L.groups)
            sizes = self._keep((T, k), (P, mx.mx_fp4_experts_workspace_size(L, P)))
        P, n = sizes
        mx.mx_fp4_experts(L, blob, P, ids, X, weights, out, blob.new_empty(n), gscale=self.act_scale,
                          status=self._status)
        return out

    __call__ = forward


def _microscaled_weights(L: mx.Fp4Layout, W: torch.Tensor, scale: torch.Tensor | None) -> torch.Tensor:
    blob = torch.empty(L.total_bytes, dtype=torch.uint8, device=W.device)
    if scale is None and L.format == mx.FP4_E4M3_16:
        scale = mx.mx_fp4_gscale(L, W)
    mx.mx_fp4_quant(L, W, blob, gscale=scale)
    return blob


def _reopen(blob: torch.Tensor) -> mx.Fp4Layout:
    if blob.dtype != torch.uint8:
        raise ValueError(f"blob has dtype {blob.dtype}, expected uint8")
    L = mx.mx_fp4_layout_from_header(blob[:mx.HEADER_BYTES].cpu())
    if blob.numel() < L.total_bytes:
        raise ValueError("blob shorter than its header says")
    return L
