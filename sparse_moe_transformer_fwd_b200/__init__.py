"""B200 (sm_100a) forward pass of one DeepSeek-V3/R1 Mixture-of-Experts FFN
layer: sigmoid-affinity router with a routing-only bias and top-k, per-expert
permutation, blockwise e4m3 quantisation, grouped SwiGLU expert GEMMs on the
tcgen05 tensor cores, and a weighted combine with the always-on shared
expert.  The work happens in libmoe_fwd.so (include/moe_fwd.h); this package
is its binding.

    layer = MoELayer(w_router, bias, w13, w2, top_k=8, precision="fp8")
    out = layer(x)          # x: bf16 [T, d_model] on the GPU
"""
from __future__ import annotations

import torch

from ._native import (EXPORTS, MOE_BF16, MOE_FP8_BLOCK, MOE_FP8_UE8M0, MOE_LAYOUT_ROWMAJOR, MOE_LAYOUT_TILED,
                      MoeError, moe_pack_tiles, moe_forward_prenorm, MoeShape, alloc_workspace,
                      fp8_block_quant, lib, make_shape, moe_check_status, moe_combine,
                      moe_forward, moe_grouped_swiglu, moe_last_error, moe_last_launch_count,
                      moe_last_launch_names,
                      moe_permute, moe_route, moe_route_noalloc, moe_set_kernel_events,
                      moe_workspace_size, MOE_ROUTE_NOALLOC_MAX_SCORES, MoeDenseShape,
                      make_dense_shape, moe_dense_workspace_size, alloc_dense_workspace,
                      moe_dense_ffn, moe_dense_ffn_prenorm, moe_workspace_layout,
                      moe_quant_scatter, moe_ep_dispatch, moe_ep_workspace_size,
                      moe_ep_grouped_swiglu, MOE_EP_MAX_RANKS, MoeLinearShape, make_linear_shape,
                      moe_linear_workspace_size, alloc_linear_workspace, fp8_block_gemm, moe_linear,
                      moe_linear_prenorm, MOE_FEW_MAX_TOKENS, moe_few_workspace_size,
                      alloc_few_workspace, moe_forward_few, moe_forward_few_prenorm, Workspaces, new_output)

__all__ = [
    "MoELayer", "MoeError", "MoeShape", "make_shape", "alloc_workspace", "lib", "EXPORTS",
    "moe_workspace_size", "moe_route", "moe_permute", "fp8_block_quant", "moe_grouped_swiglu",
    "moe_combine", "moe_forward", "moe_check_status", "moe_last_error", "moe_last_launch_count",
    "quantize_weights", "MOE_BF16", "MOE_FP8_BLOCK", "MOE_FP8_UE8M0", "moe_set_kernel_events",
    "moe_route_noalloc", "MOE_ROUTE_NOALLOC_MAX_SCORES", "moe_pack_tiles", "pack_weights",
    "MOE_LAYOUT_ROWMAJOR", "MOE_LAYOUT_TILED", "moe_forward_prenorm", "moe_last_launch_names",
    "DenseFFN", "MoeDenseShape", "make_dense_shape", "moe_dense_workspace_size",
    "alloc_dense_workspace", "moe_dense_ffn", "moe_dense_ffn_prenorm", "moe_workspace_layout",
    "moe_quant_scatter", "moe_ep_dispatch", "moe_ep_workspace_size", "moe_ep_grouped_swiglu",
    "MOE_EP_MAX_RANKS", "Fp8Linear", "MoeLinearShape", "make_linear_shape",
    "moe_linear_workspace_size", "alloc_linear_workspace", "fp8_block_gemm", "moe_linear",
    "moe_linear_prenorm", "MOE_FEW_MAX_TOKENS", "moe_few_workspace_size", "alloc_few_workspace",
    "moe_forward_few", "moe_forward_few_prenorm",
]


def quantize_weights(w13: torch.Tensor, w2: torch.Tensor, stream=None, ue8m0: bool = False,
                     layout=MOE_LAYOUT_TILED):
    """128x128 e4m3 block quantisation of the stacked expert weights (done
    once, ahead of the forward passes), codes in `layout` (tiled by default,
    or row-major); ue8m0: power-of-two scales.  Returns (w13q, w13s, w2q, w2s)."""
    S, n13, d = w13.shape
    _, d2, de = w2.shape
    w13q = torch.empty(S, n13, d, dtype=torch.uint8, device=w13.device)
    w13s = torch.empty(S, n13 // 128, d // 128, dtype=torch.float32, device=w13.device)
    w2q = torch.empty(S, d2, de, dtype=torch.uint8, device=w2.device)
    w2s = torch.empty(S, d2 // 128, de // 128, dtype=torch.float32, device=w2.device)
    fp8_block_quant(w13, 128, w13q, w13s, layout=layout, stream=stream, ue8m0=ue8m0)
    fp8_block_quant(w2, 128, w2q, w2s, layout=layout, stream=stream, ue8m0=ue8m0)
    return w13q, w13s, w2q, w2s


def pack_weights(w13: torch.Tensor, w2: torch.Tensor, stream=None):
    """bf16 expert weights repacked into the tiled layout the GEMMs read."""
    a, b = torch.empty_like(w13), torch.empty_like(w2)
    moe_pack_tiles(w13.contiguous(), a, stream=stream)
    moe_pack_tiles(w2.contiguous(), b, stream=stream)
    return a, b


def _tokens(t, cols: int, name: str) -> int:
    """T of an input [T, cols].  (The calls below take tensors that are longer
    than their shape; what an object is given says the shape itself.)"""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    T = t.shape[0] if t.dim() else -1
    if t.numel() != T * cols:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [T, {cols}]")
    return T


def _rows(t, T: int, cols: int, name: str) -> None:
    """Refuses a tensor (None passes) of other rows than [T, cols]; more rows may follow."""
    if t is not None and isinstance(t, torch.Tensor) and t.numel() != T * cols and (t.dim() < 2 or t.shape[-1] != cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{T}, {cols}]")


class MoELayer:
    """One MoE FFN layer with resident weights.

    w_router bf16 [E, d]; bias fp32 [E]; w13 bf16 [E + n_shared, 2*d_expert, d]
    (gate rows then up rows); w2 bf16 [E + n_shared, d, d_expert]; the shared
    expert, if any, is the last slot.  precision "fp8" (fp32 block scales) or
    "fp8_ue8m0" (power-of-two block scales) quantises the expert weights once
    at construction (the bf16 copies are then not needed); "bf16" repacks
    them.  weight_layout "tiled" (default: 128 x 128-byte tiles, one
    contiguous 16 KB read per TMA box) or "rowmajor" (the weights as given,
    e4m3 codes row-major).

    __call__ and forward_prenorm keep one workspace for each batch size: calls of
    one size do not overlap (a layer object, or moe_forward with a workspace, for
    each stream).  forward_few's calls may."""

    def __init__(self, w_router, bias, w13, w2, *, top_k: int, n_shared: int = 1,
                 routed_scale: float = 1.0, precision: str = "fp8", keep_bf16: bool = False,
                 weight_layout: str = "tiled"):
        lib()  # fail loudly now if the CUDA library is missing
        self.E, self.d = w_router.shape
        self.de = w2.shape[2]
        self.top_k, self.n_shared, self.routed_scale = top_k, n_shared, routed_scale
        self.precision = precision
        if weight_layout not in ("tiled", "rowmajor"):
            raise ValueError(weight_layout)
        self.weight_layout = weight_layout
        lay = MOE_LAYOUT_TILED if weight_layout == "tiled" else MOE_LAYOUT_ROWMAJOR
        self.w_router, self.bias = w_router.contiguous(), bias.contiguous()
        if precision in ("fp8", "fp8_ue8m0"):
            self.w13, self.w13s, self.w2, self.w2s = quantize_weights(
                w13.contiguous(), w2.contiguous(), ue8m0=precision == "fp8_ue8m0", layout=lay)
            self.w13_bf16 = w13 if keep_bf16 else None
            self.w2_bf16 = w2 if keep_bf16 else None
        elif precision == "bf16":
            self.w13, self.w2 = pack_weights(w13, w2) if lay == MOE_LAYOUT_TILED else \
                (w13.contiguous(), w2.contiguous())
            self.w13s = self.w2s = None
        else:
            raise ValueError(precision)
        self._ws, self._few_ws, self._few_shapes = {}, Workspaces(self.w13.device), {}

    def shape(self, T: int) -> MoeShape:
        return make_shape(T, self.d, self.E, self.top_k, self.de, self.n_shared,
                          self.routed_scale, self.precision, self.weight_layout)

    def workspace(self, T: int) -> torch.Tensor:
        ws = self._ws.get(T)
        if ws is None:
            ws = alloc_workspace(self.shape(T), self.w13.device)
            self._ws[T] = ws
        return ws

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None,
                 topk_idx_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        T = x.shape[0]
        if out is None:
            out = new_output(T, self.d, torch.bfloat16, x.device, stream)
        moe_forward(self.shape(T), x, self.w_router, self.bias, self.w13, self.w13s, self.w2,
                    self.w2s, out, self.workspace(T), topk_idx_out=topk_idx_out, stream=stream)
        return out

    def forward_prenorm(self, h: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                        out: torch.Tensor | None = None,
                        topk_idx_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The FFN block: out = h + MoE(RMSNorm(h) * gamma) (pre-norm fused)."""
        T = h.shape[0]
        if out is None:
            out = new_output(T, self.d, torch.bfloat16, h.device, stream)
        moe_forward_prenorm(self.shape(T), h, gamma, eps, self.w_router, self.bias, self.w13,
                            self.w13s, self.w2, self.w2s, out, self.workspace(T),
                            topk_idx_out=topk_idx_out, stream=stream)
        return out

    def few_workspace(self, T: int, stream=None) -> torch.Tensor:
        """The workspace that forward_few's calls of at most T tokens on `stream`
        take: streams have one each, captures theirs apart from eager calls'."""
        return self._few_ws.get(self._few_sized(T)[1], stream)

    def _few_sized(self, T: int):
        """The shape of T tokens and its workspace's bytes, worked out once."""
        sized = self._few_shapes.get(T)
        if sized is None:
            s = self.shape(T)
            sized = self._few_shapes[T] = s, moe_few_workspace_size(s)
        return sized

    def forward_few(self, x: torch.Tensor, out: torch.Tensor | None = None,
                    topk_idx_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The layer for at most MOE_FEW_MAX_TOKENS tokens, in one launch;
        routing as in __call__, out equal up to roundings.  Calls on several
        streams or from several threads may overlap; so may a graph's replay and
        eager calls, but not two graphs captured on one stream."""
        T = _tokens(x, self.d, "x")
        _rows(out, T, self.d, "out")
        _rows(topk_idx_out, T, self.top_k, "topk_idx_out")
        if out is None:
            out = new_output(T, self.d, torch.bfloat16, x.device, stream)
        shape, nbytes = self._few_sized(T)
        with self._few_ws.lock:
            moe_forward_few(shape, x, self.w_router, self.bias, self.w13, self.w13s, self.w2, self.w2s, out,
                            self._few_ws.get(nbytes, stream), topk_idx_out=topk_idx_out, stream=stream)
        return out

    def forward_few_prenorm(self, h: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                            out: torch.Tensor | None = None,
                            topk_idx_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """forward_prenorm for at most MOE_FEW_MAX_TOKENS tokens."""
        T = _tokens(h, self.d, "h")
        _rows(gamma, 1, self.d, "gamma")
        _rows(out, T, self.d, "out")
        _rows(topk_idx_out, T, self.top_k, "topk_idx_out")
        if out is None:
            out = new_output(T, self.d, torch.bfloat16, h.device, stream)
        shape, nbytes = self._few_sized(T)
        with self._few_ws.lock:
            moe_forward_few_prenorm(shape, h, gamma, eps, self.w_router, self.bias, self.w13, self.w13s, self.w2,
                                    self.w2s, out, self._few_ws.get(nbytes, stream), topk_idx_out=topk_idx_out,
                                    stream=stream)
        return out

    def check_status(self, T: int) -> int:
        """Status of __call__'s calls with T tokens and of all calls for few
        tokens so far: the first error that a workspace recorded."""
        few = self._few_ws.status()
        return moe_check_status(self.workspace(T)) or few


class DenseFFN:
    """One dense gated FFN layer (the model's first layers) with resident
    weights, on the expert GEMM kernels.

    w13 bf16 [2*d_ff, d] (gate rows then up rows); w2 bf16 [d, d_ff].
    precision and weight_layout as for MoELayer."""

    def __init__(self, w13, w2, *, precision: str = "fp8", weight_layout: str = "tiled"):
        lib()
        self.d, self.d_ff = w2.shape
        self.precision = precision
        if weight_layout not in ("tiled", "rowmajor"):
            raise ValueError(weight_layout)
        self.weight_layout = weight_layout
        lay = MOE_LAYOUT_TILED if weight_layout == "tiled" else MOE_LAYOUT_ROWMAJOR
        w13, w2 = w13.contiguous().unsqueeze(0), w2.contiguous().unsqueeze(0)
        if precision in ("fp8", "fp8_ue8m0"):
            self.w13, self.w13s, self.w2, self.w2s = quantize_weights(
                w13, w2, ue8m0=precision == "fp8_ue8m0", layout=lay)
        elif precision == "bf16":
            self.w13, self.w2 = pack_weights(w13, w2) if lay == MOE_LAYOUT_TILED else (w13, w2)
            self.w13s = self.w2s = None
        else:
            raise ValueError(precision)
        self._ws = {}

    def shape(self, T: int) -> MoeDenseShape:
        return make_dense_shape(T, self.d, self.d_ff, self.precision, self.weight_layout)

    def workspace(self, T: int) -> torch.Tensor:
        ws = self._ws.get(T)
        if ws is None:
            ws = alloc_dense_workspace(self.shape(T), self.w13.device)
            self._ws[T] = ws
        return ws

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None):
        T = x.shape[0]
        if out is None:
            out = new_output(T, self.d, torch.bfloat16, x.device, stream)
        moe_dense_ffn(self.shape(T), x, self.w13, self.w13s, self.w2, self.w2s, out,
                      self.workspace(T), stream=stream)
        return out

    def forward_prenorm(self, h: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                        out: torch.Tensor | None = None, stream=None):
        """The FFN block: out = h + FFN(RMSNorm(h) * gamma)."""
        T = h.shape[0]
        if out is None:
            out = new_output(T, self.d, torch.bfloat16, h.device, stream)
        moe_dense_ffn_prenorm(self.shape(T), h, gamma, eps, self.w13, self.w13s, self.w2,
                              self.w2s, out, self.workspace(T), stream=stream)
        return out

    def check_status(self, T: int) -> int:
        return moe_check_status(self.workspace(T))


class Fp8Linear:
    """One projection with resident block-scaled e4m3 weights: out = x W^T.

    w bf16 [N, K], K a multiple of 128, quantised once at construction in
    128x128 blocks; precision "fp8" (fp32 block scales) or "fp8_ue8m0"
    (power-of-two block scales).  weight_layout "tiled" (default where N is a
    multiple of 128) or "rowmajor" (any N).  x bf16 [T, K] is quantised 1x128
    on the way; out is bf16, or fp32 with out_dtype=torch.float32.

    Calls on several streams or from several threads may overlap (every stream
    has a workspace, of its largest call); so may a graph's replay and eager
    calls, but not two graphs captured on one stream, which share a workspace."""

    def __init__(self, w, *, precision: str = "fp8", weight_layout: str | None = None,
                 out_dtype: torch.dtype = torch.bfloat16):
        lib()
        if precision not in ("fp8", "fp8_ue8m0"):
            raise ValueError(precision)
        if weight_layout is None:
            weight_layout = "tiled" if w.shape[0] % 128 == 0 else "rowmajor"
        if weight_layout not in ("tiled", "rowmajor"):
            raise ValueError(weight_layout)
        self.N, self.K = w.shape
        self.precision, self.weight_layout, self.out_dtype = precision, weight_layout, out_dtype
        self.shape(1)  # refuses what the library would
        self.w = torch.empty(self.N, self.K, dtype=torch.uint8, device=w.device)
        self.w_scales = torch.empty(-(-self.N // 128), self.K // 128, dtype=torch.float32,
                                    device=w.device)
        with torch.cuda.device(w.device):
            fp8_block_quant(w.contiguous(), 128, self.w, self.w_scales,
                            layout=MOE_LAYOUT_TILED if weight_layout == "tiled" else MOE_LAYOUT_ROWMAJOR,
                            ue8m0=precision == "fp8_ue8m0")
        self._ws, self._shapes = Workspaces(w.device), {}

    def _sized(self, T: int):
        """The shape of T tokens and its workspace's bytes, worked out once."""
        key = T, self.out_dtype
        sized = self._shapes.get(key)
        if sized is None:
            s = self.shape(T)
            sized = self._shapes[key] = s, moe_linear_workspace_size(s)
        return sized

    def shape(self, T: int) -> MoeLinearShape:
        s = make_linear_shape(T, self.K, self.N, self.precision, self.weight_layout, self.out_dtype)
        moe_linear_workspace_size(s)
        return s

    def workspace(self, T: int, stream=None) -> torch.Tensor:
        """The workspace that calls of T tokens on `stream` take."""
        return self._ws.get(self._sized(T)[1], stream)

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None,
                 residual: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x W^T, plus the residual before the one rounding of a bf16 output."""
        T = _tokens(x, self.K, "x")
        _rows(out, T, self.N, "out")
        _rows(residual, T, self.N, "residual")
        if out is None:
            out = new_output(T, self.N, self.out_dtype, self.w.device, stream)
        shape, nbytes = self._sized(T)
        with self._ws.lock:
            moe_linear(shape, x, self.w, self.w_scales, out, self._ws.get(nbytes, stream), residual=residual,
                       stream=stream)
        return out

    def quantized(self, a: torch.Tensor, a_scales: torch.Tensor, out: torch.Tensor | None = None,
                  residual: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The product of codes that are quantised already (fp8_block_quant,
        block_rows 1): several projections of one x quantise it once."""
        T = _tokens(a, self.K, "a")
        _rows(a_scales, T, self.K // 128, "a_scales")
        _rows(out, T, self.N, "out")
        _rows(residual, T, self.N, "residual")
        if out is None:
            out = new_output(T, self.N, self.out_dtype, self.w.device, stream)
        shape, nbytes = self._sized(T)
        with self._ws.lock:
            fp8_block_gemm(shape, a, a_scales, self.w, self.w_scales, out, self._ws.get(nbytes, stream),
                           residual=residual, stream=stream)
        return out

    def forward_prenorm(self, h: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """bf16(RMSNorm(h) * gamma) W^T (pre-norm fused)."""
        T = _tokens(h, self.K, "h")
        _rows(gamma, 1, self.K, "gamma")
        _rows(out, T, self.N, "out")
        if out is None:
            out = new_output(T, self.N, self.out_dtype, self.w.device, stream)
        shape, nbytes = self._sized(T)
        with self._ws.lock:
            moe_linear_prenorm(shape, h, gamma, eps, self.w, self.w_scales, out, self._ws.get(nbytes, stream),
                               stream=stream)
        return out

    def check_status(self, T: int = 0) -> int:
        """Status of all calls so far: the first error that a workspace recorded."""
        return self._ws.status()
