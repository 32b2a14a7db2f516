"""Local-Hessian NVFP4 block-scale calibration for B200 (sm_100a).

The work happens in liblh.so (C ABI in include/lh.h); this package is its
binding plus `calibrate`, which chains the four calls of the hot path for one
layer:

    lh_absmax -> lh_accumulate_hessian -> lh_sweep_scales_ws -> lh_fake_quant

`calibrate_routed` does so for an expert bank from the router's choices
(lh_route_tokens -> lh_gather_tokens first), and `QuantizedLayer` runs what was
calibrated (lh_quantize_nvfp4 and lh_nvfp4_tile_scales once, then
lh_nvfp4_linear, with lh_combine_tokens for a bank).

Method: "NVIDIA Model Optimizer Local-Hessian: 基于局部 Hessian 的 NVFP4 逐块
权重缩放算法实战指南" (xxmr.cn/news/266017), sections "算法原理" and
"入口 API 与校准流程".
"""
from __future__ import annotations

from ._binding import (  # noqa: F401
    EXPORTS, LH_BF16, LH_F32, LH_OK, LHError, lh_absmax, lh_accumulate_hessian, lh_fake_quant,
    lh_accumulate_hessian_noalloc, lh_noalloc_status, lh_debug_wait_timeout, lh_hessian_workspace_bytes, lh_last_error_message, lh_status_string,
    lh_quantize_nvfp4, lh_sweep_scales, lh_workspace_status, lh_baseline_scales, LH_SCALE_MAX,
    LH_SCALE_FOUR_OVER_SIX, LH_SCALE_MSE, lh_search_amax, lh_sweep_scales_ws, lh_sweep_workspace_bytes,
    lh_probe_fma, lh_probe_fma_flop,
    lh_route_tokens, lh_gather_tokens, lh_combine_tokens, lh_combine_tokens_grad, lh_quantize_tokens,
    lh_nvfp4_weight_scale_bytes, lh_nvfp4_token_scale_bytes, lh_nvfp4_tile_scales, lh_nvfp4_matmul, lh_nvfp4_status,
    lh_debug_nvfp4_wait_timeout,
    lh_nvfp4_linear_workspace_bytes, lh_nvfp4_linear,
)


class Calibrator:
    """Device buffers for calibrating one layer shape; `run` launches the
    whole hot path on the current stream, or on the one that it is given. Inputs are torch CUDA tensors:
    W [n_mats, c_out, c_in] (bf16 or f32), X [n_tok, c_in] bf16, optional
    offsets int64 [n_mats + 1] on the device (one token group per matrix)."""

    def __init__(self, n_mats: int, c_out: int, c_in: int, n_tok: int, grouped: bool, out_dtype=None,
                 device="cuda"):
        import torch
        self.n_mats, self.c_out, self.c_in, self.n_tok = n_mats, c_out, c_in, n_tok
        self.grouped = grouped
        if not grouped and n_mats > 1:
            raise ValueError("several matrices need grouped tokens (offsets, one group per matrix)")
        J = c_in // 16
        n_groups = n_mats if grouped else 1
        self.n_groups = n_groups
        self.out_dtype = out_dtype
        self.amax = torch.empty(n_mats, dtype=torch.float32, device=device)
        self.H = torch.zeros(n_groups, J, 16, 16, dtype=torch.float32, device=device)
        self.ws_bytes = lh_hessian_workspace_bytes(n_tok, c_in, n_groups)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=device)
        self.sweep_ws_bytes = lh_sweep_workspace_bytes(n_mats, c_in)
        self.sweep_ws = torch.empty(max(self.sweep_ws_bytes, 16), dtype=torch.uint8, device=device)
        self.best_amax = torch.empty(n_mats, c_out, J, dtype=torch.float32, device=device)
        self.best_code = torch.empty(n_mats, c_out, J, dtype=torch.uint8, device=device)
        self.Wq = None

    def run(self, W, X, offsets=None, stream=None, zero_h: bool = True):
        import torch
        n_mats, c_out, c_in = self.n_mats, self.c_out, self.c_in
        if X.dtype != torch.bfloat16:
            raise ValueError(f"X must be bf16, not {X.dtype}")
        if X.dim() != 2 or X.shape[1] != c_in:
            raise ValueError(f"X must be [n_tok, {c_in}], not {tuple(X.shape)}")
        if W.dim() not in (2, 3) or tuple(W.shape) != (n_mats, c_out, c_in)[3 - W.dim():] or W.numel() != n_mats * c_out * c_in:
            raise ValueError(f"W must be [{n_mats}, {c_out}, {c_in}], not {tuple(W.shape)}")
        if self.grouped:
            _typed("offsets", offsets, torch.int64, self.n_groups + 1)
        with _on(stream):
            W, X = _matrices(W), _rows(X, "X")
            if self.Wq is None or self.Wq.dtype != (self.out_dtype or W.dtype):
                self.Wq = torch.empty(n_mats, c_out, c_in, dtype=self.out_dtype or W.dtype, device=W.device)
            if zero_h:
                self.H.zero_()
            lh_absmax(W, W, n_mats, c_out, c_in, W.stride(-2), self.amax)
            lh_accumulate_hessian(X, LH_BF16, X.shape[0], c_in, X.stride(0), offsets if self.grouped else None,
                                  self.n_groups, self.H, self.ws, self.ws_bytes)
            lh_sweep_scales_ws(W, W, n_mats, c_out, c_in, W.stride(-2), self.amax, self.H, self.best_amax,
                               self.best_code, self.sweep_ws, self.sweep_ws_bytes)
            lh_fake_quant(W, W, n_mats, c_out, c_in, W.stride(-2), self.amax, self.best_code, self.Wq, self.Wq)
        return self.best_code, self.best_amax, self.Wq


def calibrate(W, X, offsets=None, out_dtype=None, stream=None):
    """One-shot Local-Hessian calibration of a layer (see Calibrator)."""
    if W.dim() == 2:
        W = W.unsqueeze(0)
    with _on(stream):
        cal = Calibrator(W.shape[0], W.shape[1], W.shape[2], X.shape[0], offsets is not None, out_dtype,
                         device=W.device)
        codes, amax, Wq = cal.run(W, X, offsets)
    return dict(codes=codes, best_amax=amax, Wq=Wq, H=cal.H, global_amax=cal.amax)


def _on_current_device(**tensors):
    """The library works on the current device; a tensor of another one would be read through the wrong context."""
    import torch
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.device.index != torch.cuda.current_device()):
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _typed(name, t, dtype, n):
    """The library is given addresses: t has to begin with n values of this type, one after another."""
    if t.dtype != dtype or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous values of {dtype}, not {tuple(t.shape)} of {t.dtype}")


def _no_gradient(**tensors):
    """The results are not part of autograd's graph: a gradient would be lost without a word."""
    import torch
    for name, t in tensors.items():
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient, which an NVFP4 layer does not give: call it under torch.no_grad()")


def _on(stream):
    """Makes `stream` (a torch stream, its handle, or None for the current one) current, so that what is allocated for
    its kernels is not handed out again before they are done. Its device becomes the current one: tensors are checked after."""
    import contextlib
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):  # 0 and 1 name the default stream; ExternalStream(0) would be a new one
        stream = torch.cuda.ExternalStream(stream) if stream > 1 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _rows(t, what):
    """t with 16-byte aligned rows, copied if it has none."""
    import torch
    per = 16 // t.element_size()
    if t.dim() != 2 or t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{what} must be a bf16 or f32 matrix")
    if t.stride(1) == 1 and t.stride(0) % per == 0 and t.stride(0) >= t.shape[1] and t.data_ptr() % 16 == 0:
        return t
    out = torch.empty(t.shape[0], -(-max(t.shape[1], 1) // per) * per, dtype=t.dtype, device=t.device)[:, :t.shape[1]]
    return out.copy_(t)


def _matrices(W):
    """W [n_mats, c_out, c_in] (or one matrix) as rows at one distance, matrix after matrix: copied if it does not lie so."""
    import torch
    if W.stride(-1) == 1 and W.stride(-2) >= W.shape[-1] and (W.dim() == 2 or W.shape[0] == 1 or
                                                              W.stride(0) == W.stride(1) * W.shape[1]):
        return W
    return W.clone(memory_format=torch.contiguous_format)  # contiguous() would keep any stride of a dimension of one


class Routing:
    """Tokens sorted by expert (lh_route_tokens): `offsets` int64 [n_experts + 1], `order` (flat slot t * k + s of each
    sorted row) and its inverse `pos`, int32 [n_tok * k]. expert_ids: int32 CUDA tensor [n_tok, k]; ids outside
    [0, n_experts) are slots without an expert. `route` may be called again with other ids of the same shape."""

    def __init__(self, n_tok: int, k: int, n_experts: int, device="cuda"):
        import torch
        self.n_tok, self.k, self.n_experts = n_tok, k, n_experts
        self.offsets = torch.empty(n_experts + 1, dtype=torch.int64, device=device)
        self.order = torch.empty(n_tok * k, dtype=torch.int32, device=device)
        self.pos = torch.empty(n_tok * k, dtype=torch.int32, device=device)

    def route(self, expert_ids, stream=None):
        import torch
        if expert_ids.dtype != torch.int32 or tuple(expert_ids.shape) != (self.n_tok, self.k):
            raise ValueError(f"expert_ids must be int32 [{self.n_tok}, {self.k}]")
        with _on(stream):
            _on_current_device(expert_ids=expert_ids, offsets=self.offsets)
            lh_route_tokens(expert_ids.contiguous(), self.n_tok, self.k, self.n_experts, self.offsets, self.order, self.pos)
        return self


def calibrate_routed(W, X, expert_ids, out_dtype=None, stream=None):
    """Local-Hessian calibration of an expert bank W [n_experts, c_out, c_in] from unsorted tokens X [n_tok, c_in]
    (bf16) and the experts that each was routed to (int32 [n_tok, k]): calibrate() on the sorted rows. Experts without
    tokens have H = 0 (every block gets code 1)."""
    import torch
    if X.dtype != torch.bfloat16:
        raise ValueError(f"X must be bf16, not {X.dtype}")
    n_tok, k = expert_ids.shape
    if X.shape[0] != n_tok or X.shape[1] != W.shape[2]:
        raise ValueError("X must be [n_tok, c_in]")
    with _on(stream):
        _on_current_device(W=W, X=X, expert_ids=expert_ids)
        X = _rows(X, "X")
        r = Routing(n_tok, k, W.shape[0], W.device).route(expert_ids)
        # rows of slots without an expert lie behind the last group and are never used
        rows = torch.empty(n_tok * k, W.shape[2], dtype=X.dtype, device=X.device)
        lh_gather_tokens(X, X, n_tok, X.shape[1], X.stride(0), r.order, k, n_tok * k, rows, rows.stride(0))
        return calibrate(W, rows, r.offsets, out_dtype)


class QuantizedLayer:
    """A calibrated layer in NVFP4, run with NVFP4 tokens (W4A4): Y = Xq Wq^T.

    W [n_mats, c_out, c_in] (or one matrix [c_out, c_in]), global_amax (f32 [n_mats]) and codes (uint8 [n_mats, c_out,
    c_in / 16]) as `calibrate` returns them; x_amax: the calibrated amax of the activations (f32 CUDA tensor [1]), or None
    for one scale per token. The packed weights and their scale tiles are made once; every call has a workspace of its own
    from torch's allocator, so calls on several streams and captured graphs do not share one. There is no backward pass:
    tokens or weights of the combination that require a gradient are refused outside torch.no_grad(). The products' waits
    are bounded: a GPU that stops answering for a second leaves results incomplete, which `check` reports."""

    def __init__(self, W, global_amax, codes, x_amax=None, stream=None):
        import torch
        if W.dim() == 2:
            W = W.unsqueeze(0)
        self.n_mats, self.c_out, self.c_in = W.shape
        if self.c_in % 32:
            raise ValueError(f"c_in={self.c_in} is not a multiple of 32")
        J = self.c_in // 16
        _typed("global_amax", global_amax, torch.float32, self.n_mats)
        if codes.dtype != torch.uint8 or codes.numel() != self.n_mats * self.c_out * J:
            raise ValueError(f"codes must be uint8 [{self.n_mats}, {self.c_out}, {J}], not {tuple(codes.shape)} of {codes.dtype}")
        if x_amax is not None:
            _typed("x_amax", x_amax, torch.float32, 1)
        with _on(stream):
            _on_current_device(W=W, global_amax=global_amax, codes=codes, x_amax=x_amax)
            codes = codes.reshape(self.n_mats, self.c_out, J).contiguous()
            W = _matrices(W)
            dev = W.device
            self.packed = torch.empty(self.n_mats, self.c_out, self.c_in // 2, dtype=torch.uint8, device=dev)
            self.block_scales = torch.empty_like(codes)
            self.global_scale = torch.empty(self.n_mats, dtype=torch.float32, device=dev)
            self.scale_tiles = torch.empty(lh_nvfp4_weight_scale_bytes(self.n_mats, self.c_out, self.c_in),
                                           dtype=torch.uint8, device=dev)
            lh_quantize_nvfp4(W, W, self.n_mats, self.c_out, self.c_in, W.stride(1), global_amax, codes, self.packed,
                              self.block_scales, self.global_scale)
            lh_nvfp4_tile_scales(self.block_scales, self.n_mats, self.c_out, self.c_in, self.scale_tiles)
        self.x_amax = x_amax

    @staticmethod
    def check(stream=None):
        """Waits for `stream` and raises LHError if a product on the current device, of any layer, has given up a wait
        since the last look: results since then may be incomplete."""
        from ._binding import _check
        _check(lh_nvfp4_status(stream), "lh_nvfp4_status")

    def _linear(self, X, rows, row_div, n_rows, offsets, out_dtype):
        import torch
        X = _rows(X, "X")
        if X.shape[1] != self.c_in:
            raise ValueError(f"X has {X.shape[1]} columns, the layer takes {self.c_in}")
        _on_current_device(X=X, packed=self.packed, rows=rows, offsets=offsets)
        out_dtype = out_dtype or X.dtype
        per = 8 if out_dtype == torch.bfloat16 else 4
        Y = torch.empty(n_rows, -(-self.c_out // per) * per, dtype=out_dtype, device=X.device)[:, :self.c_out]
        if n_rows == 0:
            return Y
        need = lh_nvfp4_linear_workspace_bytes(n_rows, self.c_in, self.n_mats)
        ws = torch.empty(need, dtype=torch.uint8, device=X.device)
        lh_nvfp4_linear(X, X, X.shape[0], self.c_in, X.stride(0), rows, row_div, n_rows, offsets, self.n_mats,
                        self.x_amax, self.packed, self.scale_tiles, self.global_scale, self.c_out, Y, Y, Y.stride(0), ws,
                        need)
        return Y

    def forward(self, X, offsets=None, out_dtype=None, stream=None):
        """Y [n_tok, c_out] of X [n_tok, c_in]; with several matrices the tokens of each are those of its group
        (offsets int64 [n_mats + 1] on the device); rows of tokens in no group are left unset."""
        import torch
        if (offsets is None) != (self.n_mats == 1):
            raise ValueError("several matrices need offsets, and one takes none")
        _no_gradient(X=X)
        if offsets is not None:
            _typed("offsets", offsets, torch.int64, self.n_mats + 1)
        with _on(stream):
            return self._linear(X, None, 1, X.shape[0], offsets, out_dtype)

    __call__ = forward

    def forward_routed(self, X, routing: Routing, weights=None, out_dtype=None, stream=None):
        """The bank's output for tokens X [n_tok, c_in]: sum over a token's experts of weights[t, s] (f32 [n_tok, k], or
        None for ones) times the expert's product. A token without any expert gets zeros."""
        import torch
        n_tok, k = routing.n_tok, routing.k
        if X.shape[0] != n_tok or routing.n_experts != self.n_mats:
            raise ValueError("the routing is for another number of tokens or experts")
        if weights is not None and (weights.dtype != torch.float32 or tuple(weights.shape) != (n_tok, k)):
            raise ValueError(f"weights must be f32 [{n_tok}, {k}]")
        _no_gradient(X=X, weights=weights)
        with _on(stream):
            _on_current_device(weights=weights, routing=routing.pos)
            rows = self._linear(X, routing.order, k, n_tok * k, routing.offsets, out_dtype)
            Y = torch.empty(n_tok, rows.stride(0), dtype=rows.dtype, device=X.device)[:, :self.c_out]
            if n_tok == 0:
                return Y
            weights = weights.contiguous() if weights is not None else None
            lh_combine_tokens(rows, rows, n_tok * k, self.c_out, rows.stride(0), routing.pos, weights, n_tok, k, Y,
                              Y.stride(0))
            return Y
