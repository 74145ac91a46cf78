"""Device buffers for one layer shape (torch supplies the memory; every step
of the layer runs in libmoe.so)."""
from __future__ import annotations

import torch

from . import _abi


class MoELayerBuffers:
    """Outputs, permutation arrays and workspace for a shape, on one device."""

    def __init__(self, T, H, E, I, top_k, act="bf16", wfmt="dense", device="cuda", tiled=False,
                 check_finite=False, fused=False):
        flags = ((_abi.MOE_F_TILED_WEIGHTS if tiled else 0) | (_abi.MOE_F_CHECK_FINITE if check_finite else 0)
                 | (_abi.MOE_F_FUSED_FFN if fused else 0))
        self.shape = _abi.make_shape(T, H, E, I, top_k, act, wfmt, flags)
        self.T, self.H, self.E, self.I, self.k = T, H, E, I, top_k
        self.act = act
        dt = torch.float32 if act == "f32" else torch.bfloat16
        P = T * top_k
        i32 = dict(dtype=torch.int32, device=device)
        self.topk_ids = torch.empty((T, top_k), **i32)
        self.topk_w = torch.empty((T, top_k), dtype=torch.float32, device=device)
        self.logits = torch.empty((T, E), dtype=torch.float32, device=device)
        self.counts = torch.empty(E, **i32)
        self.offsets = torch.empty(E + 1, **i32)
        self.sorted_pair = torch.empty(P, **i32)
        self.pair_row = torch.empty(P, **i32)
        self.active = torch.empty(E, **i32)
        self.n_active = torch.empty(1, **i32)
        self.y = torch.empty((P, H), dtype=dt, device=device)
        self.h = torch.empty((P, I), dtype=dt, device=device)
        self.out = torch.empty((T, H), dtype=dt, device=device)
        self.ws_bytes = _abi.moe_workspace_size(self.shape)
        self.workspace = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=device)
        self.perm = _abi.make_perm(self.counts, self.offsets, self.sorted_pair, self.pair_row,
                                   self.active, self.n_active)

    def route(self, x, w_router, bias=None, logits=True, stream=None):
        return _abi.moe_route(self.shape, x, w_router, bias, self.topk_ids, self.topk_w,
                              self.logits if logits else None, self.workspace, self.ws_bytes,
                              stream)

    def route_permute(self, x, w_router, bias=None, logits=True, stream=None):
        """moe_route_permute: routes into topk_ids / topk_w (and logits), the
        permutation into this buffer's perm, the tile plan into the workspace."""
        return _abi.moe_route_permute(self.shape, x, w_router, bias, self.topk_ids, self.topk_w,
                                      self.logits if logits else None, self.perm, self.workspace,
                                      self.ws_bytes, stream)

    def ffn_down_combine(self, experts, residual=None, out=None, h=None, stream=None):
        """moe_ffn_down_combine from this buffer's h into out (default self.out)."""
        return _abi.moe_ffn_down_combine(self.shape, self.h if h is None else h, experts, self.perm,
                                         self.topk_w, residual, self.out if out is None else out,
                                         self.workspace, self.ws_bytes, stream)

    def permute(self, topk_ids=None, stream=None):
        return _abi.moe_permute(self.shape, self.topk_ids if topk_ids is None else topk_ids,
                                self.perm, self.workspace, self.ws_bytes, stream)

    def ffn_fused(self, x, experts, wave_tiles=0, item_clock=None, perm=None, stream=None):
        """moe_ffn_fused into self.y (needs fused=True and tiled=True)."""
        return _abi.moe_ffn_fused(self.shape, x, experts, self.perm if perm is None else perm, self.y,
                                  wave_tiles, item_clock, self.workspace, self.ws_bytes, stream)

    def stage_experts(self, src, dst, parts=None, stream=None):
        """Copy the records of this call's active experts (the permutation
        already built by permute()) from `src` to `dst` (moe_experts structs;
        src may be pinned host memory); `parts` selects gate/up and/or down."""
        return _abi.moe_stage_experts(self.shape, src, dst, self.perm, parts, stream)

    def route_locality(self, topk_ids=None, stream=None):
        """(overlap_prev [T], [block_unique for B = 1..5]) as device tensors."""
        if not hasattr(self, "overlap_prev"):
            dev = self.topk_ids.device
            self.overlap_prev = torch.empty(self.T, dtype=torch.int32, device=dev)
            self.block_unique = torch.empty(max(_abi.moe_route_locality_blocks(self.T), 1),
                                            dtype=torch.int32, device=dev)
        _abi.moe_route_locality(self.shape, self.topk_ids if topk_ids is None else topk_ids,
                                self.overlap_prev, self.block_unique, stream)
        parts, o = [], 0
        for B in range(1, 6):
            nb = (self.T + B - 1) // B
            parts.append(self.block_unique[o:o + nb])
            o += nb
        return self.overlap_prev, parts

    def grouped_ffn(self, x, experts, perm=None, stream=None):
        return _abi.moe_grouped_ffn(self.shape, x, experts, self.perm if perm is None else perm,
                                    self.y, self.workspace, self.ws_bytes, stream)

    def ffn_gate_up(self, x, experts, perm=None, h=None, stream=None):
        return _abi.moe_ffn_gate_up(self.shape, x, experts, self.perm if perm is None else perm,
                                    self.h if h is None else h, self.workspace, self.ws_bytes,
                                    stream)

    def ffn_down(self, experts, h=None, y=None, stream=None):
        return _abi.moe_ffn_down(self.shape, self.h if h is None else h, experts,
                                 self.y if y is None else y, self.workspace, self.ws_bytes, stream)

    def combine(self, residual=None, y=None, pair_row=None, topk_w=None, out=None, stream=None):
        return _abi.moe_combine(self.shape, self.y if y is None else y,
                                self.pair_row if pair_row is None else pair_row,
                                self.topk_w if topk_w is None else topk_w, residual,
                                self.out if out is None else out, stream)

    def combine_norm(self, norm, w, gate=None, residual=None, w_next=None, z=None, out=None,
                     n_next=None, y=None, stream=None):
        """moe_combine_norm from this buffer's y, pair_row and topk_w into out
        (default self.out) and n_next (with w_next)."""
        return _abi.moe_combine_norm(self.shape, norm, self.y if y is None else y, self.pair_row,
                                     self.topk_w, w, gate, residual, w_next, z,
                                     self.out if out is None else out, n_next, stream)

    def block(self, x, norm_in, w_in, w_router, bias, experts, norm_out, w_out, gate=None,
              residual=None, w_next=None, n=None, out=None, n_next=None, stream=None, z=None):
        """One block around the routed experts: norm before, route, grouped
        FFN (moe_ffn_fused in a buffer made with fused), then combine, norm
        after, gate, residual and the next block's norm in one launch.  n
        [T][H] receives the normed rows, or holds them already (the previous
        block's n_next) when norm_in is None; z [T][H], if given, the branch
        before the norm after it, for moe_norm_out_backward.  A buffer with
        check_finite is refused (MOE_E_FLAGS): these steps do not check."""
        if self.shape.flags & _abi.MOE_F_CHECK_FINITE:
            raise _abi.MoEError(10, "MoELayerBuffers.block with check_finite")
        if norm_in is not None:
            _abi.moe_norm_in(norm_in, x, w_in, n, stream)
        self.route_permute(n, w_router, bias, logits=False, stream=stream)
        if self.shape.flags & _abi.MOE_F_FUSED_FFN:
            self.ffn_fused(n, experts, stream=stream)
        else:
            self.ffn_gate_up(n, experts, stream=stream)
            self.ffn_down(experts, stream=stream)
        return self.combine_norm(norm_out, w_out, gate, residual, w_next, z, out, n_next,
                                 stream=stream)

    def dispatch(self, x, rows, weighted=False, stream=None):
        """moe_dispatch of x into expert-ordered rows [T*k][H]; weighted: the
        route weights multiply the rows."""
        return _abi.moe_dispatch(self.shape, x, self.pair_row, self.topk_w if weighted else None,
                                 rows, stream)

    def dispatch_backward(self, drows, dx, dx_in=None, x=None, dw=None, weighted=False, stream=None):
        """moe_dispatch_backward; dw (with x) for weighted rows."""
        return _abi.moe_dispatch_backward(self.shape, drows, self.pair_row,
                                          self.topk_w if weighted else None, x, dx_in, dx, dw, stream)

    def combine_backward(self, dout, dy, dw=None, y=None, stream=None):
        """moe_combine_backward with this buffer's y, pair_row and topk_w."""
        return _abi.moe_combine_backward(self.shape, dout, self.y if y is None else y, self.pair_row,
                                         self.topk_w, dy, dw, stream)

    def route_backward(self, dw, dlogits, stream=None):
        """moe_route_backward of this buffer's topk_ids and topk_w."""
        return _abi.moe_route_backward(self.shape, self.topk_ids, self.topk_w, dw, dlogits, stream)

    def layer(self, x, w_router, bias, experts, residual=None, out=None, use_perm=True,
              stream=None):
        return _abi.moe_layer(self.shape, x, w_router, bias, experts, residual,
                              self.out if out is None else out, self.topk_ids, self.topk_w,
                              self.perm if use_perm else None, self.workspace, self.ws_bytes,
                              stream)
