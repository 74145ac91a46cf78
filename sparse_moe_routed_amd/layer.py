"""Device buffers for one layer shape (torch supplies the memory; every step
of the layer runs in libmoe.so)."""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _abi


def _made_on(stream):
    """Memory that a call makes belongs to the stream that the call uses: taken
    from the pool of another one it could be memory whose last use there is
    still to come."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


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
            with _made_on(stream):
                made = [torch.empty(n, dtype=torch.int32, device=self.topk_ids.device)
                        for n in (self.T, max(_abi.moe_route_locality_blocks(self.T), 1))]
            self.overlap_prev, self.block_unique = made
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

    def _products(self, where, saved=False):
        """Refuses, before the first step of `where`, a shape that the training's
        products refuse (tiled or low-bit weights, sizes past their limits) and,
        with `saved`, a gradient without anything saved."""
        if not hasattr(self, "_products_status"):
            # without pointers: what is wrong with the shape, else MOE_E_NULL (or nothing to do)
            st = _abi.load().moe_ffn_gate_up_save(ctypes.byref(self.shape), *[None] * 6, 0, None)
            self._products_status = 0 if st == 1 else st
        if self._products_status:
            raise _abi.MoEError(self._products_status, f"MoELayerBuffers.{where}")
        if saved and not hasattr(self, "saved"):
            raise _abi.MoEError(1, f"MoELayerBuffers.{where} before ffn_gate_up_save or layer_save")

    def _train(self, kept=None, stream=None):
        """Memory for training, made once and kept as long as the buffer (work
        that is queued or captured in a graph may hold its addresses): the
        workspace, and a set of g and u for each form that was asked for ('act',
        or '8bit' with their scales), which is returned.  Nothing is kept of a
        set whose memory is not all there."""
        if kept not in (None, "act", "8bit"):
            raise ValueError(f"kept must be 'act' or '8bit', not {kept!r}")
        dev = self.topk_ids.device
        if not hasattr(self, "train_ws"):
            n = _abi.moe_train_workspace_size(self.shape)
            with _made_on(stream):
                self.train_ws, self.train_ws_bytes = torch.empty(max(n, 1), dtype=torch.uint8, device=dev), n
            self._kept_sets = {}
        if kept is None:
            return None
        if kept not in self._kept_sets:
            P, q8 = self.T * self.k, kept == "8bit"
            dt = torch.int8 if q8 else self.y.dtype
            with _made_on(stream):
                g, u = (torch.empty((P, self.I), dtype=dt, device=dev) for _ in range(2))
                gs, us = (torch.empty((P, self.I // 32), dtype=torch.uint8, device=dev) if q8 else None
                          for _ in range(2))
            self._kept_sets[kept] = (g, u, gs, us, _abi.make_saved(g, u, gs, us))
        return self._kept_sets[kept]

    def ffn_gate_up_save(self, x, experts, kept="act", perm=None, h=None, stream=None):
        """moe_ffn_gate_up_save into this buffer's h and saved (g and u, kept in
        the activation type or in 8 bits).  Each form has memory of its own,
        which stays; ffn_backward reads that of the last call of this method
        (the replay of a graph is none)."""
        self._products("ffn_gate_up_save")
        kept_set = self._train(kept, stream)
        st = _abi.moe_ffn_gate_up_save(self.shape, x, experts, self.perm if perm is None else perm,
                                       kept_set[4], self.h if h is None else h, self.train_ws,
                                       self.train_ws_bytes, stream)
        self.kept = kept
        self.g, self.u, self.g_scale, self.u_scale, self.saved = kept_set
        return st

    def ffn_backward(self, dy, x, experts, drows=None, dexperts=None, x_scale=None, perm=None,
                     stream=None):
        """moe_ffn_backward from this buffer's saved."""
        self._products("ffn_backward", saved=True)
        self._train(stream=stream)
        return _abi.moe_ffn_backward(self.shape, dy, x, x_scale, self.saved, experts,
                                     self.perm if perm is None else perm, drows, dexperts,
                                     self.train_ws, self.train_ws_bytes, stream)

    def router_backward(self, dw, x, w_router, dx=None, dw_router=None, dbias=None, dx_in=None,
                        stream=None):
        """moe_router_backward of this buffer's topk_ids, topk_w and perm."""
        self._train(stream=stream)
        return _abi.moe_router_backward(self.shape, self.topk_ids, self.topk_w, dw, x, w_router,
                                        self.perm, dx_in, dx, dw_router, dbias, self.train_ws,
                                        self.train_ws_bytes, stream)

    def layer_save(self, x, w_router, bias, experts, residual=None, out=None, kept="act", stream=None):
        """The whole layer, keeping in this buffer what layer_backward needs (the
        routes, the permutation, y, g and u).  experts are dense and row-major,
        and no pair is dropped.  A buffer made tiled, fused or with check_finite
        (these steps do not check) is refused (MOE_E_FLAGS), and one of low-bit
        weights (MOE_E_FORMAT)."""
        if self.shape.flags & _abi.MOE_F_CHECK_FINITE:
            raise _abi.MoEError(10, "MoELayerBuffers.layer_save with check_finite")
        self._products("layer_save")
        self._train(kept, stream)
        self.route_permute(x, w_router, bias, logits=False, stream=stream)
        self.ffn_gate_up_save(x, experts, kept, stream=stream)
        self.ffn_down(experts, stream=stream)
        return self.combine(residual, out=out, stream=stream)

    def layer_backward(self, dout, x, w_router, experts, dx, dw_router=None, dbias=None,
                       dexperts=None, dx_in=None, x_scale=None, stream=None):
        """Gradient of layer_save for the gradient dout of its output: dx [T][H]
        (plus dx_in, for instance dout where the residual was x), dw_router,
        dbias and dexperts (a moe_experts of the weights' gradients), each of
        the last three only if given.  x may be its 8-bit checkpoint
        (x_scale).  dx is rounded to the activation type twice: what comes
        through the experts with dx_in, and that with what comes through the
        router."""
        self._products("layer_backward", saved=True)
        self._train(stream=stream)
        if not hasattr(self, "dy"):
            with _made_on(stream):
                made = [torch.empty_like(t) for t in (self.y, self.y, self.topk_w, self.out)]
            self.dy, self.drows, self.dw, self.dx_rows = made
        if x_scale is not None:
            if not hasattr(self, "x_back"):
                with _made_on(stream):
                    self.x_back = torch.empty_like(self.out)
            _abi.moe_restore8(self.act, self.T, self.H, x, x_scale, self.x_back, stream)
            x = self.x_back
        self.combine_backward(dout, self.dy, self.dw, stream=stream)
        self.ffn_backward(self.dy, x, experts, self.drows, dexperts, stream=stream)
        self.dispatch_backward(self.drows, self.dx_rows, dx_in, stream=stream)
        return self.router_backward(self.dw, x, w_router, dx, dw_router, dbias, self.dx_rows,
                                    stream=stream)

    def layer(self, x, w_router, bias, experts, residual=None, out=None, use_perm=True,
              stream=None):
        return _abi.moe_layer(self.shape, x, w_router, bias, experts, residual,
                              self.out if out is None else out, self.topk_ids, self.topk_w,
                              self.perm if use_perm else None, self.workspace, self.ws_bytes,
                              stream)
