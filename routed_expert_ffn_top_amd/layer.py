"""One MoE layer set up on the GPU through the C ABI.

Allocation (torch) and argument marshalling only: routing, descriptors, the
expert projections and the combine all run in the HIP library.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import binding as B
from .inputs import LayerInputs


class MoELayer:
    """Holds the device buffers of one layer: X, router weight, the slot
    arena with the experts, route descriptors and the workspace.

    phi      placement map for a resident layer (default: identity, P = E+S)
    paged    keep experts in pinned host memory, page them through an arena
             of cfg.P slots in banks of cfg.G (moe_layer_prefill's paged path)
    capacity route capacity C (default T*K': no split)
    """

    def __init__(self, inp: LayerInputs, phi: Optional[Sequence[int]] = None,
                 P: Optional[int] = None, capacity: Optional[int] = None,
                 paged: bool = False, device="cuda", stream=None):
        cfg = inp.cfg
        self.cfg = cfg
        self.device = torch.device(device)
        ne = cfg.n_exp
        if paged:
            P = cfg.slots if P is None else P
        elif phi is not None:
            P = (max(phi) + 1) if P is None else P
        else:
            P = ne if P is None else P
        self.shape = B.make_shape(cfg.T, cfg.d, cfg.f, cfg.E, cfg.k, cfg.n_shared, P=P,
                                  capacity=capacity, dtype=cfg.dtype, renorm=cfg.renorm)
        self.X = inp.X.to(self.device).contiguous()
        # router weight as [E][d] (one row per expert), the layout the C ABI takes
        self.Wr = inp.Wr.to(self.device).t().contiguous()
        self.bias = None if inp.bias is None else inp.bias.to(self.device).contiguous()
        self.routes = B.alloc_routes(self.shape, self.device)
        self.ws = B.alloc_workspace(self.shape, self.device)
        self._xq = None     # MXFP4 blocks of X (forward_mxfp4)
        self._decode = {}   # by token count: shape, routes, workspace
        self.paged = paged
        self.arena = B.Arena(self.shape, G=(cfg.G if paged else None), device=self.device)
        Wg = inp.Wg.to(self.device)
        Wu = inp.Wu.to(self.device)
        Wd = inp.Wd.to(self.device)
        scales = None
        if cfg.quant_weights:
            scales = tuple(t.to(self.device) for t in (inp.Sg, inp.Su, inp.Sd))
        if paged:
            # prepacked experts in two pinned host planes, expert after expert,
            # so that consecutive experts load with one transfer per plane
            gu_shape = tuple(self.arena.plane_gu.shape[1:])
            d_shape = tuple(self.arena.plane_d.shape[1:])
            self.host_gu_plane = torch.empty((ne,) + gu_shape, dtype=self.arena.plane_gu.dtype, pin_memory=True)
            self.host_d_plane = torch.empty((ne,) + d_shape, dtype=self.arena.plane_d.dtype, pin_memory=True)
            tmp = torch.empty(gu_shape, dtype=self.arena.plane_gu.dtype, device=self.device)
            tmp_d = torch.empty(d_shape, dtype=self.arena.plane_d.dtype, device=self.device)
            with B.on_stream(stream):   # a slice is copied out behind its packing
                for e in range(ne):
                    g, u, dn = B.expert_slices(Wg, Wu, Wd, scales, e)
                    B.moe_pack_gate_up(self.shape, g, u, tmp, 1, 0, 0)
                    B.moe_pack_down(self.shape, dn, tmp_d, 1, 0, 0)
                    self.host_gu_plane[e].copy_(tmp)
                    self.host_d_plane[e].copy_(tmp_d)
            self.host_gu = [self.host_gu_plane[e] for e in range(ne)]
            self.host_d = [self.host_d_plane[e] for e in range(ne)]
            self.phi = None
        else:
            self.phi = list(range(ne)) if phi is None else [int(x) for x in phi]
            self.arena.load_resident(Wg, Wu, Wd, self.phi, stream, scales=scales)
            self.host_gu = self.host_d = None
        torch.cuda.synchronize(self.device)

    def forward(self, Y: torch.Tensor, logits: Optional[torch.Tensor] = None,
                compute=None, copy=None) -> torch.Tensor:
        """Y holds the residual A on entry and the layer output on return
        (enqueued on `compute`; not synchronized)."""
        Wr = None if logits is not None else self.Wr
        bias = None if logits is not None else self.bias
        B.moe_layer_prefill(self.shape, self.X, Wr, bias, logits, Y, self.arena,
                            self.host_gu, self.host_d, self.routes, self.ws, compute, copy)
        return Y

    def forward_mxfp4(self, Y: torch.Tensor, logits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The resident layer with MXFP4 weights on MXFP4 activations: X is
        routed as it is, then quantised, and H is quantised between the
        projections. Y holds the residual on entry and the layer output on
        return. One call at a time, as with ``forward``: they share the workspace."""
        s, cfg = self.shape, self.cfg
        if not cfg.fp4_weights or self.paged or s.capacity < cfg.T * cfg.kp:
            raise ValueError("needs a resident layer with MXFP4 weights and capacity for every route")
        B.check_rows(Y, torch.float32, cfg.d, "Y")
        if logits is not None:
            B.check_rows(logits, torch.float32, cfg.E, "logits")
        for t, name in ((Y, "Y"), (logits, "logits")):
            if t is not None and (t.shape[0] != cfg.T or not t.is_contiguous()):
                raise ValueError(f"{name}: need {cfg.T} rows, contiguous")
        B.check_device((self.X, Y, logits), stream)
        if cfg.T == 0:
            return Y
        n = cfg.T * cfg.d
        if self._xq is None:
            self._xq = torch.empty(n // 2 + n // 32, dtype=torch.uint8, device=self.device)
            self._logits = torch.empty((cfg.T, cfg.E), dtype=torch.float32, device=self.device)
            torch.cuda.synchronize(self.device)   # whatever stream comes next, its memory's last use is over
        if logits is None:
            logits = self._logits
            B.moe_router_logits(s, self.X, self.Wr, self.bias, logits, stream)
        B.moe_quantize_mxfp4(self.X, self._xq[: n // 2], self._xq[n // 2:], stream)
        B.moe_route_build(s, 0, cfg.T, logits, self.phi, B.MOE_ROUTE_RESET, self.routes, self.ws, stream)
        B.moe_expert_ffn(s, self._xq, Y, self.routes, self.arena, self.phi,
                         B.MOE_FFN_EXPERTS | B.MOE_FFN_FINALIZE | B.MOE_FFN_ACT_MXFP4, self.ws, stream)
        return Y

    def decode(self, X: torch.Tensor, Y: torch.Tensor, logits: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """The layer on a few new tokens X [T][d] (rows may be strided), with
        the resident experts: Y [T][d] holds the residual on entry and the
        layer output on return. Route ids and weights are in
        ``decode_routes(T)``. One call at a time with a token count, graphs
        included: they share its workspace. It is made by the first call, which
        waits for the device and so cannot be a captured one, and is kept (64
        experts of 2048 x 1024, top-8: 7.4 MB for 64 tokens, 240 MB once every
        count up to 64 has been seen; ``moe_layer_decode`` itself takes any
        workspace that is large enough)."""
        B.check_rows(X, self.X.dtype, self.cfg.d, "X")
        B.check_rows(Y, torch.float32, self.cfg.d, "Y")
        if X.shape[0] != Y.shape[0] or (logits is not None and tuple(logits.shape) != (X.shape[0], self.cfg.E)):
            raise ValueError("X, Y and logits need as many rows")
        shape, routes, ws = self._decode_buffers(X.shape[0])
        shape.ldx, shape.ldy = B.row_stride(X), B.row_stride(Y)
        if logits is not None:
            B.check_rows(logits, torch.float32, self.cfg.E, "logits")
            if not logits.is_contiguous():   # a copy made here could be reused before another stream has read it
                raise ValueError("logits must be contiguous")
        B.moe_layer_decode(shape, X, None if logits is not None else self.Wr, None if logits is not None else self.bias,
                           logits, Y, self.arena, routes, ws, stream)
        return Y

    def decode_routes(self, T: int) -> dict:
        """topk_idx and topk_w [T][K'] of the last decode call with T tokens."""
        return self._decode_buffers(T)[1]

    def _decode_buffers(self, T: int):
        if T not in self._decode:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError(f"decode {T} tokens once, or ask for decode_routes({T}), before capturing it")
            c = self.cfg
            shape = B.make_shape(T, c.d, c.f, c.E, c.k, c.n_shared, P=self.shape.P, capacity=1, dtype=c.dtype,
                                 renorm=c.renorm)
            ws = B.alloc_decode_workspace(shape, self.device)
            routes = dict(topk_idx=torch.zeros((T, c.kp), dtype=torch.int32, device=self.device),
                          topk_w=torch.zeros((T, c.kp), dtype=torch.float32, device=self.device))
            torch.cuda.synchronize(self.device)   # cleared for whatever stream comes next
            self._decode[T] = (shape, routes, ws)
        return self._decode[T]

    def close(self):
        self.arena.close()
