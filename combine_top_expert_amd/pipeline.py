"""One GPU's MoE layer: device buffers plus the entry points in order.

torch provides device memory and the stream; every step of the layer runs
in libmoe_ep.so:

    moe_dispatch_layout -> moe_permute -> moe_grouped_gemm_w13 (fused SiLU*up)
      -> moe_grouped_gemm_w2 -> moe_combine

or, unfused, moe_grouped_gemm_w13 (G) -> moe_silu_mul -> moe_grouped_gemm_w2.
With 4-bit weights both products are moe_grouped_gemv_w4 (for decode steps);
token rows that are in block FP8 already go through moe_permute_fp8.  With
microscaled 4-bit weights ("mx4") the rows are quantised too: moe_permute_mx4
and moe_grouped_gemm_mx4, for any number of rows.  After a backward, step()
updates the weights (moe_adamw_step).
Buffers are sized from capacity bounds once, so a step never allocates and
its launch shapes never depend on the routing.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (MOE_EPI_SILU_MUL, MOE_EPI_STORE_G, moe_combine, moe_dispatch_layout,
               moe_dispatch_layout_workspace_bytes, moe_grouped_gemm_w2, moe_grouped_gemm_w13,
               moe_grouped_gemm_workspace_bytes, moe_pack_w13, MOE_W_PACKED, MOE_W_ROW_MAJOR,
               moe_combine_backward, moe_silu_mul_backward, moe_permute_backward,
               moe_transpose_weights, moe_grouped_gemm_wgrad, moe_grouped_gemm_w13_silu_backward,
               moe_permute, moe_silu_mul, MOE_W4_E2M1, MOE_W4_INT4, moe_grouped_gemv_w4, moe_pack_w4,
               moe_permute_fp8, moe_adamw_step, moe_grouped_gemm_mx4, moe_pack_mx4, moe_permute_mx4,
               moe_quantize_mx4)

_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}
_W4 = {"int4": MOE_W4_INT4, "fp4": MOE_W4_E2M1}


@dataclass(frozen=True)
class LayerShape:
    T: int
    K: int
    E: int              # global experts
    expert_begin: int
    L: int              # local experts
    H: int
    I: int
    R: int              # capacity per local expert, 0 = exact-fit
    act: str            # token activations: "f32" | "bf16"
    wdt: str            # expert weights: "f32" | "bf16" | "fp8" | "int4" | "fp4" (e2m1) | "mx4" (rows too)
    BM: int = 128
    x_fp8: bool = False  # token rows arrive in block FP8 (forward takes x_scales)

    def __post_init__(self):
        if self.x_fp8 and self.wdt in ("f32", "bf16"):
            raise ValueError("FP8 token rows need FP8 or 4-bit weights")
        if self.x_fp8 and self.wdt == "mx4":
            raise ValueError("MX4 weights take rows that are quantised to MX4 on dispatch, not FP8 rows")
        if self.wdt in _W4 and self.act == "f32" and not self.x_fp8:
            raise ValueError("4-bit weights take bf16 or FP8 rows")

    @property
    def rows_cap(self) -> int:
        return self.L * self.R if self.R > 0 else self.T * self.K

    @property
    def buf_dt(self) -> str:
        return "fp8" if self.wdt == "fp8" or self.x_fp8 else self.act

    @property
    def z_dt(self) -> str:
        return "fp8" if self.wdt == "fp8" else ("f32" if self.wdt == "f32" else "bf16")

    @property
    def out_dt(self) -> str:
        return "f32" if self.act == "f32" else "bf16"


class MoELayer:
    def __init__(self, shape: LayerShape, device="cuda", fused: bool = True):
        s = self.shape = shape
        self.fused = fused
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        rc = s.rows_cap
        mx4 = s.wdt == "mx4"
        if mx4 and not fused:
            raise ValueError("MX4 layers quantise Z in the gate/up product's epilogue: they are fused")
        self.counts = torch.zeros(s.L, **i32)
        self.offsets = torch.zeros(s.L + 1, **i32)
        self.slot_of = torch.zeros(s.T, s.K, **i32)
        self.row_src = torch.zeros(max(rc, 1), **i32)[:rc]
        self.tile_offsets = torch.zeros(s.L + 1, **i32)
        self.dev_status = torch.zeros(2, **i32)
        ws = moe_dispatch_layout_workspace_bytes(s.T, s.K, s.L)
        self.workspace = torch.zeros(max(ws, 4), dtype=torch.uint8, device=dev)
        # K-split partial sums of the GEMMs' last round (both GEMMs run on one
        # stream, one after the other, so they share it; the 4-bit products
        # have none)
        self.gemm_workspace = torch.empty(0 if s.wdt in _W4 or mx4 else moe_grouped_gemm_workspace_bytes(),
                                          dtype=torch.uint8, device=dev)
        if mx4:
            u8 = dict(dtype=torch.uint8, device=dev)
            self.buf, self.buf_scales = torch.empty(rc, s.H // 2, **u8), torch.empty(rc, s.H // 32, **u8)
            self.z, self.z_scales = torch.empty(rc, s.I // 2, **u8), torch.empty(rc, s.I // 32, **u8)
        else:
            self.buf = torch.empty(rc, s.H, dtype=_TORCH[s.buf_dt], device=dev)
            self.buf_scales = (torch.empty(rc, s.H // 128, dtype=torch.float32, device=dev)
                               if s.buf_dt == "fp8" else None)
            self.z = torch.empty(rc, s.I, dtype=_TORCH[s.z_dt], device=dev)
            self.z_scales = (torch.empty(rc, s.I // 128, dtype=torch.float32, device=dev)
                             if s.z_dt == "fp8" else None)
        self.g = None if fused else torch.empty(rc, 2 * s.I, dtype=torch.float32, device=dev)
        self.out = torch.empty(rc, s.H, dtype=_TORCH[s.out_dt], device=dev)
        self.y = torch.empty(s.T, s.H, dtype=_TORCH[s.out_dt], device=dev)
        self.w13 = self.w13_scales = self.w2 = self.w2_scales = self.w13_packed = None
        self.w4 = None                                       # packed 4-bit weights: (codes, scales) of W13 and W2
        self.adamw = None                                    # the optimizer's state (prepare_step)
        self._forget_weight_grads()

    def _forget_weight_grads(self):
        self.has_weight_grads = False                        # dw13 and dw2 hold gradients that no step has applied
        self._grads_made = False                             # some backward of these weights, run or captured, fills them
        self._captured_grads = None                          # whether the last captured backward does (None: there is none)

    def set_fused(self, fused: bool):
        """Switch the gate/up GEMM between the fused SiLU*up epilogue (the
        inference forward; a backward recomputes G) and the unfused pair
        (stores fp32 G, which the backward then reuses)."""
        s = self.shape
        if not fused and s.wdt == "mx4":
            raise ValueError("MX4 layers quantise Z in the gate/up product's epilogue: they are fused")
        if not fused and self.g is None:
            g = getattr(self, "g_saved", None)
            self.g = g if g is not None else torch.empty(s.rows_cap, 2 * s.I, dtype=torch.float32,
                                                         device=self.buf.device)
        if fused:
            self.g = None
        self.fused = fused

    def set_weights(self, w13, w2, w13_scales=None, w2_scales=None, pack_w13=True):
        """Device weights in the pages' layouts.  With pack_w13 (the default)
        the gate/up weights are also packed once into the GEMM's staging
        order (moe_pack_w13), which the gate/up GEMM then reads.

        4-bit layers: w13 [L,2I,H/2] and w2 [L,H,I/2] are codes (uint8, two a
        byte), the scales [L,2I,H/group] and [L,H,I/group] (fp32 or bf16);
        both are packed (moe_pack_w4), and only the packed copies are kept.
        New weights of the same sizes and dtypes are packed over the old copies,
        so bound and captured steps read them (on the current stream: steps on
        others have to be over, or wait for it); with another scale group or
        scale dtype such steps have to be bound and captured again, as with
        every other weight type.

        MX4 layers: likewise codes with scales [L,2I,H/32] and [L,H,I/32]
        (uint8, powers of two), or fp32 or bf16 weights [L,2I,H] and [L,H,I]
        without scales, which are quantised here (moe_quantize_mx4)."""
        wdt = self.shape.wdt
        if wdt in _W4 or wdt == "mx4":
            pairs = [(w13, w13_scales), (w2, w2_scales)]
            if wdt == "mx4" and w13_scales is None and w2_scales is None and w13.dtype != torch.uint8:
                pairs = [self._to_mx4(w) for w in (w13, w2)]
            elif w13_scales is None or w2_scales is None:
                raise ValueError("w13_scales and w2_scales are required for 4-bit weights")
            same = lambda o, t: o is not None and (o.shape, o.dtype, o.device) == (t.shape, t.dtype, t.device)  # noqa: E731
            old = self.w4 or [(None, None)] * 2
            held = [tuple(o if same(o, t) else torch.empty_like(t) for o, t in zip(*p)) for p in zip(old, pairs)]
            # Sizes and addresses are refused before anything is written.  Copies that steps may read are
            # written once neither is: W2 goes beside the old one until W13 has been taken.
            w2_new = tuple(torch.empty_like(h) if h is o else h for h, o in zip(held[1], old[1]))
            for (codes, scales), packed in ((pairs[1], w2_new), (pairs[0], held[0])):
                if wdt == "mx4":
                    moe_pack_mx4(codes, scales, *packed)
                else:
                    moe_pack_w4(codes, scales, _W4[wdt], *packed)
            for h, n in zip(held[1], w2_new):
                if h is not n:
                    h.copy_(n)
            self.w4 = held
            return
        packed = torch.empty_like(w13) if pack_w13 else None
        if pack_w13:
            moe_pack_w13(w13, packed)                        # refused: the layer stays as it was
        self.w13, self.w2, self.w13_scales, self.w2_scales, self.w13_packed = w13, w2, w13_scales, w2_scales, packed
        self._forget_weight_grads()                          # they were of the weights before

    @staticmethod
    def _to_mx4(w):
        """(codes, scales) of weights [L,N,K]."""
        u8 = dict(dtype=torch.uint8, device=w.device)
        L, N, K = w.shape
        codes, scales = torch.empty(L, N, K // 2, **u8), torch.empty(L, N, K // 32, **u8)
        moe_quantize_mx4(w, codes, scales)
        return codes, scales

    # ---- the six steps
    def layout(self, topk_ids):
        s = self.shape
        moe_dispatch_layout(topk_ids, s.E, s.expert_begin, s.L, s.R, s.BM, self.counts,
                            self.offsets, self.slot_of, self.row_src, self.tile_offsets,
                            self.dev_status, self.workspace)

    def permute(self, x, x_scales=None, bind=False):
        if self.shape.x_fp8:
            if x_scales is None:
                raise ValueError("x_scales is required for FP8 token rows")
            return moe_permute_fp8(x, x_scales, self.slot_of, self.buf, self.buf_scales, bind=bind)
        if x_scales is not None:
            raise ValueError("x_scales goes with FP8 token rows (LayerShape.x_fp8)")
        if self.shape.wdt == "mx4":
            return moe_permute_mx4(x, self.slot_of, self.buf, self.buf_scales, bind=bind)
        return moe_permute(x, self.slot_of, self.buf, self.buf_scales, bind=bind)

    def gemm_w13(self, bind=False):
        epi, out, scales = ((MOE_EPI_SILU_MUL, self.z, self.z_scales) if self.fused
                            else (MOE_EPI_STORE_G, self.g, None))
        if self.shape.wdt == "mx4":
            return moe_grouped_gemm_mx4(self.buf, self.buf_scales, *self.w4[0], self.counts, self.offsets, epi, out,
                                        out_scales=scales, bind=bind)
        if self.w4 is not None:
            return moe_grouped_gemv_w4(self.buf, self.buf_scales, *self.w4[0], _W4[self.shape.wdt], self.counts,
                                       self.offsets, epi, out, bind=bind)
        w, lay = ((self.w13_packed, MOE_W_PACKED) if self.w13_packed is not None
                  else (self.w13, MOE_W_ROW_MAJOR))
        return moe_grouped_gemm_w13(self.buf, self.buf_scales, w, self.w13_scales, self.counts, self.offsets, epi,
                                    out, scales, workspace=self.gemm_workspace, w13_layout=lay, bind=bind)

    def silu_mul(self):
        if not self.fused:
            moe_silu_mul(self.g, self.counts, self.offsets, self.z, self.z_scales)

    def gemm_w2(self, bind=False):
        if self.shape.wdt == "mx4":
            return moe_grouped_gemm_mx4(self.z, self.z_scales, *self.w4[1], self.counts, self.offsets, MOE_EPI_STORE_G,
                                        self.out, bind=bind)
        if self.w4 is not None:
            return moe_grouped_gemv_w4(self.z, self.z_scales, *self.w4[1], _W4[self.shape.wdt], self.counts,
                                       self.offsets, MOE_EPI_STORE_G, self.out, bind=bind)
        return moe_grouped_gemm_w2(self.z, self.z_scales, self.w2, self.w2_scales, self.counts,
                                   self.offsets, self.out, workspace=self.gemm_workspace, bind=bind)

    def combine(self, topk_weights):
        moe_combine(self.out, self.slot_of, topk_weights, self.y)

    # ---- backward (bf16 / fp32 layers)
    def prepare_backward(self):
        """Transposed weights and gradient buffers, made once (the weights are
        transposed again when set_weights installs new tensors; in-place
        updates need refresh_transposed_weights)."""
        s = self.shape
        if s.wdt not in ("f32", "bf16"):
            raise ValueError("the backward covers bf16 and fp32 layers")
        dev = self.buf.device
        gdt = self.out.dtype                       # gradients stored like the expert output
        src = getattr(self, "_wt_src", None)
        if src is None or src[0] is not self.w13 or src[1] is not self.w2:
            self.w2_t = torch.empty(s.L, s.I, s.H, dtype=self.w2.dtype, device=dev)
            self.w13_t = torch.empty(s.L, s.H, 2 * s.I, dtype=self.w13.dtype, device=dev)
            self._wt_src = (self.w13, self.w2)
            self.refresh_transposed_weights()
        rc = s.rows_cap
        if getattr(self, "d_out", None) is None:
            self.d_out = torch.empty(rc, s.H, dtype=gdt, device=dev)
            self.d_w = torch.empty(s.T, s.K, dtype=torch.float32, device=dev)
            self.dz = torch.empty(rc, s.I, dtype=gdt, device=dev)
            self.dg = torch.empty(rc, 2 * s.I, dtype=gdt, device=dev)
            self.da = torch.empty(rc, s.H, dtype=gdt, device=dev)
            self.dx = torch.empty(s.T, s.H, dtype=gdt, device=dev)
            self.dw2 = torch.empty(s.L, s.H, s.I, dtype=torch.float32, device=dev)
            self.dw13 = torch.empty(s.L, 2 * s.I, s.H, dtype=torch.float32, device=dev)

    def refresh_transposed_weights(self):
        """Rewrite W2^T and W13^T from the current weights.  prepare_backward
        does it when set_weights installs new weight tensors; a caller that
        updates the weights in place (an optimizer step) calls this before
        the next backward."""
        moe_transpose_weights(self.w2, self.w2_t)
        moe_transpose_weights(self.w13, self.w13_t)

    def backward_stages(self, dy, topk_weights, weight_grads=True, fuse_silu=True):
        """The backward as (name, launch) pairs in run order, for dy [T,H]:
        combine backward, dZ = d_out W2 (on W2^T), dG, dA = dG W13 (on
        W13^T), permute backward, then with weight_grads dW2 = d_out^T Z and
        dW13 = dG^T A per expert.  dG comes from G and dZ: after the unfused
        forward, which kept G, the SiLU*up backward reads it; after the fused
        forward the gate/up GEMM recomputes G with the SiLU*up gradient in its
        epilogue ("gemm_g_silu_bw"), or, with fuse_silu=False, stores fp32 G
        (g_saved) for a separate SiLU*up backward (the same values)."""
        self.prepare_backward()
        s = self.shape
        w, lay = ((self.w13_packed, MOE_W_PACKED) if self.w13_packed is not None
                  else (self.w13, MOE_W_ROW_MAJOR))
        st = [
            ("combine_bw", lambda: self._combine_bw(dy, topk_weights)),
            ("gemm_dz", lambda: moe_grouped_gemm_w2(self.d_out, None, self.w2_t, None, self.counts,
                                                    self.offsets, self.dz, workspace=self.gemm_workspace)),
        ]
        if self.g is None and fuse_silu:
            st.append(("gemm_g_silu_bw", lambda: moe_grouped_gemm_w13_silu_backward(
                self.buf, w, self.counts, self.offsets, self.dz, self.dg, workspace=self.gemm_workspace,
                w13_layout=lay)))
        else:
            if self.g is not None:
                self.g_saved = self.g                # kept by the unfused forward
            else:
                if getattr(self, "g_saved", None) is None:
                    self.g_saved = torch.empty(s.rows_cap, 2 * s.I, dtype=torch.float32,
                                               device=self.buf.device)
                st.append(("gemm_g", lambda: moe_grouped_gemm_w13(
                    self.buf, self.buf_scales, w, self.w13_scales, self.counts, self.offsets,
                    MOE_EPI_STORE_G, self.g_saved, workspace=self.gemm_workspace, w13_layout=lay)))
            st.append(("silu_mul_bw", lambda: moe_silu_mul_backward(self.g_saved, self.dz, self.counts,
                                                                    self.offsets, self.dg)))
        st += [
            ("gemm_da", lambda: moe_grouped_gemm_w2(self.dg, None, self.w13_t, None, self.counts,
                                                    self.offsets, self.da, workspace=self.gemm_workspace)),
            ("permute_bw", lambda: moe_permute_backward(self.da, self.slot_of, self.dx)),
        ]
        if weight_grads:
            st += [
                ("wgrad_w2", lambda: moe_grouped_gemm_wgrad(self.d_out, self.z, self.counts,
                                                            self.offsets, self.dw2)),
                ("wgrad_w13", self._wgrad_w13),
            ]
        return st

    def _capturing(self):
        with torch.cuda.device(self.buf.device):
            return torch.cuda.is_current_stream_capturing()

    def _combine_bw(self, dy, topk_weights):
        moe_combine_backward(dy, self.out, self.slot_of, topk_weights, self.d_out, self.d_w)
        if self._capturing():
            self._captured_grads = False
        else:
            self.has_weight_grads = False

    def _wgrad_w13(self):
        moe_grouped_gemm_wgrad(self.dg, self.buf, self.counts, self.offsets, self.dw13)
        self._grads_made = True
        if self._capturing():                                # nothing has run yet
            self._captured_grads = True
        else:
            self.has_weight_grads = True

    def backward(self, dy, topk_weights, weight_grads=True, fuse_silu=True):
        """Gradients of the last forward for dy [T,H]: returns (dx [T,H],
        d_w [T,K]); with weight_grads also fills dw2 [L,H,I] = d_out^T Z and
        dw13 [L,2I,H] = dG^T A per expert.  Reuses the forward's routing
        (slot_of, counts, offsets), its permuted activations, Z and expert
        outputs; G is the unfused forward's, else recomputed."""
        for _, f in self.backward_stages(dy, topk_weights, weight_grads, fuse_silu):
            f()
        return self.dx, self.d_w

    # ---- the optimizer's step (bf16 / fp32 layers)
    def prepare_step(self, state="f32", betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, seed=0):
        """AdamW's state for W13 and W2: moments in fp32 ("f32") or in 8 bits
        ("fp8"), zero, and for bf16 weights fp32 masters, made from the weights
        now.  New tensors in set_weights need it again; weights that were
        written in place need refresh_masters."""
        s = self.shape
        if s.wdt not in ("f32", "bf16"):
            raise ValueError("the optimizer's step covers bf16 and fp32 layers")
        if state not in ("f32", "fp8"):
            raise ValueError(f'state is {state!r}, expected "f32" or "fp8"')
        if self.w13 is None:
            raise ValueError("prepare_step needs weights (set_weights)")
        self.prepare_backward()
        w = [self.w13, self.w2]
        dt = torch.float32 if state == "f32" else torch.float8_e4m3fn
        zeros = lambda d, n: torch.zeros(n, dtype=torch.uint8, device=self.buf.device).view(d)  # noqa: E731
        moments = [[zeros(dt, t.numel() * dt.itemsize) for t in w] for _ in range(2)]
        scales = [[zeros(torch.float32, (t.numel() + 127) // 128 * 4) for t in w] if state == "fp8" else None
                  for _ in range(2)]
        masters = [t.float() for t in w] if s.wdt == "bf16" else None
        self.adamw = dict(weights=w, moments=moments, scales=scales, masters=masters, number=0,
                          hyper=dict(betas=betas, eps=eps, weight_decay=weight_decay, seed=seed))

    def refresh_masters(self):
        """The fp32 masters again from the weights, after those were written in place."""
        if self.adamw is not None and self.adamw["masters"] is not None:
            for m, w in zip(self.adamw["masters"], self.adamw["weights"]):
                m.copy_(w)

    def step(self, lr, number=None, grad_scale=None, reuse_grads=False):
        """One AdamW update of W13 and W2 (the tensors of set_weights), in place,
        from the dw13 and dw2 of the last backward, which has to have made them
        (weight_grads); the copies that the forward and the backward read
        (packed and transposed weights) are written again.  lr and number (of
        this update; counted here if not given) are numbers, or device tensors
        (fp32, int64) that a captured step reads anew; grad_scale: a device
        factor of the gradients (not finite: the weights and moments stay, and
        the count goes on).  Nothing waits.  After a device number the count is
        the caller's, until a step is given a number from the host; a captured
        step has to be given one either way.

        A backward's gradients are applied once.  reuse_grads takes dw13 and dw2
        as they are: again, the last ones that a backward made, or those of a
        captured backward that has been replayed (a captured step behind its
        captured backward needs no such word)."""
        o = self.adamw
        if o is None or o["weights"][0] is not self.w13 or o["weights"][1] is not self.w2:
            raise ValueError("step needs prepare_step after set_weights")
        capturing = self._capturing()
        fresh = self.has_weight_grads
        if capturing:
            fresh = self._grads_made if self._captured_grads is None else self._captured_grads
        if not (fresh or reuse_grads and self._grads_made):
            raise ValueError("step needs a backward with weight_grads whose gradients it has not applied yet "
                             "(reuse_grads takes those of a replayed graph, or the same again)")
        if number is None and o["number"] is None:
            raise ValueError("step needs the update's number: those before it were on the device")
        if number is None and capturing:
            raise ValueError("a captured step needs number: its replays would all be the update that is counted now")
        moe_adamw_step(o["weights"], [self.dw13, self.dw2], *o["moments"], lr, o["number"] + 1 if number is None else number,
                       masters=o["masters"], exp_avg_scales=o["scales"][0], exp_avg_sq_scales=o["scales"][1],
                       grad_scale=grad_scale, **o["hyper"])
        self.has_weight_grads = False                        # applied, or a graph's to apply
        if number is None:
            o["number"] += 1
        else:
            o["number"] = None if isinstance(number, torch.Tensor) else number
        if self.w13_packed is not None:
            moe_pack_w13(self.w13, self.w13_packed)
        self.refresh_transposed_weights()

    def bind_forward(self, x, topk_ids, topk_weights, x_scales=None):
        """The forward's launches as (name, callable) pairs, each marshalled
        once (shapes checked, pointers and the current stream looked up), so
        calling them runs the path with a few microseconds of host time per
        launch.  The tensors must stay alive and unchanged in shape, and the
        weights be those of the last set_weights (4-bit weights: or later ones
        of the same sizes)."""
        s = self.shape
        st = [
            ("layout", moe_dispatch_layout(topk_ids, s.E, s.expert_begin, s.L, s.R, s.BM, self.counts,
                                           self.offsets, self.slot_of, self.row_src, self.tile_offsets,
                                           self.dev_status, self.workspace, bind=True)),
            ("permute", self.permute(x, x_scales, bind=True)),
            ("gemm_w13", self.gemm_w13(bind=True)),
        ]
        if not self.fused:
            st.append(("silu_mul", moe_silu_mul(self.g, self.counts, self.offsets, self.z, self.z_scales,
                                                bind=True)))
        st += [
            ("gemm_w2", self.gemm_w2(bind=True)),
            ("combine", moe_combine(self.out, self.slot_of, topk_weights, self.y, bind=True)),
        ]
        return st

    def forward(self, x, topk_ids, topk_weights, x_scales=None):
        """The whole path on the current stream; returns y [T,H] (no sync).
        x: [T,H] activations, or with LayerShape.x_fp8 e4m3fn codes with
        x_scales [T,H/128] (as moe_add_rms_norm writes them)."""
        self.layout(topk_ids)
        self.permute(x, x_scales)
        self.gemm_w13()
        self.silu_mul()
        self.gemm_w2()
        self.combine(topk_weights)
        return self.y
