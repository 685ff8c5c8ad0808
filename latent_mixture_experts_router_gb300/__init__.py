"""GB300 (sm_103a) latent mixture-of-experts block of Muse Spark Open.

    out = x + RMSNorm_post( F( RMSNorm_pre(x) ) )

F routes on the full-width normalised input (softmax over all experts, top-k,
renormalised weights), pools 8192 -> 4096 and normalises, runs the selected
SwiGLU experts, RMS-normalises each expert output with its own gamma before the
routing weight multiplies it, sums in FP32, and unpools 4096 -> 8192 (LMSYS
"SGLang and Miles Add Day-0 Support for Muse Spark Open", section "MoE with
pooler, unpooler and per-expert normalization"; vLLM "Day 0 support for Muse
Spark Open", sections "Sandwich normalization" and "Latent MoE").

The computation runs in the hand-written CUDA kernels of ``liblatent_moe.so``
behind the C ABI of ``include/latent_moe.h``; this package only marshals
arguments.  Importing it fails if the library has not been built.
"""
from __future__ import annotations

import contextlib

import torch

from ._lib import (Config, LmoeError, lmoe_workspace_size, lmoe_workspace_size_host_io,  # noqa: F401
                   lmoe_get_workspace_layout, latent_moe_forward, latent_moe_forward_ex,
                   latent_moe_forward_host_io, latent_moe_forward_host_io_ex, lmoe_check_status,
                   lmoe_wait_selftest, lmoe_expert_pair, load,
                   LIB_PATH, STAGES, NUM_STAGE_EVENTS, lmoe_kernel_launches, SINGLE_TOKEN_DEFAULT,
                   SINGLE_TOKEN_KERNEL, SINGLE_TOKEN_CHAIN,
                   lmoe_quantize_nvfp4, lmoe_nvfp4_block_scales, SCALES_ROW_MAJOR, SCALES_BLOCKED,
                   GUARD_BYTES, lmoe_workspace_guards, lmoe_validate_routing,
                   lmoe_permute_noalloc, lmoe_router_losses, lmoe_router_losses_workspace_size, lmoe_router_grad,
                   lmoe_quantize_fp8_rows, lmoe_quantize_fp8_weight, lmoe_quantize_fp8_cols,
                   lmoe_fp8_padded_rows, lmoe_matmul_fp8, lmoe_matmul_fp8_wgrad,
                   lmoe_fp8_check_status, lmoe_fp8_wait_selftest, _raw_stream)

load()


class LatentMoEBlock:
    """Device-resident weights of one block plus a reusable workspace.

    Weights: W_router [E, D]; W_pool [L, D]; W_gate, W_up [E, I, L]; W_down [E, L, I];
    W_unpool [D, L]; gammas g_pre [D], g_pool [L], g_expert [E, L], g_post [D] (fp32).
    NVFP4 weights are (codes, row-major E4M3 scales, tensor scale) triples; their scales are
    converted once into the block layout the kernels read.

    What a method allocates (its results, workspaces) belongs to the stream it is given, or the
    current one.  The forward calls of a block share its workspace, and the router methods read it:
    calls on several streams must be ordered by the caller.  A workspace that a captured call uses
    lives as long as the block, so graphs stay valid when a larger call replaces it.
    """

    def __init__(self, W_router, W_pool, g_pool, W_gate, W_up, W_down, g_expert, W_unpool, g_pre,
                 g_post, top_k: int, eps: float = 1e-6, weight_dtype: str = "bf16"):
        if weight_dtype == "nvfp4":   # (codes, row-major scales, s) -> scales in block layout
            def blocked(w, block_rows=128):
                codes, scales, s = w[:3]
                return codes, lmoe_nvfp4_block_scales(scales, codes.shape[-1] * 2, block_rows), s, SCALES_BLOCKED
            W_pool, W_gate, W_up, W_down, W_unpool = map(blocked, (W_pool, W_gate, W_up, W_down, W_unpool))
        self.W = dict(W_router=W_router, W_pool=W_pool, g_pool=g_pool, W_gate=W_gate, W_up=W_up,
                      W_down=W_down, g_expert=g_expert, W_unpool=W_unpool, g_pre=g_pre, g_post=g_post)
        self.top_k, self.eps, self.weight_dtype = top_k, eps, weight_dtype
        self.E, self.D = W_router.shape
        self.L = g_pool.shape[0]
        self.I = (W_gate[0] if isinstance(W_gate, tuple) else W_gate).shape[1]
        self._device = g_pre.device
        self._ws = None
        self._ran = None   # the configuration whose call left its routing in the workspace
        self._routed = None   # it, and the views of that routing
        self._loss_ws = self._loss_stream = None
        # the workspace's stream (handles), an event behind its zeroing (None: waited for), other streams that used it
        self._ws_stream = self._ws_zeroed = None
        self._ws_users = {}
        self._ws_captured, self._ws_of_graph, self._kept = False, False, []

    def config(self, T: int, act_dtype="bf16", out_dtype="f32") -> Config:
        return Config(T, self.D, self.L, self.E, self.I, self.top_k, self.eps, act_dtype,
                      self.weight_dtype, out_dtype)

    def _on(self, stream):
        """A context in which torch allocates on ``stream`` (a torch stream or a raw handle; None: the current)."""
        if stream is None:
            return contextlib.nullcontext()
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=self._device)
        return torch.cuda.stream(stream)

    def _current(self) -> int:
        """The current stream's handle."""
        return _raw_stream(self._device.index) if self._device.type == "cuda" else 0

    def _capturing(self) -> bool:
        return self._device.type == "cuda" and torch.cuda.is_current_stream_capturing()

    def _use_workspace(self, cur: int, capturing: bool):
        """The current stream ``cur`` is about to use the workspace."""
        if self._ws is None:
            return
        if capturing:
            self._ws_captured = True
            return
        if cur == self._ws_stream:
            return
        if self._ws_zeroed is not None:
            torch.cuda.current_stream(self._device).wait_event(self._ws_zeroed)
            self._ws_zeroed = None
        if cur not in self._ws_users:
            self._ws_users[cur] = torch.cuda.current_stream(self._device)

    def workspace(self, cfg: Config, host_io: bool = False, stream=None) -> torch.Tensor:
        n = lmoe_workspace_size_host_io(cfg) if host_io else lmoe_workspace_size(cfg)
        with self._on(stream):
            cur, capturing = self._current(), self._capturing()
            # (one allocated by a captured call is zeroed when its graph runs, and no other call's)
            if self._ws is None or self._ws.numel() < n or (self._ws_of_graph and not capturing):
                if self._ws is not None and (self._ws_captured or capturing):
                    self._kept.append(self._ws)
                else:
                    for s in self._ws_users.values():   # the old one is free once they are done with it
                        self._ws.record_stream(s)
                self._ws = torch.zeros(max(n, 256), dtype=torch.uint8, device=self._device)
                self._ran = self._routed = None
                self._ws_stream, self._ws_users = cur, {}
                self._ws_captured, self._ws_of_graph = False, capturing
                if not capturing and self._device.type == "cuda":
                    self._ws_zeroed = torch.cuda.current_stream(self._device).record_event()
                else:
                    self._ws_zeroed = None
            self._use_workspace(cur, capturing)
        return self._ws

    def forward(self, x: torch.Tensor, out_dtype="f32", out=None, stream=None, **ex) -> torch.Tensor:
        act = "f32" if x.dtype == torch.float32 else "bf16"
        cfg = self.config(x.shape[0], act, out_dtype)
        if out is None:
            with self._on(stream):
                out = torch.empty(x.shape, dtype=torch.float32 if out_dtype == "f32" else torch.bfloat16,
                                  device=x.device)
        ws = self.workspace(cfg, stream=stream)
        w = self.W
        fn = latent_moe_forward_ex if ex else latent_moe_forward
        self._ran = None
        fn(cfg, x, w["W_router"], w["W_pool"], w["g_pool"], w["W_gate"], w["W_up"], w["W_down"],
           w["g_expert"], w["W_unpool"], w["g_pre"], w["g_post"], self.top_k, out, ws, stream, **ex)
        self._ran = cfg
        return out

    def _routing(self, cfg: Config):
        """Views of the logits [T, E] and expert ids [T, k] that the last forward call, of ``cfg``, left."""
        # where they are depends on all of it but the types of x and out
        def shape(c):
            return c.T, c.d_model, c.d_latent, c.n_experts, c.d_ff, c.top_k, c.eps, c.weight_dtype
        if cfg.T > 0 and (self._ran is None or shape(cfg) != shape(self._ran)):
            raise ValueError("the last forward call was not one of this configuration")
        T, ld = cfg.T, (self.E + 31) // 32 * 32
        if T == 0:
            dev = self._device
            return (torch.empty(0, self.E, device=dev), torch.empty(0, self.top_k, dtype=torch.int32, device=dev))
        if self._routed is not None and self._routed[0] == shape(cfg):
            return self._routed[1:]
        lay = lmoe_get_workspace_layout(cfg)

        def view(name, n, dtype):
            return self._ws[lay[name]:lay[name] + 4 * n].view(dtype)
        self._routed = (shape(cfg), view("logits", T * ld, torch.float32).view(T, ld)[:, :self.E],
                        view("topk_idx", T * self.top_k, torch.int32).view(T, self.top_k))
        return self._routed[1:]

    def router_losses(self, cfg: Config, router_bias=None, row_mask=None, stream=None):
        """(losses [2], mean_probs [E], counts [E + 1]) of the last forward call, which had ``cfg``
        and ``router_bias``: the balance loss and the z loss, as lmoe_router_losses defines them.
        ``row_mask`` [T]: tokens that are 0 (padding) are left out."""
        logits, idx = self._routing(cfg)
        dev = logits.device
        with self._on(stream):
            cur, capturing = self._current(), self._capturing()
            self._use_workspace(cur, capturing)
            ws = self._loss_workspace(cfg.T, cur, capturing)
            losses, mean = torch.empty(2, device=dev), torch.empty(self.E, device=dev)
            counts = torch.empty(self.E + 1, dtype=torch.int32, device=dev)
        lmoe_router_losses(logits, idx, counts, mean, losses, ws, router_bias, row_mask, stream)
        return losses, mean, counts

    def _loss_workspace(self, T: int, cur: int, capturing: bool):
        """Workspace of the losses of T tokens: one that is kept, for any T, on the stream that first asked; another
        stream's, and a captured call's (in its graph's memory), is its own, so that none of them overlap."""
        if not capturing:
            if self._loss_ws is None:
                n = lmoe_router_losses_workspace_size(1 << 20, self.E)
                self._loss_ws, self._loss_stream = torch.empty(n, dtype=torch.uint8, device=self._device), cur
            if cur == self._loss_stream:
                return self._loss_ws
        return torch.empty(lmoe_router_losses_workspace_size(T, self.E), dtype=torch.uint8, device=self._device)

    def router_grad(self, cfg: Config, topk_w_grad=None, loss_grads=None, counts=None, router_bias=None,
                    row_mask=None, out=None, stream=None):
        """Gradient [T, E] fp32 of the last forward call's router logits from that of its routing
        weights ``topk_w_grad`` [T, k] and of router_losses' two losses, ``loss_grads`` [2] (with
        its ``counts``).  Summed over the tokens it is router_bias' gradient."""
        logits, idx = self._routing(cfg)
        with self._on(stream):
            self._use_workspace(self._current(), self._capturing())
            if out is None:
                out = torch.empty(logits.shape, device=logits.device)
        lmoe_router_grad(logits, idx, counts, out, topk_w_grad, loss_grads, router_bias, row_mask, stream)
        return out
