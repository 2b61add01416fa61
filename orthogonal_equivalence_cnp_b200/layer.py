"""Device buffers of one POET-X layer and the call sequence of one training step.

Plumbing only: torch provides device memory and the stream; every step of the layer runs in
libpoetx's kernels through the C ABI (see the package __init__).
"""
from __future__ import annotations

import numpy as np
import torch

from . import (POETX_BF16, POETX_F32, POETX_FAST, POETX_MEM, poetx_absorb, poetx_adamw_cfg, poetx_adamw_reset,
               poetx_adamw_step, poetx_backward, poetx_cnp, poetx_cnp_forward, poetx_desc, poetx_fourperm_backward,
               poetx_fourperm_forward, poetx_fourperm_workspace_size, poetx_forward,
               poetx_merge, poetx_mx4_backward, poetx_mx4_forward, poetx_mx4_merge, poetx_mx4_quantize,
               poetx_wc_backward, poetx_wc_forward, poetx_wc_saved_size, poetx_wc_workspace_size,
               poetx_workspace_size, poetx_xq_backward, poetx_xq_forward, poetx_xq_merge, poetx_xq_quantize)
from .optim import MultiAdamW

TORCH_DTYPE = {POETX_F32: torch.float32, POETX_BF16: torch.bfloat16}


def make_desc(d_in: int, d_out: int, b: int, k: int, dtype: str, mode: str) -> poetx_desc:
    return poetx_desc(d_in, d_out, b, k, POETX_BF16 if dtype == "bf16" else POETX_F32,
                      POETX_MEM if mode == "mem" else POETX_FAST)


class PoetxLayer:
    """Holds W0', theta, permutations, Q and scratch of one layer on one device.  moments: the AdamW moments that
    optimizer_step and train_step use, "f32" (m and v), "e4m3" (8 bits each, in `optimizer`), or None where theta is
    stepped from outside, by a MultiAdamW over several layers.  workspace: scratch to use instead of the layer's own, a
    uint8 tensor of at least workspace_bytes(desc, n_tokens); layers that run one after another on one stream
    may share one (its merge part alone is two bf16 weights)."""

    def __init__(self, desc: poetx_desc, n_tokens: int, device="cuda", moments="f32", workspace=None):
        if moments not in ("f32", "e4m3", None):
            raise ValueError(f"moments: 'f32', 'e4m3' or None, got {moments!r}")
        self.desc = desc
        self.n = int(n_tokens)
        self.device = torch.device(device)
        dt = TORCH_DTYPE[desc.dtype]
        self.dtype = dt
        b, din, dout = desc.b, desc.d_in, desc.d_out
        P = b * (b - 1) // 2
        dev = self.device
        self.W0p = torch.empty(dout, din, dtype=dt, device=dev)
        # POET-XQ (after quantize()): W0' as int8 codes W0q [d_out, d_in] and scales W0s [d_out]; MX4
        # (after quantize("mx4")): 4-bit codes W0q uint8 [d_out, d_in / 2], scales W0s uint8 [d_out, d_in / 32].
        self.xq = self.mx4 = False
        self.W0q = self.W0s = None
        self.W0 = None  # the un-absorbed weight (load_state), for the four-permutation comparator
        # theta_R and theta_P (and their gradients and AdamW moments) are stored back to back so
        # that one optimiser launch covers both sides.
        nbo, nbi = dout // b, din // b
        self.theta = torch.zeros(nbo + nbi, P, dtype=torch.float32, device=dev)
        self.theta_R, self.theta_P = self.theta[:nbo], self.theta[nbo:]
        self.perm_L = torch.arange(dout, dtype=torch.int32, device=dev)
        self.perm_R = torch.arange(din, dtype=torch.int32, device=dev)
        self.Q_R = torch.empty(dout // b, b, b, dtype=dt, device=dev)
        self.Q_P = torch.empty(din // b, b, b, dtype=dt, device=dev)
        self.Y = torch.empty(self.n, dout, dtype=dt, device=dev)
        # POET-Xfast keeps Z [N, d_out] and U = X[:, pi_R] [N, d_in] for the backward pass.
        self.saved = torch.empty(self.n * (dout + din), dtype=dt, device=dev) if desc.mode == POETX_FAST else None
        self.dX = torch.empty(self.n, din, dtype=dt, device=dev)
        self.grad = torch.zeros_like(self.theta)
        self.g_R, self.g_P = self.grad[:nbo], self.grad[nbo:]
        self.m = self.v = self.optimizer = None
        if moments == "f32":
            self.m, self.v = torch.zeros_like(self.theta), torch.zeros_like(self.theta)
        elif moments == "e4m3":
            self.optimizer = MultiAdamW.from_params([self.theta], [self.grad])
        self.t = 0       # AdamW step count of the current moments
        self.steps = 0   # training steps taken (drives the merge schedule)
        ws = self.workspace_bytes(desc, self.n)
        self.ws = torch.empty(ws, dtype=torch.uint8, device=dev) if workspace is None else workspace
        if self.ws.dtype != torch.uint8 or not self.ws.is_contiguous() or self.ws.numel() < ws:
            raise ValueError(f"workspace: a contiguous uint8 tensor of at least {ws} bytes")
        if self.ws.device != self.theta.device:
            raise ValueError(f"workspace is on {self.ws.device}, the layer on {self.theta.device}")

    @staticmethod
    def workspace_bytes(desc: poetx_desc, n_tokens: int) -> int:
        return max(poetx_workspace_size(desc, n_tokens), 256)

    # ------------------------------------------------------------------ state upload helpers
    def to_dev(self, a: np.ndarray, dtype=None) -> torch.Tensor:
        t = torch.from_numpy(np.ascontiguousarray(a))
        return t.to(device=self.device, dtype=dtype or self.dtype)

    def load_state(self, W0: np.ndarray, theta_R, theta_P, pi_L, pi_R):
        """Uploads the original-basis W0 and absorbs the two permutations on the device."""
        if self.W0p is None:
            raise ValueError("the layer's weight is quantised; load the state into a new layer")
        self.perm_L.copy_(torch.from_numpy(np.asarray(pi_L, np.int32)))
        self.perm_R.copy_(torch.from_numpy(np.asarray(pi_R, np.int32)))
        self.theta_R.copy_(torch.from_numpy(np.asarray(theta_R, np.float32)))
        self.theta_P.copy_(torch.from_numpy(np.asarray(theta_P, np.float32)))
        W0_dev = self.to_dev(W0)
        poetx_absorb(self.desc, W0_dev, self.perm_L, self.perm_R, self.W0p)
        self.W0 = W0_dev

    # ------------------------------------------------------------------------- the step
    def cnp(self):
        poetx_cnp(self.desc, self.theta_R, self.theta_P, self.Q_R, self.Q_P, self.ws)

    def forward(self, X: torch.Tensor):
        if self.xq:
            poetx_xq_forward(self.desc, self.n, X, self.W0q, self.W0s, self.perm_L, self.perm_R, self.Q_R, self.Q_P,
                             self.Y, self.ws)
        elif self.mx4:
            poetx_mx4_forward(self.desc, self.n, X, self.W0q, self.W0s, self.perm_L, self.perm_R, self.Q_R, self.Q_P,
                              self.Y, self.ws)
        else:
            poetx_forward(self.desc, self.n, X, self.W0p, self.perm_L, self.perm_R, self.Q_R, self.Q_P, self.Y,
                          self.saved, self.ws)
        return self.Y

    def backward(self, dY: torch.Tensor, X: torch.Tensor):
        if self.xq:
            poetx_xq_backward(self.desc, self.n, dY, X, self.W0q, self.W0s, self.perm_L, self.perm_R, self.Q_R,
                              self.Q_P, self.theta_R, self.theta_P, self.dX, self.g_R, self.g_P, self.ws)
        elif self.mx4:
            poetx_mx4_backward(self.desc, self.n, dY, X, self.W0q, self.W0s, self.perm_L, self.perm_R, self.Q_R,
                               self.Q_P, self.theta_R, self.theta_P, self.dX, self.g_R, self.g_P, self.ws)
        else:
            poetx_backward(self.desc, self.n, dY, X, self.W0p, self.perm_L, self.perm_R, self.Q_R, self.Q_P,
                           self.theta_R, self.theta_P, self.saved, self.dX, self.g_R, self.g_P, self.ws)
        return self.dX, self.g_R, self.g_P

    def quantize(self, bits: str = "int8"):
        """Switches the layer (mem mode, bf16) to a quantised W0' and releases the bf16 one and the
        un-absorbed W0 (the four-permutation comparator ends with it): "int8" (POET-XQ, one scale per row)
        or "mx4" (4 bits, one scale per 32 columns)."""
        if bits not in ("int8", "mx4"):
            raise ValueError(f"bits: 'int8' or 'mx4', got {bits!r}")
        if self.xq or self.mx4:
            raise ValueError("the layer's weight is quantised already")
        d = self.desc
        if bits == "mx4":
            if d.dtype != POETX_BF16 or d.mode != POETX_MEM:
                raise ValueError("an MX4 weight needs a bf16 layer in mem mode")
            W0q = torch.empty(d.d_out, d.d_in // 2, dtype=torch.uint8, device=self.device)
            W0s = torch.empty(d.d_out, d.d_in // 32, dtype=torch.uint8, device=self.device)
            poetx_mx4_quantize(d.dtype, d.d_out, d.d_in, self.W0p, W0q, W0s)
            self.mx4 = True
        else:
            W0q = torch.empty(d.d_out, d.d_in, dtype=torch.int8, device=self.device)
            W0s = torch.empty(d.d_out, dtype=torch.float32, device=self.device)
            poetx_xq_quantize(d, self.W0p, W0q, W0s)
            self.xq = True
        self.W0q, self.W0s = W0q, W0s
        self.W0p = self.W0 = None  # stream-ordered release: the quantiser has been enqueued before it

    def cnp_forward(self, X: torch.Tensor):
        """CNP and layer forward in one library call (the CNP overlaps the input gather)."""
        poetx_cnp_forward(self.desc, self.n, X, self.W0p, self.perm_L, self.perm_R, self.theta_R, self.theta_P,
                          self.Q_R, self.Q_P, self.Y, self.saved, self.ws)
        return self.Y

    def step(self, X: torch.Tensor, dY: torch.Tensor, grad_ready=None):
        """CNP forward + layer forward + layer backward (incl. the CNP adjoint).  grad_ready (for
        data parallelism, e.g. GradBuckets.layer_done of this layer) is called once the backward
        pass, which writes the packed gradients, has been enqueued."""
        if self.xq or self.mx4:
            self.cnp()
            self.forward(X)
        else:
            self.cnp_forward(X)
        self.backward(dY, X)
        if grad_ready is not None:
            grad_ready()

    def optimizer_step(self, cfg: poetx_adamw_cfg, seed: int = 0):
        """AdamW on the packed theta (both sides in one launch).  seed: of the 8-bit moments' rounding (0: to
        nearest; another each step: stochastic)."""
        if self.optimizer is not None:
            x = self.optimizer.tensors[0]
            if x.param is not self.theta or x.grad is not self.grad:  # moved, as into a flat gradient buffer
                self.optimizer = MultiAdamW([x._replace(param=self.theta, grad=self.grad)])
            self.optimizer.step(cfg, t=self.t + 1, seed=seed)
        elif self.m is not None:
            poetx_adamw_step(cfg, self.theta.numel(), self.t + 1, self.theta, self.grad, self.m, self.v)
        else:
            raise ValueError("the layer holds no moments (moments=None): step theta from outside")
        self.t += 1

    def train_step(self, X: torch.Tensor, dY: torch.Tensor, cfg: poetx_adamw_cfg, reset_gap: int = 400,
                   new_perms=None, seed: int = 0):
        """One training step with the merge schedule: CNP, forward, backward, AdamW (seed: as
        optimizer_step's); after every reset_gap steps merge-then-reinitialise with the permutations
        new_perms() returns (host int32 arrays pi_L, pi_R) and restart the moments."""
        self.step(X, dY)
        self.optimizer_step(cfg, seed)
        self.steps += 1
        if reset_gap and self.steps % reset_gap == 0:
            if new_perms is None:
                raise ValueError("the merge schedule needs new permutations")
            pL, pR = new_perms()
            self.cnp()  # Q of the theta being folded in
            self.merge(torch.from_numpy(np.asarray(pL, np.int32)).to(self.device),
                       torch.from_numpy(np.asarray(pR, np.int32)).to(self.device))
            if self.optimizer is not None:
                self.optimizer.reset()
            else:
                poetx_adamw_reset(self.m.numel(), self.m, self.v)
            self.t = 0

    def fourperm_step(self, X: torch.Tensor, dY: torch.Tensor):
        """The same step with none of the permutations absorbed (comparator): R and P applied around
        the original W0, four activation permutations per pass.  Same outputs as step()."""
        if self.W0 is None:
            raise ValueError("the four-permutation comparator needs the un-absorbed weight: load_state() keeps it, "
                             "quantize() releases it")
        if getattr(self, "fp_saved", None) is None:
            self.fp_saved = torch.empty(self.n * (self.desc.d_in + self.desc.d_out), dtype=self.dtype,
                                        device=self.device)
            self.fp_ws = torch.empty(max(poetx_fourperm_workspace_size(self.desc, self.n), 256), dtype=torch.uint8,
                                     device=self.device)
        poetx_cnp(self.desc, self.theta_R, self.theta_P, self.Q_R, self.Q_P, self.fp_ws)
        poetx_fourperm_forward(self.desc, self.n, X, self.W0, self.perm_L, self.perm_R, self.Q_R, self.Q_P, self.Y,
                               self.fp_saved, self.fp_ws)
        poetx_fourperm_backward(self.desc, self.n, dY, self.W0, self.perm_L, self.perm_R, self.Q_R, self.Q_P,
                                self.theta_R, self.theta_P, self.fp_saved, self.dX, self.g_R, self.g_P, self.fp_ws)

    def wc_step(self, X: torch.Tensor, dY: torch.Tensor):
        """The same step in the weight-centric order (comparator): CNP, form W = R W0 P, Y = X W^T,
        dX = dY W, dW = dY^T X and the gradients of theta from dW.  Same outputs as step()."""
        if getattr(self, "wc_saved", None) is None:
            self.wc_saved = torch.empty(poetx_wc_saved_size(self.desc), dtype=torch.uint8, device=self.device)
            self.wc_ws = torch.empty(max(poetx_wc_workspace_size(self.desc), 256), dtype=torch.uint8,
                                     device=self.device)
        poetx_cnp(self.desc, self.theta_R, self.theta_P, self.Q_R, self.Q_P, self.wc_ws)
        poetx_wc_forward(self.desc, self.n, X, self.W0p, self.perm_L, self.perm_R, self.Q_R, self.Q_P, self.Y,
                         self.wc_saved, self.wc_ws)
        poetx_wc_backward(self.desc, self.n, dY, X, self.W0p, self.perm_L, self.perm_R, self.Q_R, self.theta_R,
                          self.theta_P, self.wc_saved, self.dX, self.g_R, self.g_P, self.wc_ws)

    def merge(self, pi_L_new: torch.Tensor, pi_R_new: torch.Tensor):
        """Folds R and P into W0', absorbs the new permutations and resets theta (Q must be current)."""
        if self.xq:
            poetx_xq_merge(self.desc, self.W0q, self.W0s, self.Q_R, self.Q_P, self.perm_L, self.perm_R, pi_L_new,
                           pi_R_new, self.theta_R, self.theta_P, self.ws)
        elif self.mx4:
            poetx_mx4_merge(self.desc, self.W0q, self.W0s, self.Q_R, self.Q_P, self.perm_L, self.perm_R, pi_L_new,
                            pi_R_new, self.theta_R, self.theta_P, self.ws)
        else:
            poetx_merge(self.desc, self.W0p, self.Q_R, self.Q_P, self.perm_L, self.perm_R, pi_L_new, pi_R_new,
                        self.theta_R, self.theta_P, self.ws)
        self.perm_L.copy_(pi_L_new)
        self.perm_R.copy_(pi_R_new)
