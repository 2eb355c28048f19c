"""Sparse linear layer with autograd, built from the four CSR operations.

This is the sparse-adaptation pattern the spops README's SDDMM and csr_add
serve (robust sparse adaptation of a dense weight W by a sparse S): a layer
computes S·x, training needs the gradients with respect to S's stored values
and to the input, and the trained S is finally merged into W.  Activations
are kept feature-major (X^T is in_features x tokens, row-major), which makes
every step one call into libspops and needs no dense transpose:

    forward    Y^T  = S · X^T                         spmm
    backward   dS   = dY^T · (X^T)^T sampled at S     sddmm (A = dY^T, BT = X^T)
               dX^T = S^T · dY^T                      values of S^T (the
                                                      transpose's permutation,
                                                      found once) + spmm
    merge      W   += S                               csr_add
    optimizer  values -= Adam step (masked)           masked_adam (MaskedAdam)

The module only marshals tensors: outputs are allocated here and every value
is computed by the library's kernels (it raises if libspops.so is missing).
"""
from __future__ import annotations

from typing import Optional, Union

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from .spops import (Mx4Matrix, SddmmPlan, SpmmPlan, _marshal, csr_add, csr_transpose_permutation,
                    low_rank_add, low_rank_backward, low_rank_project, masked_adam, mx4_matmul,
                    mx4_quantize, permute_values, sddmm, sort_rows_by_nnz, spmm)


class SparsePattern:
    """A CSR sparsity pattern of S (out_features x in_features) and what is
    derived from it once: the row order, the SpMM / SDDMM plans, the pattern
    of S^T with its own row order and plan, and the permutation that takes
    S's values to S^T's."""

    def __init__(self, row_offsets: torch.Tensor, col_idx: torch.Tensor,
                 out_features: int, in_features: int):
        self.ro, self.ci = row_offsets, col_idx
        self.m, self.n = out_features, in_features
        self.nnz = col_idx.numel()
        self.ri = sort_rows_by_nnz(row_offsets, in_features)
        self.spmm_plan = SpmmPlan(row_offsets, self.ri, col_idx, in_features)
        self.sddmm_plan = SddmmPlan(row_offsets, col_idx, out_features, in_features)
        self.srcT, self.roT, self.ciT = csr_transpose_permutation(row_offsets, col_idx,
                                                                  out_features, in_features)
        self.riT = sort_rows_by_nnz(self.roT, out_features)
        self.spmmT_plan = SpmmPlan(self.roT, self.riT, self.ciT, out_features)

    def transposed_values(self, values: torch.Tensor,
                          out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Values of S^T in the order of the transposed pattern (what
        csr_transpose gives, bit for bit)."""
        return permute_values(values, self.srcT, out=out)


class _SparseLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, values: torch.Tensor, xt: torch.Tensor, pattern: SparsePattern):
        P = pattern
        yt = spmm(values, P.ro, P.ri, P.ci, xt, P.m, out_dtype=xt.dtype, plan=P.spmm_plan)
        ctx.save_for_backward(values, xt)
        ctx.pattern = P
        return yt

    @staticmethod
    @once_differentiable
    def backward(ctx, dyt: torch.Tensor):
        values, xt = ctx.saved_tensors
        P = ctx.pattern
        dyt = dyt.contiguous()
        dv = dxt = None
        if ctx.needs_input_grad[0]:
            dv = sddmm(P.ro, P.ri, P.ci, dyt, xt, plan=P.sddmm_plan, out_dtype=values.dtype)
        if ctx.needs_input_grad[1]:
            vt = P.transposed_values(values)
            dxt = spmm(vt, P.roT, P.riT, P.ciT, dyt, P.n, out_dtype=xt.dtype,
                       plan=P.spmmT_plan)
        return dv, dxt, None


def sparse_linear(values: torch.Tensor, xt: torch.Tensor, pattern: SparsePattern) -> torch.Tensor:
    """Y^T = S · X^T with S = (pattern, values); differentiable in values and X^T.
    values and X^T share a dtype (f32, f16 or bf16); Y^T has that dtype too
    (fp32 accumulation, one rounding)."""
    if values.dtype != xt.dtype:
        raise ValueError("values and X^T must share a dtype")
    if xt.dim() != 2 or xt.shape[0] != pattern.n:
        raise ValueError("X^T must be in_features x tokens")
    return _SparseLinearFn.apply(values, xt, pattern)


class SparseAdapter(torch.nn.Module):
    """A trainable sparse matrix S on a fixed pattern: forward(X^T) = S · X^T;
    merge_into(W) adds S into a dense out_features x in_features weight."""

    def __init__(self, pattern: SparsePattern, values: torch.Tensor):
        super().__init__()
        if values.numel() != pattern.nnz:
            raise ValueError("one value per stored entry of the pattern")
        self.pattern = pattern
        self.values = torch.nn.Parameter(values)

    def forward(self, xt: torch.Tensor) -> torch.Tensor:
        return sparse_linear(self.values, xt, self.pattern)

    @torch.no_grad()
    def merge_into(self, W: torch.Tensor) -> torch.Tensor:
        P = self.pattern
        return csr_add(self.values.detach(), P.ro, P.ri, P.ci, W)


def _apply_keeping(module, types, apply, fn, *args, **kwargs):
    """Moves and casts of a module (apply: torch.nn.Module._apply, by which type() reaches
    integers too): the buffers in `types` move, but keep the type given there, with the
    values they had."""
    kept = {n: module._buffers[n] for n in types if module._buffers.get(n) is not None}
    apply(fn, *args, **kwargs)
    for n, t in kept.items():
        now = module._buffers[n]
        if now.dtype != types[n]:
            module._buffers[n] = t.to(now.device)
    return module


class _Mx4LinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, xt, codes, scales, cols, transposed):
        ctx.save_for_backward(codes, scales)
        ctx.cols, ctx.transposed = cols, transposed
        return mx4_matmul(Mx4Matrix(codes, scales, cols), xt, transposed)

    @staticmethod
    def backward(ctx, dyt):
        codes, scales = ctx.saved_tensors
        return (_Mx4LinearFn.apply(dyt.contiguous(), codes, scales, ctx.cols, not ctx.transposed),
                None, None, None, None)


def mx4_linear(W: Mx4Matrix, xt: torch.Tensor) -> torch.Tensor:
    """W · X^T for a frozen W in four bits; differentiable in X^T (any number of
    times: the gradient is mx4_matmul with W transposed)."""
    return _Mx4LinearFn.apply(xt, W.codes, W.scales, W.cols, False)


class Mx4Linear(torch.nn.Module):
    """A frozen layer of out_features x in_features in 4-bit microscaled form:
    forward(X^T) = W · X^T in the dtype of X^T, differentiable in X^T.  `weight` is a
    matrix to quantise or an Mx4Matrix.  Adapters train on top of it:
    adapters(base(xt), xt, offsets, adapter).  A state of another number of columns does
    not load, also where codes and scales have the same shapes."""

    def __init__(self, weight: Union[torch.Tensor, Mx4Matrix]):
        super().__init__()
        W = weight if isinstance(weight, Mx4Matrix) else mx4_quantize(weight.detach())
        self.cols = W.cols
        self.register_buffer("codes", W.codes)
        self.register_buffer("scales", W.scales)

    @property
    def weight(self) -> Mx4Matrix:
        return Mx4Matrix(self.codes, self.scales, self.cols)

    def state_dict(self, *args, **kwargs):
        """codes and scales; the number of columns, which they do not tell, goes with them
        as the version of a module does."""
        state = super().state_dict(*args, **kwargs)
        prefix = kwargs.get("prefix", args[1] if len(args) > 1 else "")
        getattr(state, "_metadata", {}).get(prefix[:-1], {})["cols"] = self.cols
        return state

    def _load_from_state_dict(self, state_dict, prefix, local_metadata, strict, missing_keys,
                              unexpected_keys, error_msgs):
        cols, codes = local_metadata.get("cols", self.cols), state_dict.get(prefix + "codes")
        if cols != self.cols:
            error_msgs.append(f"{prefix}codes are of {cols} columns, those of the layer of "
                              f"{self.cols}.")
            return
        if (isinstance(codes, torch.Tensor) and codes.shape == self.codes.shape
                and not codes.is_meta):
            # without that number: what lies past the last column has to be zero
            past = codes[:, (self.cols + 1) // 2:]
            if past.any() or self.cols % 2 and (codes[:, self.cols // 2] > 15).any():
                error_msgs.append(f"{prefix}codes hold elements past column {self.cols}.")
                return
        super()._load_from_state_dict(state_dict, prefix, local_metadata, strict, missing_keys,
                                      unexpected_keys, error_msgs)

    def _apply(self, fn, *args, **kwargs):
        types = {"codes": torch.uint8, "scales": torch.uint8}
        return _apply_keeping(self, types, super()._apply, fn, *args, **kwargs)

    def forward(self, xt: torch.Tensor) -> torch.Tensor:
        return _Mx4LinearFn.apply(xt, self.codes, self.scales, self.cols, False)


class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, step):
        ctx.p, ctx.step = p, step
        ctx.seed = seed
        if isinstance(seed, torch.Tensor):
            ctx.save_for_backward(seed)
            ctx.seed = None
        return _marshal().dropout(x, p, seed, step, None)

    @staticmethod
    def backward(ctx, dy):
        seed = ctx.saved_tensors[0] if ctx.seed is None else ctx.seed
        return _DropoutFn.apply(dy.contiguous(), ctx.p, seed, ctx.step), None, None, None


def dropout(x: torch.Tensor, p: float, seed: Union[int, torch.Tensor], step: int = 0,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x with each element set to zero with probability p and the others scaled up to
    keep the mean; the mask is a function of the element's place, seed and step alone
    and is never stored.

    The place is (row, column): of a matrix, or of a contiguous tensor whose last
    dimension are the columns.  An element is dropped when 16 random bits of it are
    below limit = round(65536 p), and kept ones are scaled by 65536 / (65536 - limit).
    `seed` is a number or an int64 vector of seed and step on the device, which is read
    when the kernel runs (a captured call then takes what it holds at each replay; `step`
    is not used).
    Differentiable in x (the gradient is the same call on dy; a vector `seed` must not
    change before it; forward mode raises), unless `out` is given, which may be x."""
    if out is not None:
        if any(t.requires_grad and torch.is_grad_enabled() or _has_tangent(t) for t in (x, out)):
            raise ValueError("dropout into out has no gradient; detach x")
        return _marshal().dropout(x, p, seed, step, out)
    if x.requires_grad and torch.is_grad_enabled() or _has_tangent(x):
        return _DropoutFn.apply(x, p, seed, step)
    return _marshal().dropout(x, p, seed, step, None)


def _has_tangent(t: torch.Tensor) -> bool:
    """Whether t is a dual tensor, whose tangent only an autograd function can refuse.  (The
    level is looked at first: unpack_dual alone is 0.4 us of a call of 4.5.)"""
    return forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None


class _LowRankLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, yt, xt, A, B, offsets, adapter, scale, ranks):
        ctx.save_for_backward(xt, A, B, offsets, adapter, scale, ranks)
        return low_rank_add(yt, xt, A, B, offsets, adapter, scale, ranks)

    @staticmethod
    @once_differentiable
    def backward(ctx, dyt):
        xt, A, B, offsets, adapter, scale, ranks = ctx.saved_tensors
        dx = dA = dB = None
        if any(ctx.needs_input_grad[1:4]):
            dx, dA, dB = low_rank_backward(dyt.contiguous(), xt, A, B, offsets, adapter, scale,
                                           ranks)
        need = ctx.needs_input_grad
        return (dyt if need[0] else None, dx if need[1] else None, dA if need[2] else None,
                dB if need[3] else None, None, None, None, None)


def low_rank_linear(yt: torch.Tensor, xt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                    offsets: torch.Tensor, adapter: torch.Tensor,
                    scale: Optional[torch.Tensor] = None,
                    ranks: Optional[torch.Tensor] = None) -> torch.Tensor:
    """low_rank_add, differentiable once in yt, xt, A and B.  scale has no gradient:
    one that requires it is refused."""
    if scale is not None and scale.requires_grad and torch.is_grad_enabled():
        raise ValueError("scale has no gradient; detach it")
    return _LowRankLinearFn.apply(yt, xt, A, B, offsets, adapter, scale, ranks)


class LowRankAdapters(torch.nn.Module):
    """A pool of low-rank adapters on one layer of out_features x in_features:
    A starts random, B at zero, so a new adapter changes nothing.

      forward(yt, xt, offsets, adapter)   yt + the requests' adapters, for
                                          training and prompts
      project(W, xt, offsets, adapter)    W xt + the same in one pass over W,
                                          for decode steps (no gradient, no
                                          dropout)

    yt may come from any layer on xt, a dense product, a SparseAdapter or an Mx4Linear;
    W may be an Mx4Matrix (whose product is rounded before the adapters' part is added,
    in two passes).  scale and ranks (one value per adapter, of any device and
    type) are kept as float32 and int32 buffers, also where the module is cast.

    With dropout = p, forward in training drops elements of xt on the adapters' side
    (not in yt) with probability p.  The masks follow from `dropout_state`, an int64
    buffer of a seed and a step that each such call advances on the device.  Modules of
    equal seeds and input sizes draw equal masks at a step: each layer, and each rank of a
    data-parallel job, needs a seed of its own (which a broadcast of buffers undoes).  By
    default it is a number of torch's generator.  A forward pass that is run again in the
    backward pass (for activations that were not kept) needs the mask it had: take the
    state before, and give it to both:

      checkpoint(layer, yt, xt, offsets, adapter, layer.next_dropout_state())

    Without it such a pass raises, unless dropout_state was set back by hand."""

    # the version of dropout_state that next_dropout_state left
    _dropout_version: Optional[int] = None

    def __init__(self, adapters: int, rank: int, in_features: int, out_features: int,
                 scale: Optional[torch.Tensor] = None, ranks: Optional[torch.Tensor] = None,
                 dtype: torch.dtype = torch.float32, device="cuda", dropout: float = 0.0,
                 seed: Optional[int] = None):
        super().__init__()
        if not 0.0 <= dropout <= 1.0:
            raise ValueError("dropout must be between 0 and 1")
        A = torch.randn(adapters, rank, in_features, device=device) * in_features ** -0.5
        self.A = torch.nn.Parameter(A.to(dtype))
        self.B = torch.nn.Parameter(torch.zeros(adapters, out_features, rank, dtype=dtype,
                                                device=device))
        # the calls take them in these types alone, whatever the factors' dtype
        self.register_buffer("scale", scale if scale is None else
                             scale.to(device, torch.float32))
        self.register_buffer("ranks", ranks if ranks is None else ranks.to(device, torch.int32))
        self.dropout = dropout
        if dropout > 0.0:
            if seed is None:
                seed = int(torch.randint(1 << 62, (), dtype=torch.int64))
            self.register_buffer("dropout_state",
                                 torch.tensor([seed, 0], dtype=torch.int64, device=device))

    def _apply(self, fn, *args, **kwargs):
        types = {"scale": torch.float32, "ranks": torch.int32, "dropout_state": torch.int64}
        return _apply_keeping(self, types, super()._apply, fn, *args, **kwargs)

    def _drops(self) -> bool:
        # the constructor's own number: a module that was kept whole before it had one has
        # none, and a class made from this one may have a layer of that name
        return self.training and self.__dict__.get("dropout", 0.0) > 0.0

    def next_dropout_state(self) -> Optional[torch.Tensor]:
        """The seed and step of the next forward pass in training, a copy that forward
        takes as `state`; dropout_state advances.  None where nothing is dropped."""
        if not self._drops():
            return None
        at = self.dropout_state
        # a pass that is run again here would draw the mask of another step
        if torch._C._current_graph_task_id() != -1 and _version(at) == self._dropout_version:
            raise RuntimeError("a forward pass with dropout inside a backward pass draws another "
                               "mask; take next_dropout_state() before and give it as state")
        state = at.clone()
        at[1].add_(1)
        self._dropout_version = _version(at)
        return state

    def forward(self, yt: torch.Tensor, xt: torch.Tensor, offsets: torch.Tensor,
                adapter: torch.Tensor, state: Optional[torch.Tensor] = None) -> torch.Tensor:
        """`state`: of next_dropout_state, which is called where none is given."""
        if self._drops():
            # the backward pass draws the mask again from the state, which is a copy
            xt = dropout(xt, self.dropout, self.next_dropout_state() if state is None else state)
        return low_rank_linear(yt, xt, self.A, self.B, offsets, adapter, self.scale, self.ranks)

    @torch.no_grad()
    def project(self, W: Union[torch.Tensor, Mx4Matrix], xt: torch.Tensor, offsets: torch.Tensor,
                adapter: torch.Tensor) -> torch.Tensor:
        if isinstance(W, Mx4Matrix):
            yt = mx4_matmul(W, xt)
            return low_rank_add(yt, xt, self.A, self.B, offsets, adapter, self.scale, self.ranks,
                                out=yt)
        return low_rank_project(W, xt, self.A, self.B, offsets, adapter, self.scale, self.ranks)


def _version(t: torch.Tensor) -> int:
    return -1 if t.is_inference() else t._version


class MaskedAdam(torch.optim.Optimizer):
    """The masked Adam of the SparseAdam page (tensorplay.optim.sparse_adam)
    for value vectors, each step one launch of the library's kernel
    (spops_masked_adam).  A dense gradient updates every value; a 1-D sparse
    COO gradient (coalesced) updates only the values it names, leaving the
    others and their moments untouched.  Moments are kept in f32."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 maximize: bool = False):
        if not (lr >= 0.0 and eps >= 0.0 and 0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0):
            raise ValueError("need lr >= 0, eps >= 0 and betas in [0, 1)")
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps, maximize=maximize))

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            for p in group["params"]:
                if p.grad is None:
                    continue
                if p.dim() != 1 or not p.is_contiguous():
                    raise ValueError("MaskedAdam trains contiguous 1-D value vectors")
                st = self.state[p]
                if not st:
                    st["step"] = 0
                    st["exp_avg"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                    st["exp_avg_sq"] = torch.zeros(p.shape, dtype=torch.float32,
                                                   device=p.device)
                st["step"] += 1
                g = p.grad
                kw = dict(lr=group["lr"], betas=group["betas"], eps=group["eps"],
                          maximize=group["maximize"])
                if g.is_sparse:
                    if not g.is_coalesced():
                        raise ValueError("sparse gradients must be coalesced")
                    pos = g.indices()[0].to(torch.int32)
                    masked_adam(p.data, g.values().contiguous(), st["exp_avg"],
                                st["exp_avg_sq"], st["step"], positions=pos, **kw)
                else:
                    masked_adam(p.data, g.contiguous(), st["exp_avg"], st["exp_avg_sq"],
                                st["step"], **kw)
        return loss
