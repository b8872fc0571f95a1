"""The training step around HSTURunner: the stack's gradients, the gradient of
the embedding table's touched rows, the clipping norm and the AdamW update, in
that order on one stream, with no host synchronisation.  Allocation goes
through torch; the computation is the library's."""
from __future__ import annotations

from typing import Optional

from . import binding as _b
from .runner import HSTURunner

# parameter -> (its gradient, whether weight decay applies to it)
_PARAMS = {"W1": ("dW1", True), "W2": ("dW2", True), "b1": ("db1", False), "b2": ("db2", False),
           "ln_gamma": ("dln_gamma", False), "ln_beta": ("dln_beta", False),
           "rab_pos": ("drab_pos", False), "rab_time": ("drab_time", False)}


class HSTUTrainer:
    """Optimizer state of a runner's weights (bf16 layers), and of an embedding
    table if one is given.

    The 16-bit weights get fp32 masters; where the runner holds fp16 copies of
    W1 and W2 the update writes them too, so the next forward needs no
    conversion.  `table`: device [rows, d_model] (for hstu_sl_embed_ids: the
    content rows, then the action rows); at most `max_tokens` tokens per step.
    Only the rows that a step's tokens touch are updated.  A 16-bit table has an
    fp32 master like the weights (4 bytes an element); a table that is to do
    without one can be updated by hstu_adamw_step directly.

    The state is made on torch's current stream; a step on another stream has
    to be ordered behind that (`stream.wait_stream`), as for its inputs.  The step
    number is counted on the host: a captured step() would replay its own (for
    a graph, hstu_adamw_step takes the number from the device)."""

    def __init__(self, runner: HSTURunner, table=None, max_tokens: int = 0, state_bits: int = 32,
                 lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, table_decay: float = 0.0, max_norm: float = 1.0,
                 seed: int = 0):
        if runner.dtype != "bf16" or state_bits not in (8, 32):
            raise _b.HstuError(2, "HSTUTrainer")
        t = runner.torch
        self.torch, self.runner, self.table = t, runner, table
        self.lr, self.betas, self.eps = lr, betas, eps
        self.max_norm, self.seed, self.state_bits, self.steps = max_norm, seed, state_bits, 0
        dev = runner.device
        self.grads = [{g: t.zeros(w[p].shape, dtype=t.float32, device=dev)
                       for p, (g, _) in _PARAMS.items()} for w in runner.weights]
        self.tensors = []
        for w, gs in zip(runner.weights, self.grads):
            for p, (g, decayed) in _PARAMS.items():
                e = dict(param=w[p], grad=gs[g], weight_decay=weight_decay if decayed else 0.0,
                         copy_f16=w.get(p + "_f16"))
                self.tensors.append(self._states(e, (w[p].numel(),)))
        if table is not None:
            rows, d = table.shape
            cap = max(1, min(int(max_tokens), rows))
            self.max_tokens = int(max_tokens)
            self.row_ids = t.zeros(cap, dtype=t.int64, device=dev)
            self.row_grad = t.zeros(cap, d, dtype=t.float32, device=dev)
            self.n_rows = t.zeros(1, dtype=t.int64, device=dev)
            e = dict(param=table, grad=self.row_grad, row_ids=self.row_ids, n_rows=self.n_rows,
                     weight_decay=table_decay)
            self.tensors.append(self._states(e, (rows, d)))
            self._ews = self._workspace(_b.hstu_embed_bwd_workspace_size(self.max_tokens, rows, d))
        self.list = _b.AdamWTensors(self.tensors)
        self.norm = t.zeros(2, dtype=t.float32, device=dev)
        self._nws = self._workspace(_b.hstu_grad_norm_workspace_size())
        self._ows = self._workspace(_b.hstu_adamw_workspace_size())

    def _workspace(self, nbytes: int):
        ws = self.torch.empty(nbytes, dtype=self.torch.uint8, device=self.runner.device)
        ws[:4] = 0  # the status word: HSTU_OK until a call writes it
        return ws

    def _states(self, e, shape):
        t = self.torch
        p = e["param"]
        dev = p.device
        if p.dtype != t.float32:
            e["master"] = p.float()
        dt = t.float32 if self.state_bits == 32 else t.float8_e4m3fn
        for k in ("m", "v"):
            e[k] = t.zeros(p.shape, dtype=t.uint8 if self.state_bits == 8 else dt,
                           device=dev).view(dt)
            if self.state_bits == 8:
                e[k + "_scale"] = t.zeros(_b.state_scales(shape), dtype=t.uint8, device=dev)
        return e

    def step(self, offsets, X, timestamps, dY, max_len: int, ids=None, embed_scale: float = 1.0,
             pad_id: int = -1, lr=None, stream=None):
        """One update from the gradient dY of a loss with respect to the
        stack's output.  `ids` (with a table): the table row of each row of X,
        which was looked up with the factor `embed_scale`.  `lr`: this step's
        rate (default: the constructor's).  Returns dX; `norm` holds the
        gradient norm and the clip factor.  A step whose gradients are not all
        finite, or whose backward pass failed on the device (a bad batch;
        status() tells), has a clip factor of NaN and changes nothing, but is
        counted in `steps`; dX is not written by a failed pass."""
        if (ids is None) != (self.table is None):
            raise _b.HstuError(1, "HSTUTrainer.step: ids and a table come together")
        if ids is not None and ids.numel() > self.max_tokens:
            raise _b.HstuError(3, "HSTUTrainer.step: more tokens than max_tokens")
        dX, _ = self.runner.stack_bwd(offsets, X, timestamps, dY, max_len, grads=self.grads,
                                      stream=stream)
        if ids is not None:
            _b.hstu_embed_bwd_rows(ids, dX, self.table.shape[0], self.row_ids, self.row_grad,
                                   self.n_rows, self._ews, scale=embed_scale, pad_id=pad_id,
                                   stream=stream)
        _b.hstu_grad_norm_after(self.list, self.max_norm, self.runner._bws, self.norm, self._nws,
                                stream=stream)
        self.steps += 1
        _b.hstu_adamw_step(self.list, self._ows, lr=self.lr if lr is None else lr,
                           step=self.steps, beta1=self.betas[0], beta2=self.betas[1],
                           eps=self.eps, grad_scale=self.norm[1:], seed=self.seed, stream=stream)
        return dX

    def status(self, stream=None) -> int:
        """The first status that is not HSTU_OK of the last step's calls (HSTU_OK
        before the first one)."""
        for ws in [self.runner._bws] + ([self._ews] if self.table is not None else []) + \
                [self._nws, self._ows]:
            s = 0 if ws is None else _b.hstu_read_status(ws, stream)
            if s != 0:
                return s
        return 0
