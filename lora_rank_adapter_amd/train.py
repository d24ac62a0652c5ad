"""Binding of the operators of a training step around the adapter linears:
embedding lookup and gradient, the losses on next-token logits, their
alternatives and entropy, distillation, AdamW.

As in ``ops``: argument marshalling only. Vectors (ids, targets, log
probabilities, ...) are checked here for dtype, length and layout, since the
library takes them as bare pointers; matrices are checked by the library.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import LoraAdamwState, LoraAdamwTensor, check, pack_hyper, pack_mat, pack_policy, pack_teacher
from .ops import _DT, _dtype_code, _stream

_I32, _F32 = torch.int32, torch.float32
_data_ptr = torch.Tensor.data_ptr


def _vector(name: str, t: torch.Tensor, n: int, dtype: torch.dtype, device: torch.device) -> int:
    """The address of a contiguous vector of n elements of dtype on device."""
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements, "
                         f"got {t.dtype} {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.data_ptr()


def _queue(device: torch.device):
    """torch's current stream on a GPU; tensors elsewhere are refused before their addresses get there."""
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a GPU, got {device}")
    return _stream(device)


def _here(device: torch.device):
    """_queue for tensors on the current device, which is where a launch goes."""
    queue = _queue(device)
    if device.index is not None and device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device}, which is not the current device")
    return queue


def _capturing(stream) -> bool:
    """Whether a graph is being captured on torch's current stream, `stream` (the default stream cannot be)."""
    return stream.value is not None and torch.cuda.is_current_stream_capturing()


def _matrix(name: str, t: torch.Tensor, device: torch.device) -> bytes:
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected a 2-D tensor, got shape {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    row, col = t.stride()
    return pack_mat(t.data_ptr(), _DT.get(t.dtype, -1), 0, shape[0], shape[1], row, col)


def _given(workspace, need, device):
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    return workspace, workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------

def lora_embed(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0, out: torch.Tensor | None = None,
               dtype: torch.dtype | None = None) -> torch.Tensor:
    """out[t] = scale * table[ids[t]] (zeros for ids outside [0, V)). ids: int32 [T], table: V x D. Returns out
    [T x D]: the given tensor, else a new one of `dtype` (default the table's; float32, or bfloat16 with a
    bfloat16 table)."""
    lib = _lib.load()
    T, dev = ids.numel(), table.device
    p = _vector("ids", ids, T, _I32, dev)
    if out is None:
        out = torch.empty((T, table.shape[1]), dtype=dtype or table.dtype, device=dev)
    elif out.shape[0] != T:
        raise ValueError(f"out has {out.shape[0]} rows for {T} ids")
    check("lora_embed", lib.lora_embed(p, _matrix("table", table, dev), float(scale), _matrix("out", out, dev),
                                       _queue(dev)))
    return out


def lora_embed_grad(ids: torch.Tensor, dy: torch.Tensor, num_rows: int, scale: float = 1.0,
                    dtable: torch.Tensor | None = None, accumulate: bool = False,
                    workspace: torch.Tensor | None = None, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """dtable[v] = scale * sum of dy[t] over the tokens with ids[t] = v. ids: int32 [T], dy: T x D. Returns dtable
    [num_rows x D]: the given tensor (overwritten, or with accumulate added to), else a new one of `dtype`
    (float32, or bfloat16 with bfloat16 dy)."""
    lib = _lib.load()
    T, D = dy.shape
    dev = dy.device
    p = _vector("ids", ids, T, _I32, dev)
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs the dtable to add to")
        dtable = torch.empty((num_rows, D), dtype=dtype, device=dev)
    elif dtable.shape[0] != num_rows:
        raise ValueError(f"dtable has {dtable.shape[0]} rows, expected {num_rows}")
    ws, nbytes = _given(workspace, lib.lora_embed_grad_workspace_bytes(T, num_rows, D), dev)
    check("lora_embed_grad", lib.lora_embed_grad(p, _matrix("dy", dy, dev), float(scale),
                                                 _matrix("dtable", dtable, dev), int(bool(accumulate)), ws.data_ptr(),
                                                 nbytes, _queue(dev)))
    return dtable


# ---------------------------------------------------------------------------
# losses
# ---------------------------------------------------------------------------

def lora_token_logp(logits: torch.Tensor, targets: torch.Tensor,
                    workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Log probabilities of the targets (0 where a target lies outside [0, V)) and the rows' softmax statistics.
    logits: T x V, targets: int32 [T]. Returns (logp [T], stats [T x 2]: the largest logit m and the sum of
    exp(x - m)), both float32."""
    lib = _lib.load()
    T, V = logits.shape
    dev = logits.device
    y = _vector("targets", targets, T, _I32, dev)
    logp = torch.empty(T, dtype=_F32, device=dev)
    stats = torch.empty((T, 2), dtype=_F32, device=dev)
    ws, nbytes = _given(workspace, lib.lora_loss_workspace_bytes(T, V), dev)
    check("lora_token_logp", lib.lora_token_logp(_matrix("logits", logits, dev), y, logp.data_ptr(), stats.data_ptr(),
                                                 ws.data_ptr(), nbytes, _queue(dev)))
    return logp, stats


def _pairs(seq_offsets: torch.Tensor) -> int:
    n = seq_offsets.numel() - 1
    if n < 2 or n % 2:
        raise ValueError(f"seq_offsets must hold 2 * pairs + 1 offsets, got {n + 1}")
    return n // 2


def lora_pref_loss(logp: torch.Tensor, seq_offsets: torch.Tensor, ref_logp: torch.Tensor, beta: float,
                   label_smoothing: float = 0.0) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Preference loss of paired sequences from their tokens' log probabilities. seq_offsets: int32
    [2 * pairs + 1], sequences 2p (preferred) and 2p + 1 of pair p; ref_logp: float32 [2 * pairs].
    Returns (loss [], seq_logp [2 * pairs], coef [T]: d loss / d logp)."""
    lib = _lib.load()
    T, dev, pairs = logp.numel(), logp.device, _pairs(seq_offsets)
    loss = torch.empty((), dtype=_F32, device=dev)
    seq = torch.empty(2 * pairs, dtype=_F32, device=dev)
    coef = torch.empty(T, dtype=_F32, device=dev)
    check("lora_pref_loss", lib.lora_pref_loss(
        _vector("logp", logp, T, _F32, dev), T, _vector("seq_offsets", seq_offsets, 2 * pairs + 1, _I32, dev), pairs,
        _vector("ref_logp", ref_logp, 2 * pairs, _F32, dev), float(beta), float(label_smoothing), loss.data_ptr(),
        seq.data_ptr(), coef.data_ptr(), _queue(dev)))
    return loss, seq, coef


def _policy(targets, T, old_logp, advantages, weights, clip_low, clip_high, ref_logp, kl_coef, dev) -> bytes:
    if kl_coef != 0.0 and ref_logp is None:
        raise ValueError("kl_coef needs ref_logp")
    return pack_policy(_vector("targets", targets, T, _I32, dev), _vector("old_logp", old_logp, T, _F32, dev),
                       0 if ref_logp is None else _vector("ref_logp", ref_logp, T, _F32, dev),
                       _vector("advantages", advantages, T, _F32, dev), _vector("weights", weights, T, _F32, dev),
                       clip_low, clip_high, kl_coef)


def lora_policy_loss(logp: torch.Tensor, targets: torch.Tensor, vocab: int, old_logp: torch.Tensor,
                     advantages: torch.Tensor, weights: torch.Tensor, clip_low: float, clip_high: float,
                     ref_logp: torch.Tensor | None = None,
                     kl_coef: float = 0.0) -> tuple[torch.Tensor, torch.Tensor]:
    """Clipped policy loss with a KL term from the tokens' log probabilities (all vectors float32 [T], targets
    int32; a target outside [0, vocab) masks its token). Returns (loss [], coef [T]: d loss / d logp)."""
    lib = _lib.load()
    T, dev = logp.numel(), logp.device
    args = _policy(targets, T, old_logp, advantages, weights, clip_low, clip_high, ref_logp, kl_coef, dev)
    loss = torch.empty((), dtype=_F32, device=dev)
    coef = torch.empty(T, dtype=_F32, device=dev)
    check("lora_policy_loss", lib.lora_policy_loss(_vector("logp", logp, T, _F32, dev), T, int(vocab),
                                                   args, loss.data_ptr(), coef.data_ptr(), _queue(dev)))
    return loss, coef


def lora_logit_grad(logits: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor, coef: torch.Tensor,
                    grad_out: torch.Tensor | None = None, scale: float = 1.0, dlogits: torch.Tensor | None = None,
                    logp: torch.Tensor | None = None) -> torch.Tensor:
    """dlogits[t] = scale * grad_out * coef[t] * (one at targets[t] - softmax(logits[t])). stats from
    lora_token_logp on the same logits and targets, logp its log probabilities (without them rows with a likely
    target are read once more), grad_out: float32 [] on the device or None. Returns dlogits [T x V] of the logits'
    dtype: the given tensor (it may be the logits), else a new one."""
    lib = _lib.load()
    T = logits.shape[0]
    dev = logits.device
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    head = (_matrix("logits", logits, dev), _vector("targets", targets, T, _I32, dev),
            _vector("stats", stats, 2 * T, _F32, dev))
    lp = None if logp is None else _vector("logp", logp, T, _F32, dev)
    rest = (_vector("coef", coef, T, _F32, dev),
            None if grad_out is None else _vector("grad_out", grad_out, 1, _F32, dev), float(scale),
            _matrix("dlogits", dlogits, dev), _queue(dev))
    if logp is None:
        check("lora_logit_grad", lib.lora_logit_grad(*head, *rest))
    else:
        check("lora_logit_grad_logp", lib.lora_logit_grad_logp(*head, lp, *rest))
    return dlogits


def lora_pref_step(logits: torch.Tensor, targets: torch.Tensor, seq_offsets: torch.Tensor, ref_logp: torch.Tensor,
                   beta: float, label_smoothing: float = 0.0, grad_scale: float = 1.0,
                   dlogits: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Preference loss and the gradient of its logits in one call (see lora_pref_loss, lora_logit_grad). Returns
    (loss [], seq_logp [2 * pairs], logp [T], dlogits [T x V], times grad_scale)."""
    lib = _lib.load()
    T, V = logits.shape
    dev, pairs = logits.device, _pairs(seq_offsets)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    logp = torch.empty(T, dtype=_F32, device=dev)
    seq = logp.new_empty(2 * pairs)
    loss = logp.new_empty(())
    ws, nbytes = _given(workspace, lib.lora_loss_workspace_bytes(T, V), dev)
    check("lora_pref_step", lib.lora_pref_step(
        _matrix("logits", logits, dev), _vector("targets", targets, T, _I32, dev),
        _vector("seq_offsets", seq_offsets, 2 * pairs + 1, _I32, dev), pairs,
        _vector("ref_logp", ref_logp, 2 * pairs, _F32, dev), float(beta), float(label_smoothing), float(grad_scale),
        loss.data_ptr(), seq.data_ptr(), logp.data_ptr(), _matrix("dlogits", dlogits, dev), ws.data_ptr(), nbytes,
        _queue(dev)))
    return loss, seq, logp, dlogits


def lora_policy_step(logits: torch.Tensor, targets: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
                     weights: torch.Tensor, clip_low: float, clip_high: float, ref_logp: torch.Tensor | None = None,
                     kl_coef: float = 0.0, grad_scale: float = 1.0, dlogits: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None):
    """Policy loss and the gradient of its logits in one call (see lora_policy_loss, lora_logit_grad). Returns
    (loss [], logp [T], dlogits [T x V], times grad_scale)."""
    lib = _lib.load()
    T, V = logits.shape
    dev = logits.device
    args = _policy(targets, T, old_logp, advantages, weights, clip_low, clip_high, ref_logp, kl_coef, dev)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    logp = torch.empty(T, dtype=_F32, device=dev)
    loss = logp.new_empty(())
    ws, nbytes = _given(workspace, lib.lora_loss_workspace_bytes(T, V), dev)
    check("lora_policy_step", lib.lora_policy_step(
        _matrix("logits", logits, dev), args, float(grad_scale), loss.data_ptr(), logp.data_ptr(),
        _matrix("dlogits", dlogits, dev), ws.data_ptr(), nbytes, _queue(dev)))
    return loss, logp, dlogits


# ---------------------------------------------------------------------------
# alternatives and entropy
# ---------------------------------------------------------------------------

def lora_token_top(logits: torch.Tensor, targets: torch.Tensor | None = None, k: int = 0, temperature: float = 1.0,
                   workspace: torch.Tensor | None = None):
    """What softmax(logits / temperature) holds in each row: the log probabilities of the targets (None without
    them), the entropy, and the k largest logits' ids and log probabilities (in order, ties to the lowest id; id -1
    and -inf past the vocabulary). logits: T x V, targets: int32 [T]; a target outside [0, V) masks its row (0, 0,
    -1 and -inf). Returns (logp [T], entropy [T], top_ids int32 [T x k], top_logp [T x k], stats [T x 3])."""
    lib = _lib.load()
    T, V = logits.shape
    dev = logits.device
    k = int(k)
    y = None if targets is None else _vector("targets", targets, T, _I32, dev)
    entropy = torch.empty(T, dtype=_F32, device=dev)
    logp = None if targets is None else torch.empty(T, dtype=_F32, device=dev)
    ids = torch.empty((T, max(k, 0)), dtype=_I32, device=dev)
    top = torch.empty((T, max(k, 0)), dtype=_F32, device=dev)
    stats = torch.empty((T, 3), dtype=_F32, device=dev)
    ws, nbytes = _given(workspace, lib.lora_token_top_workspace_bytes(T, V, k), dev)
    check("lora_token_top", lib.lora_token_top(
        _matrix("logits", logits, dev), y, k, float(temperature), None if logp is None else logp.data_ptr(),
        entropy.data_ptr(), ids.data_ptr(), top.data_ptr(), stats.data_ptr(), ws.data_ptr(), nbytes, _here(dev)))
    return logp, entropy, ids, top, stats


def lora_token_top_grad(logits: torch.Tensor, targets: torch.Tensor | None, stats: torch.Tensor,
                        dlogp: torch.Tensor | None = None, dentropy: torch.Tensor | None = None,
                        temperature: float = 1.0, dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of the logits of a loss with d loss / d logp = dlogp and d loss / d entropy = dentropy (float32 [T]
    or None; dlogp needs targets). stats from lora_token_top on the same logits, targets and temperature. Returns
    dlogits [T x V] of the logits' dtype: the given tensor (it may be the logits), else a new one."""
    lib = _lib.load()
    T = logits.shape[0]
    dev = logits.device
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    check("lora_token_top_grad", lib.lora_token_top_grad(
        _matrix("logits", logits, dev), None if targets is None else _vector("targets", targets, T, _I32, dev),
        _vector("stats", stats, 3 * T, _F32, dev), None if dlogp is None else _vector("dlogp", dlogp, T, _F32, dev),
        None if dentropy is None else _vector("dentropy", dentropy, T, _F32, dev), float(temperature),
        _matrix("dlogits", dlogits, dev), _here(dev)))
    return dlogits


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

def _teacher(top_ids, top_logp, T, temperature, rest, dev) -> tuple[bytes, int]:
    if top_ids.dim() != 2 or top_ids.shape != top_logp.shape:
        raise ValueError(f"top_ids and top_logp must have one 2-D shape, got {tuple(top_ids.shape)} and "
                         f"{tuple(top_logp.shape)}")
    k = top_ids.shape[1]
    return pack_teacher(_vector("top_ids", top_ids, T * k, _I32, dev), _vector("top_logp", top_logp, T * k, _F32, dev),
                        k, temperature, int(bool(rest))), k


def lora_distill_kl(logits: torch.Tensor, top_ids: torch.Tensor, top_logp: torch.Tensor, temperature: float = 1.0,
                    rest: bool = True, workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Divergence of softmax(logits / temperature) from a teacher's top tokens in each row. top_ids int32 [T x k],
    top_logp float32 [T x k]: the teacher's, as lora_token_top gives them at that temperature; ids outside [0, V)
    are no entries, a row without any is masked. rest: the other tokens' probability counts as one more class,
    otherwise the teacher's are normalised over its ids (top_logp may then be its logits over the temperature).
    Returns (kl [T], state [T x (k + 2)] for lora_distill_grad)."""
    lib = _lib.load()
    T, V = logits.shape
    dev = logits.device
    teacher, k = _teacher(top_ids, top_logp, T, temperature, rest, dev)
    kl = torch.empty(T, dtype=_F32, device=dev)
    state = torch.empty((T, k + 2), dtype=_F32, device=dev)
    ws, nbytes = _given(workspace, lib.lora_distill_workspace_bytes(T, V, k), dev)
    check("lora_distill_kl", lib.lora_distill_kl(_matrix("logits", logits, dev), teacher, kl.data_ptr(),
                                                 state.data_ptr(), ws.data_ptr(), nbytes, _here(dev)))
    return kl, state


def lora_distill_grad(logits: torch.Tensor, top_ids: torch.Tensor, state: torch.Tensor, coef: torch.Tensor,
                      temperature: float = 1.0, grad_out: torch.Tensor | None = None, scale: float = 1.0,
                      dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """dlogits[t] = scale * grad_out * coef[t] * d kl[t] / d logits[t]. top_ids, state and temperature of the
    lora_distill_kl on the same logits, coef: float32 [T], grad_out: float32 [] on the device or None. Returns
    dlogits [T x V] of the logits' dtype: the given tensor (it may be the logits), else a new one."""
    lib = _lib.load()
    T = logits.shape[0]
    dev = logits.device
    if top_ids.dim() != 2:
        raise ValueError(f"top_ids: expected a 2-D tensor, got shape {tuple(top_ids.shape)}")
    k = top_ids.shape[1]
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    check("lora_distill_grad", lib.lora_distill_grad(
        _matrix("logits", logits, dev), _vector("top_ids", top_ids, T * k, _I32, dev), k,
        _vector("state", state, T * (k + 2), _F32, dev), _vector("coef", coef, T, _F32, dev),
        None if grad_out is None else _vector("grad_out", grad_out, 1, _F32, dev), float(scale), float(temperature),
        _matrix("dlogits", dlogits, dev), _here(dev)))
    return dlogits


def lora_distill_step(logits: torch.Tensor, top_ids: torch.Tensor, top_logp: torch.Tensor, weights: torch.Tensor,
                      temperature: float = 1.0, rest: bool = True, grad_scale: float = 1.0,
                      dlogits: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """loss = sum of weights * kl and the gradient of its logits in one call (see lora_distill_kl). weights: float32
    [T], a token's share of the loss, e.g. temperature^2 / number of tokens; a weight of zero drops its term. Returns
    (loss [], kl [T], dlogits [T x V], times grad_scale)."""
    lib = _lib.load()
    T, V = logits.shape
    dev = logits.device
    teacher, k = _teacher(top_ids, top_logp, T, temperature, rest, dev)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    kl = torch.empty(T, dtype=_F32, device=dev)
    loss = kl.new_empty(())
    ws, nbytes = _given(workspace, lib.lora_distill_workspace_bytes(T, V, k), dev)
    check("lora_distill_step", lib.lora_distill_step(
        _matrix("logits", logits, dev), teacher, _vector("weights", weights, T, _F32, dev), float(grad_scale),
        loss.data_ptr(), kl.data_ptr(), _matrix("dlogits", dlogits, dev), ws.data_ptr(), nbytes, _here(dev)))
    return loss, kl, dlogits


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

class AdamW:
    """AdamW over many tensors, one launch per step (and one for its constants).

    params: contiguous float32 or bfloat16 tensors, updated in place; grads: their gradients in the caller's
    buffers (float32 or bfloat16; the ones that lora_bwd_dx_da and lora_bwd_db write); shadows: None, or for each
    param None or a bfloat16 tensor that receives a float32 param's new value. All of a param's tensors have its
    shape: elements pair by their place, so the weights are kept the way their gradients lie (A as K x r, B as
    r x L), not as transposes of them. No two params or shadows share memory. The object holds these tensors and a
    device table of their addresses; `bind` replaces the gradients, `step` refuses tensors whose memory moved.

    The table and new states are written on the stream that is current in the constructor and in `bind`; a step on
    another stream waits for that. A step that was captured into a graph goes on with the tensors bound then, also
    after a later `bind`: its table and they are kept while the object lives (which has to be as long as the graph
    is replayed). The graph waits for nothing: it is replayed after what the current stream holds at its capture.

    state_bits 32 keeps both moments in float32, 8 as e4m3 codes with a float32 scale for every 256 elements.
    state: a dict of the tensors step, m, v (and m_scale, v_scale with 8 bits) to go on from; they are used in
    place. The new ones are zeros. All of it is in `self.state`, the layout in include/lora.h.
    """

    def __init__(self, params, grads, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 state_bits: int = 32, state: dict | None = None, shadows=None):
        self.params, self.lr, self.betas, self.eps, self.weight_decay = list(params), lr, betas, eps, weight_decay
        self.state_bits = state_bits
        self.shadows = [None] * len(self.params) if shadows is None else list(shadows)
        if not self.params:
            raise ValueError("AdamW needs a parameter")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if len(self.shadows) != len(self.params):
            raise ValueError(f"{len(self.shadows)} shadows for {len(self.params)} params")
        self._lib = _lib.load()
        self.device = self.params[0].device
        self._shapes = [p.shape for p in self.params]
        self._captured, self._kept, self._event = False, [], torch.cuda.Event()
        self._bind(grads)
        n = self._lib.lora_adamw_state_elems(self._tensors, len(self.params))
        codes = torch.float8_e4m3fn if state_bits == 8 else _F32
        want = {"step": (1, _I32), "m": (n, codes), "v": (n, codes)}
        if state_bits == 8:
            want.update(m_scale=(n // 256, _F32), v_scale=(n // 256, _F32))
        if state is None:
            state = {k: torch.zeros(c, dtype=_F32 if d is codes else d, device=self.device).to(d)
                     for k, (c, d) in want.items()}
        if set(state) != set(want):
            raise ValueError(f"state must hold {sorted(want)}, got {sorted(state)}")
        self.state = dict(state)
        at = {k: _vector(k, self.state[k], c, d, self.device) for k, (c, d) in want.items()}
        self._addresses_of_state = at
        self._mark()
        self._state = LoraAdamwState(state_bits, 0, at["m"] or None, at["v"] or None, at.get("m_scale"),
                                     at.get("v_scale"), at["step"])

    def bind(self, grads) -> None:
        """Takes these gradients from now on (writes the device table on the current stream). The params may lie
        elsewhere than before, in the shapes that they had: the states stay what they are. It checks every tensor and
        launches once for 48 of them: 0.6 ms on the host for 256 params with shadows, where a step takes 0.04,
        so a loop keeps its gradients' buffers where it can."""
        self._bind(grads)
        self._mark()

    def _bind(self, grads) -> None:
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} grads for {len(self.params)} params")
        tensors, spans, dev = (LoraAdamwTensor * len(grads))(), [], self.device
        for i, (p, g, s, shape) in enumerate(zip(self.params, grads, self.shadows, self._shapes)):
            if p.shape != shape:
                raise ValueError(f"param {i} has become {tuple(p.shape)}: its states are those of {tuple(shape)}")
            for name, t in (("param", p), ("grad", g), ("shadow", s)):
                if t is None and name == "shadow":
                    continue
                if t.device != dev or not t.is_contiguous() or t.shape != shape:
                    raise ValueError(f"{name} {i} must be contiguous on {dev} in its param's shape {tuple(shape)}, "
                                     f"got {tuple(t.shape)} on {t.device}")
            if s is not None and s.dtype is not torch.bfloat16:
                raise ValueError(f"shadow {i} must be bfloat16, got {s.dtype}")
            at, copy, n = p.data_ptr(), 0 if s is None else s.data_ptr(), p.numel()
            if n:
                spans.append((at, at + n * p.element_size()))
            if n and copy:
                spans.append((copy, copy + 2 * n))
            tensors[i] = LoraAdamwTensor(at or None, g.data_ptr() or None, copy or None, n, _dtype_code(p),
                                         _dtype_code(g))
        spans.sort()
        if any(end > start for (_, end), (start, _) in zip(spans, spans[1:])):
            raise ValueError("params and shadows share memory: each element can be updated once in a step")
        need = self._lib.lora_adamw_table_bytes(tensors, len(grads))
        table = torch.empty(max(need, 1), dtype=torch.uint8, device=self.device)
        check("lora_adamw_table", self._lib.lora_adamw_table(tensors, len(grads), table.data_ptr(), need,
                                                             _queue(self.device)))
        if self._captured:  # a graph holds the addresses of what is replaced here
            self._kept.append((self._table, self._held))
            self._captured = False
        self.grads, self._tensors, self._table, self._table_bytes = grads, tensors, table, need
        self._held = self.params + grads + [s for s in self.shadows if s is not None]
        self._addresses = list(map(_data_ptr, self._held))

    def _mark(self) -> None:
        """The current stream has written the table and the states: steps elsewhere wait for it."""
        stream = _queue(self.device)
        self._streams = {stream.value}
        # in a capture there is nothing to wait for: the graph writes them when it runs
        self._written = not _capturing(stream)
        if self._written:
            self._event.record(torch.cuda.current_stream(self.device))
        else:
            self._captured = True

    def _admit(self, stream) -> None:
        """The first step on `stream`, the current one, since it was written elsewhere: the memory that the object
        allocated there is not given away before this stream is done with it."""
        current = torch.cuda.current_stream(self.device)
        if self._written:
            current.wait_event(self._event)
        for t in (self._table, *self.state.values()):
            t.record_stream(current)
        self._streams.add(stream.value)

    def step(self, lr_scale: torch.Tensor | None = None, grad_scale: torch.Tensor | None = None) -> None:
        """One step on the current stream. lr_scale, grad_scale: None or float32 [] tensors on the device that
        multiply lr and every gradient (a schedule, a clipping factor; read when the step runs)."""
        if list(map(_data_ptr, self._held)) != self._addresses:
            raise ValueError("a bound tensor's memory moved: bind the gradients again")
        if any(self.state[k].data_ptr() != a for k, a in self._addresses_of_state.items()):
            raise ValueError("a state tensor was replaced: copy into it instead")
        dev = self.device
        stream = _queue(dev)
        if _capturing(stream):
            self._captured = True
        elif stream.value not in self._streams:
            self._admit(stream)
        hyper = pack_hyper(self.lr, self.betas[0], self.betas[1], self.eps, self.weight_decay,
                           0 if lr_scale is None else _vector("lr_scale", lr_scale, 1, _F32, dev),
                           0 if grad_scale is None else _vector("grad_scale", grad_scale, 1, _F32, dev))
        check("lora_adamw_step", self._lib.lora_adamw_step(self._tensors, len(self.params), self._table.data_ptr(),
                                                           self._table_bytes, ctypes.byref(self._state),
                                                           hyper, stream))
