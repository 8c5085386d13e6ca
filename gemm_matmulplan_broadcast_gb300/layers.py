"""Plans for the operators that stand around a language model's products
(marshalling only, over the same library as ``binding``).

    from gemm_matmulplan_broadcast_gb300 import LayerNormPlan

A plan is made for fixed sizes and one element type ("float32", "float16" or
"bfloat16"); its calls take CUDA tensors and outputs that the caller owns and
enqueue kernels on ``stream`` (torch's current stream by default).  Row
tensors are [rows, cols] (any leading dimensions when contiguous) with
unit-stride columns; a two-dimensional one may have any row pitch.  The
one-shot functions return memory of ``stream``, and read their inputs there:
where it is not torch's current stream, the two have to be ordered by the
caller (``wait_stream``), as for torch's own operators.
"""

from __future__ import annotations

import ctypes

from .binding import DTYPE_CODES, GATES, _check, _memory_of, _stream_handle, load

ROW_DTYPES = ("float32", "float16", "bfloat16")


def _torch_dtype(name: str):
    import torch
    if name not in ROW_DTYPES:
        raise ValueError("unsupported dtype %r" % (name,))
    return getattr(torch, name)


def _raw_stream(stream):
    """Handle of ``stream``, or of torch's current stream (by the call that
    makes no Stream object, where torch has it: one in five microseconds of a
    small call)."""
    if stream is None:
        import torch
        try:
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:
            pass
    return _stream_handle(stream)


def _rows(name, t, rows, cols, dtype):
    """Pointer and row pitch of a [rows, cols] tensor of the given type."""
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, the plan wants %s" % (name, t.dtype, dtype))
    shape = t.shape
    if cols and shape == (rows, cols) and t.is_cuda:      # the usual case
        pitch, unit = t.stride()
        if unit == 1 and pitch >= cols:
            return t.data_ptr(), pitch
    if not shape or shape[-1] != cols or t.numel() != rows * cols:
        raise ValueError("%s has shape %s, the plan wants [%d, %d]" % (name, tuple(shape), rows, cols))
    if t.numel() == 0:
        return None, cols
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.is_contiguous():
        return t.data_ptr(), cols
    if len(shape) != 2 or (cols > 1 and t.stride(1) != 1):
        raise ValueError("%s must be contiguous, or a matrix with unit-stride columns" % name)
    if rows > 1 and t.stride(0) < cols:
        raise ValueError("%s has overlapping rows" % name)
    return t.data_ptr(), t.stride(0)


def _flat(name, t, n, dtype):
    """Pointer of a contiguous tensor of n elements (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, the plan wants %s" % (name, t.dtype, dtype))
    if t.numel() != n:
        raise ValueError("%s has %d elements, the plan wants %d" % (name, t.numel(), n))
    if n == 0:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor" % name)
    return t.data_ptr()


def _dense(name, t, rows, cols, dtype):
    """Pointer of a contiguous [rows, cols] tensor (None stays None)."""
    if t is None:
        return None
    ptr, pitch = _rows(name, t, rows, cols, dtype)
    if rows > 1 and pitch != cols:
        raise ValueError("%s must be contiguous" % name)
    return ptr


class _PlanHandle:
    """Lifetime of a library plan: closed explicitly, by ``with``, or with
    the object."""

    _destroy = ""

    def _create(self, fn: str, *args):
        self.lib = load()
        h = ctypes.c_void_p()
        _check(getattr(self.lib, fn)(*args, ctypes.byref(h)), fn)
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            getattr(self.lib, self._destroy)(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class LayerNormPlan(_PlanHandle):
    """Layer norm over the last axis of [rows, cols]: y = (x - mean) * rstd *
    gamma + beta, and its gradients."""

    _destroy = "olc_layer_norm_plan_destroy"

    def __init__(self, rows: int, cols: int, dtype: str, eps: float = 1e-5):
        import torch
        self.rows, self.cols, self.dtype, self.eps = int(rows), int(cols), dtype, float(eps)
        self._t, self._f32 = _torch_dtype(dtype), torch.float32
        self._create("olc_layer_norm_plan_create", self.rows, self.cols, self.eps, DTYPE_CODES[dtype])

    def forward(self, X, gamma, beta, Y, mean=None, rstd=None, stream=None):
        """Y = layer norm of X.  gamma, beta: [cols] or None (ones, zeros);
        mean, rstd: float32 [rows] outputs for the backward call, or None."""
        rows, cols, t = self.rows, self.cols, self._t
        x, xp = _rows("X", X, rows, cols, t)
        y, yp = _rows("Y", Y, rows, cols, t)
        st = self.lib.olc_layer_norm_forward(
            self._h, x, xp, _flat("gamma", gamma, cols, t), _flat("beta", beta, cols, t), y, yp,
            _flat("mean", mean, rows, self._f32), _flat("rstd", rstd, rows, self._f32), _raw_stream(stream))
        _check(st, "olc_layer_norm_forward")
        return Y

    def backward(self, dY, X, gamma, mean, rstd, dX=None, dgamma=None, dbeta=None, stream=None):
        """The gradients of X, gamma and beta (each None to skip it) from dY
        and the forward call's mean and rstd."""
        rows, cols, t = self.rows, self.cols, self._t
        dy, dyp = _rows("dY", dY, rows, cols, t)
        x, xp = _rows("X", X, rows, cols, t)
        dx, dxp = (None, cols) if dX is None else _rows("dX", dX, rows, cols, t)
        st = self.lib.olc_layer_norm_backward(
            self._h, dy, dyp, x, xp, _flat("gamma", gamma, cols, t), _flat("mean", mean, rows, self._f32),
            _flat("rstd", rstd, rows, self._f32), dx, dxp, _flat("dgamma", dgamma, cols, t),
            _flat("dbeta", dbeta, cols, t), _raw_stream(stream))
        _check(st, "olc_layer_norm_backward")
        return dX, dgamma, dbeta


class GatedPlan(_PlanHandle):
    """The gated feed-forward product H = act(X Wg) * (X Wu) of X [rows,
    d_in] with Wg and Wu [d_in, d_hidden] (stored [d_hidden, d_in] with
    trans_w), and its gradients.  act: silu, gelu, relu or sigmoid."""

    _destroy = "olc_gated_plan_destroy"

    def __init__(self, rows: int, d_in: int, d_hidden: int, dtype: str, act: str = "silu", trans_w: bool = False):
        if act not in GATES:
            raise ValueError("act must be one of %s" % sorted(GATES))
        self.rows, self.d_in, self.d_hidden = int(rows), int(d_in), int(d_hidden)
        self.dtype, self.act, self.trans_w = dtype, act, bool(trans_w)
        self._t = _torch_dtype(dtype)
        self._w = (self.d_hidden, self.d_in) if self.trans_w else (self.d_in, self.d_hidden)
        self._create("olc_gated_plan_create", self.rows, self.d_in, self.d_hidden, GATES[act], int(self.trans_w),
                     DTYPE_CODES[dtype])

    def forward(self, X, Wg, Wu, H, G=None, U=None, stream=None):
        """H = act(X Wg) * (X Wu); G, U: the two products for the backward
        call, or None."""
        m, f, t, w = self.rows, self.d_hidden, self._t, self._w
        st = self.lib.olc_gated_forward(
            self._h, _dense("X", X, m, self.d_in, t), _dense("Wg", Wg, w[0], w[1], t),
            _dense("Wu", Wu, w[0], w[1], t), _dense("H", H, m, f, t), _dense("G", G, m, f, t),
            _dense("U", U, m, f, t), _raw_stream(stream))
        _check(st, "olc_gated_forward")
        return H

    def backward(self, dH, X, Wg, Wu, G, U, dX=None, dWg=None, dWu=None, stream=None):
        """The gradients of X (or None) and of both weights (or both None)
        from dH and the forward call's G and U."""
        m, d, f, t, w = self.rows, self.d_in, self.d_hidden, self._t, self._w
        st = self.lib.olc_gated_backward(
            self._h, _dense("dH", dH, m, f, t), _dense("X", X, m, d, t), _dense("Wg", Wg, w[0], w[1], t),
            _dense("Wu", Wu, w[0], w[1], t), _dense("G", G, m, f, t), _dense("U", U, m, f, t),
            _dense("dX", dX, m, d, t), _dense("dWg", dWg, w[0], w[1], t), _dense("dWu", dWu, w[0], w[1], t),
            _raw_stream(stream))
        _check(st, "olc_gated_backward")
        return dX, dWg, dWu


class TokenLogProbsPlan(_PlanHandle):
    """Log probabilities of given tokens from logits [rows, vocab], with the
    entropy and the ``top`` most likely tokens of each row, and the gradient
    of both."""

    _destroy = "olc_token_log_probs_plan_destroy"

    def __init__(self, rows: int, vocab: int, dtype: str, top: int = 0):
        import torch
        self.rows, self.vocab, self.dtype, self.top = int(rows), int(vocab), dtype, int(top)
        self._t, self._f32, self._i64 = _torch_dtype(dtype), torch.float32, torch.int64
        self._create("olc_token_log_probs_plan_create", self.rows, self.vocab, self.top, DTYPE_CODES[dtype])

    def forward(self, logits, tokens, logprob, entropy=None, lse=None, top_logprob=None, top_index=None, stream=None):
        """logprob[r] = log softmax(logits[r])[tokens[r]] (tokens: int64; a
        negative one marks a row to ignore).  entropy, lse: float32 [rows];
        top_logprob (float32), top_index (int64): [rows, top]; each may be
        None."""
        rows, f32 = self.rows, self._f32
        z, pitch = _rows("logits", logits, rows, self.vocab, self._t)
        n = rows * self.top
        st = self.lib.olc_token_log_probs_forward(
            self._h, z, pitch, _flat("tokens", tokens, rows, self._i64), _flat("logprob", logprob, rows, f32),
            _flat("entropy", entropy, rows, f32), _flat("lse", lse, rows, f32),
            _flat("top_logprob", top_logprob, n, f32), _flat("top_index", top_index, n, self._i64),
            _raw_stream(stream))
        _check(st, "olc_token_log_probs_forward")
        return logprob

    def backward(self, logits, tokens, lse, entropy, dlogprob, dlogits, dentropy=None, stream=None):
        """dlogits from the gradients of logprob and entropy (either None for
        zeros) and the forward call's lse and entropy."""
        rows, f32 = self.rows, self._f32
        z, pitch = _rows("logits", logits, rows, self.vocab, self._t)
        dz, d_pitch = _rows("dlogits", dlogits, rows, self.vocab, self._t)
        st = self.lib.olc_token_log_probs_backward(
            self._h, z, pitch, _flat("tokens", tokens, rows, self._i64), _flat("lse", lse, rows, f32),
            _flat("entropy", entropy, rows, f32), _flat("dlogprob", dlogprob, rows, f32),
            _flat("dentropy", dentropy, rows, f32), dz, d_pitch, _raw_stream(stream))
        _check(st, "olc_token_log_probs_backward")
        return dlogits


def layer_norm(X, gamma=None, beta=None, eps: float = 1e-5, out=None, stream=None):
    """Layer norm of a CUDA tensor over its last axis through a fresh plan."""
    import torch
    if out is None:
        with _memory_of(stream):
            out = torch.empty_like(X, memory_format=torch.contiguous_format)
    cols = X.shape[-1] if X.dim() else 0
    rows = X.numel() // cols if cols else 0
    with LayerNormPlan(rows, cols, str(X.dtype).replace("torch.", ""), eps) as plan:
        return plan.forward(X, gamma, beta, out, stream=stream)


def gated(X, Wg, Wu, act: str = "silu", trans_w: bool = False, out=None, stream=None):
    """act(X Wg) * (X Wu) of CUDA tensors through a fresh plan."""
    import torch
    d, f = reversed(Wg.shape) if trans_w else Wg.shape
    if out is None:
        with _memory_of(stream):
            out = torch.empty(X.shape[:-1] + (f,), dtype=X.dtype, device=X.device)
    with GatedPlan(X.shape[:-1].numel(), d, f, str(X.dtype).replace("torch.", ""), act, trans_w) as plan:
        return plan.forward(X, Wg, Wu, out, stream=stream)


def token_log_probs(logits, tokens, top: int = 0, stream=None):
    """(logprob, entropy) of CUDA logits [rows, vocab], or (logprob, entropy,
    top_logprob, top_index), through a fresh plan."""
    import torch
    rows, vocab = logits.shape
    make = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=logits.device)  # noqa: E731
    with _memory_of(stream):
        logprob, entropy = make(rows), make(rows)
        best = (make(rows, top), make(rows, top, dtype=torch.int64)) if top else (None, None)
    with TokenLogProbsPlan(rows, vocab, str(logits.dtype).replace("torch.", ""), top) as plan:
        plan.forward(logits, tokens, logprob, entropy=entropy, top_logprob=best[0], top_index=best[1], stream=stream)
    return (logprob, entropy) + (best if top else ())
