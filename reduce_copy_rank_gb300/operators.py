"""Operators of language models beside the collectives: log probabilities over
vocabulary shards and their gradient, the paged key-value cache and the
attention of single new tokens over it.

A thin binding like the rest of the package: tensors become pointers, sizes
and strides in the argument blocks of ``include/dc.h`` (read by the extension
module ``_binding``, whose checks raise ``ValueError``), and the work runs in
the library's CUDA kernels, one launch a call.  A row's or a sequence's
result depends on nothing else in the call: the same bits in a batch of one
and of a thousand, and, for the log probabilities, under every sharding.
What a call has written counts as changed in place: where autograd had kept
those numbers for a gradient, that gradient raises.
"""
from __future__ import annotations

import array
import ctypes
import struct
from typing import Sequence

import reduce_copy_rank_gb300 as _dc

MAX_TOP = 32
MAX_VOCAB = 1 << 22
ATTENTION_DIMS = (64, 96, 128, 192, 256)


class _Block:
    """The layout of an argument block of include/dc.h."""

    def __init__(self, layout: str, names: str):
        self.pack = struct.Struct("@" + layout).pack
        self.names = names.split()

    def of(self, fields: dict) -> bytes:
        unknown = set(fields) - set(self.names)
        if unknown:
            raise TypeError(f"unknown argument(s): {sorted(unknown)}")
        return self.pack(*(fields.get(n, 0) for n in self.names))


_SCORE = _Block("9Q2qd6i", "shards widths row_strides tokens logprobs entropy lse top_logprobs top_tokens "
                           "rows vocab temperature ranks dtype tokens_64 top_tokens_64 top reserved")
_GRAD = _Block("10Q2qd4i", "shards widths row_strides grads grad_row_strides tokens lse entropy grad_logprobs "
                           "grad_entropy rows vocab temperature ranks dtype tokens_64 reserved")
_CACHES = "k_cache k_page_stride k_slot_stride k_cache_head_stride v_cache v_page_stride v_slot_stride " \
          "v_cache_head_stride "
_APPEND = _Block("24Q6q8i", "q k v q_out positions seqs page_table cos_sin " + _CACHES +
                 "q_token_stride q_head_stride k_token_stride k_head_stride v_token_stride v_head_stride "
                 "q_out_token_stride q_out_head_stride tokens table_rows table_width table_stride cos_sin_rows "
                 "num_pages page_size q_heads kv_heads dim rotary_dim interleaved dtype reserved")
_ATTEND = _Block("19Q4q6ifi", "q out lse page_table lengths workspace workspace_bytes " + _CACHES +
                 "q_seq_stride q_head_stride out_seq_stride out_head_stride seqs table_width table_stride num_pages "
                 "page_size q_heads kv_heads dim window dtype scale reserved")

_HEAD = "hidden weights widths weight_row_strides tokens "
_LINEAR = _Block("11Q3qd4i", _HEAD + "logprobs entropy lse workspace workspace_bytes hidden_row_stride rows hidden_size "
                 "vocab temperature ranks dtype tokens_64 reserved")
_LINEAR_GRAD = _Block("16Q3qd4i", _HEAD + "lse entropy grad_logprobs grad_entropy grad_hidden grad_weights "
                      "grad_weight_row_strides workspace workspace_bytes hidden_row_stride grad_hidden_row_stride rows "
                      "hidden_size vocab temperature ranks dtype tokens_64 reserved")

_APPEND_NORM = _Block("24Q6q8i2Qfi", " ".join(_APPEND.names) + " q_norm k_norm eps norm_32")


def _heads(*names):
    return " ".join(f"{n} {n}_token_stride {n}_head_stride" for n in names)


_NORM = _Block("16Q2q7if", _heads("q", "k", "q_out", "k_out") + " positions cos_sin q_norm k_norm tokens cos_sin_rows q_heads "
               "kv_heads dim rotary_dim interleaved dtype norm_32 eps")
_NORM_GRAD = _Block("26Q2q7if", _heads("q", "k", "grad_q_out", "grad_k_out", "grad_q", "grad_k") + " positions cos_sin q_norm "
                    "k_norm grad_q_norm grad_k_norm workspace workspace_bytes tokens cos_sin_rows q_heads kv_heads dim "
                    "rotary_dim interleaved dtype norm_32 eps")

_PREFIX = _Block("19Q4q6ifi2Q3q", " ".join(_ATTEND.names) + " prefix_table prefix_lengths prefixes prefix_table_width "
                 "prefix_table_stride")

# the entry points, as the extension module takes them
_ENTRIES = ("dc_token_logprobs", "dc_token_logprobs_backward", "dc_kv_append", "dc_paged_attention",
            "dc_linear_logprobs", "dc_linear_logprobs_backward", "dc_kv_append_norm", "dc_qk_norm_rotate",
            "dc_qk_norm_rotate_backward", "dc_prefix_attention")

_bound = None


def _lib():
    """The library with these functions' signatures set."""
    global _bound
    if _bound is None:
        L = _dc.lib()
        for f in _ENTRIES:
            getattr(L, f).argtypes = [ctypes.c_char_p, ctypes.c_void_p]
            getattr(L, f).restype = ctypes.c_int
        L.dc_attention_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                   ctypes.c_int64]
        L.dc_attention_workspace_bytes.restype = ctypes.c_size_t
        L.dc_prefix_attention_workspace_bytes.argtypes = [ctypes.c_int64] * 2 + [ctypes.c_int] * 3 + [ctypes.c_int64] * 2
        L.dc_prefix_attention_workspace_bytes.restype = ctypes.c_size_t
        L.dc_qk_norm_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]
        L.dc_qk_norm_workspace_bytes.restype = ctypes.c_size_t
        L.dc_linear_logprobs_workspace_bytes.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int]
        L.dc_linear_logprobs_workspace_bytes.restype = ctypes.c_size_t
        _bound = L
    return _bound


# ------------------------------------------------------------ raw (C ABI) ---
# The argument blocks of include/dc.h by field name (fields left out are 0;
# the caches' strides are k_page_stride, k_slot_stride, k_cache_head_stride and
# the same for v).  Pointers are ints; host arrays (shards, widths, strides)
# are passed as sequences.  They return the status instead of raising.

def _with_arrays(block: _Block, fields: dict, keep: list) -> bytes:
    f = dict(fields)
    for name in ("shards", "widths", "row_strides", "grads", "grad_row_strides", "weights", "weight_row_strides",
                 "grad_weights", "grad_weight_row_strides"):
        if name in f and not isinstance(f[name], int):
            keep.append(array.array("Q", f[name]))
            f[name] = keep[-1].buffer_info()[0]
    return block.of(f)


def dc_token_logprobs(stream: int = 0, **fields) -> int:
    keep = []
    return _lib().dc_token_logprobs(_with_arrays(_SCORE, fields, keep), stream)


def dc_token_logprobs_backward(stream: int = 0, **fields) -> int:
    keep = []
    return _lib().dc_token_logprobs_backward(_with_arrays(_GRAD, fields, keep), stream)


def dc_kv_append(stream: int = 0, **fields) -> int:
    return _lib().dc_kv_append(_APPEND.of(fields), stream)


def dc_paged_attention(stream: int = 0, **fields) -> int:
    return _lib().dc_paged_attention(_ATTEND.of(fields), stream)


def dc_attention_workspace_bytes(seqs: int, q_heads: int, kv_heads: int, dim: int, max_tokens: int) -> int:
    return int(_lib().dc_attention_workspace_bytes(seqs, q_heads, kv_heads, dim, max_tokens))


def dc_linear_logprobs(stream: int = 0, **fields) -> int:
    keep = []
    return _lib().dc_linear_logprobs(_with_arrays(_LINEAR, fields, keep), stream)


def dc_linear_logprobs_backward(stream: int = 0, **fields) -> int:
    keep = []
    return _lib().dc_linear_logprobs_backward(_with_arrays(_LINEAR_GRAD, fields, keep), stream)


def dc_linear_logprobs_workspace_bytes(rows: int, hidden_size: int, columns: int, backward: bool) -> int:
    return int(_lib().dc_linear_logprobs_workspace_bytes(rows, hidden_size, columns, int(backward)))


def dc_kv_append_norm(stream: int = 0, **fields) -> int:
    return _lib().dc_kv_append_norm(_APPEND_NORM.of(fields), stream)


def dc_qk_norm_rotate(stream: int = 0, **fields) -> int:
    return _lib().dc_qk_norm_rotate(_NORM.of(fields), stream)


def dc_qk_norm_rotate_backward(stream: int = 0, **fields) -> int:
    return _lib().dc_qk_norm_rotate_backward(_NORM_GRAD.of(fields), stream)


def dc_qk_norm_workspace_bytes(tokens: int, q_heads: int, kv_heads: int, dim: int) -> int:
    return int(_lib().dc_qk_norm_workspace_bytes(tokens, q_heads, kv_heads, dim))


def dc_prefix_attention(stream: int = 0, **fields) -> int:
    return _lib().dc_prefix_attention(_PREFIX.of(fields), stream)


def dc_prefix_attention_workspace_bytes(seqs: int, prefixes: int, q_heads: int, kv_heads: int, dim: int,
                                        max_prefix_tokens: int, max_tokens: int) -> int:
    return int(_lib().dc_prefix_attention_workspace_bytes(seqs, prefixes, q_heads, kv_heads, dim, max_prefix_tokens, max_tokens))


# ------------------------------------------------------------ tensor API ---

_module = None


def _binding():
    """The extension module that reads the tensors, bound to the library."""
    global _module
    if _module is None:
        L = _lib()
        import torch  # noqa: F401  (its libraries first)

        try:
            from . import _binding as module
        except ImportError as e:
            raise _dc.LibraryMissing(f"the extension module _binding cannot be loaded ({e}): build it with `python -m "
                                     "reduce_copy_rank_gb300._build` or __graft_entry__.build()") from e
        module.bind(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in _ENTRIES))
        _module = module
    return _module


# ------------------------------------------------------- log probabilities ---

def token_logprobs(shards: Sequence, tokens, logprobs, entropy=None, lse=None, top_logprobs=None, top_tokens=None,
                   vocab: int | None = None, temperature: float = 1.0, stream=None):
    """Log probabilities of given tokens under logits held as P vocabulary
    shards (``shards[r]``: [rows, columns of rank r], bfloat16, float16 or
    float32; any row stride), without gathering them.

    ``logprobs[i]`` (float32) receives the log probability of ``tokens[i]``
    (int32 or int64) under ``softmax(logits[i] / temperature)`` over the first
    ``vocab`` columns (default: all; later ones are padding).  Optional
    outputs: ``entropy`` and ``lse`` (the log of the normaliser), float32
    [rows]; ``top_logprobs`` (float32) and ``top_tokens`` (int32 or int64),
    [rows, k] with k <= 32: the k largest logits, ties to the lowest index.

    A negative token is not scored (its entry is 0), a token past the
    vocabulary gives NaN.  Logits of -inf have probability 0; a row of
    nothing else gives -inf.  Bits depend on the row alone: not on the other
    rows, the number of shards or where they are cut.  Returns ``logprobs``."""
    status = (_module or _binding()).token_logprobs(shards, tokens, logprobs, entropy, lse, top_logprobs, top_tokens, vocab,
                                                    temperature, stream)
    if status:
        _dc._check(status)
    return logprobs


def token_logprobs_backward(shards: Sequence, tokens, lse, grad_logprobs, grads: Sequence, entropy=None,
                            grad_entropy=None, vocab: int | None = None, temperature: float = 1.0, stream=None):
    """The gradient of :func:`token_logprobs` with respect to the logits:
    ``grads[r]`` (of ``shards[r]``'s shape and type; it may be ``shards[r]``
    itself) receives that of ``sum(grad_logprobs * logprobs + grad_entropy *
    entropy)``.  ``lse`` and ``entropy`` are the forward call's outputs
    (``entropy`` only with ``grad_entropy``); the upstream gradients are
    float32 [rows], either may be None.  Padding columns receive 0.  Returns
    ``grads``."""
    status = (_module or _binding()).token_logprobs_backward(shards, tokens, lse, grad_logprobs, grads, entropy,
                                                             grad_entropy, vocab, temperature, stream)
    if status:
        _dc._check(status)
    return grads


_function = None


def logprobs_and_entropy(shards: Sequence, tokens, vocab: int | None = None, temperature: float = 1.0):
    """``(logprobs, entropy)`` of :func:`token_logprobs` as new tensors that
    autograd differentiates with respect to every shard (through
    :func:`token_logprobs_backward`, which computes every shard's gradient,
    wanted or not), once: a second derivative raises."""
    global _function
    import torch

    if _function is None:
        class TokenLogprobs(torch.autograd.Function):
            @staticmethod
            def forward(ctx, tokens, vocab, temperature, *shards):
                rows = shards[0].shape[0]
                logprobs, entropy, lse = (torch.empty(rows, dtype=torch.float32, device=shards[0].device)
                                          for _ in range(3))
                token_logprobs(shards, tokens, logprobs, entropy=entropy, lse=lse, vocab=vocab, temperature=temperature)
                ctx.set_materialize_grads(False)  # an output that is not used has no upstream gradient to read
                ctx.save_for_backward(tokens, lse, entropy, *shards)
                ctx.vocab, ctx.temperature = vocab, temperature
                return logprobs, entropy

            @staticmethod
            def backward(ctx, g, h):
                tokens, lse, entropy, *shards = ctx.saved_tensors
                if g is None and h is None:
                    return (None,) * (3 + len(shards))
                grads = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in shards]
                # upstream gradients may be broadcast (a sum's is one number for all rows)
                g, h = (None if u is None else u.to(torch.float32).contiguous() for u in (g, h))
                token_logprobs_backward(shards, tokens, lse, g, grads, entropy=entropy, grad_entropy=h,
                                        vocab=ctx.vocab, temperature=ctx.temperature)
                if torch.is_grad_enabled():  # create_graph: the gradients leave a kernel, no graph holds them
                    grads = FirstDerivative.apply(len(grads), *grads, *shards, *(u for u in (g, h) if u is not None))
                return (None, None, None, *grads)

        class FirstDerivative(torch.autograd.Function):
            """The gradients, with the tensors that they depend on: their own derivative is refused."""

            @staticmethod
            def forward(ctx, count, *tensors):
                return tuple(t.detach() for t in tensors[:count])

            @staticmethod
            def backward(ctx, *_):
                raise RuntimeError("logprobs_and_entropy has no second derivative: its gradients cannot be differentiated")

        _function = TokenLogprobs
    return _function.apply(tokens, vocab, temperature, *shards)


# ------------------------------------ log probabilities from hidden rows ---

def linear_logprobs_workspace(rows: int, hidden_size: int, columns: int, backward: bool = False, device=None):
    """A workspace tensor for :func:`linear_logprobs` (``backward``: for
    :func:`linear_logprobs_backward`) with up to ``rows`` rows of
    ``hidden_size`` and shards of ``columns`` columns in all.  Its contents do
    not matter; calls that may run at the same time need one each."""
    import torch

    n = dc_linear_logprobs_workspace_bytes(rows, hidden_size, columns, backward)
    if n == 0:
        raise _dc.DCError(1, _dc.last_error() or "no such head")
    return torch.empty(n, dtype=torch.uint8, device=device if device is not None else "cuda")


def linear_logprobs(hidden, weights: Sequence, tokens, logprobs, workspace, entropy=None, lse=None,
                    vocab: int | None = None, temperature: float = 1.0, stream=None):
    """:func:`token_logprobs` of the logits ``hidden @ weights.T`` without
    keeping them: ``hidden`` [rows, hidden size], the head as P vocabulary
    shards ``weights[r]`` [columns of rank r, hidden size] (bfloat16 or
    float16; 16-byte aligned rows, a hidden size that is a multiple of 8).

    ``logprobs``, and where given ``entropy`` and ``lse`` (float32 [rows]), as
    there; the logits are binary32 sums and are not rounded.  ``workspace``:
    :func:`linear_logprobs_workspace`.

    A negative token is not scored (its entry is 0), a token past the
    vocabulary gives NaN.  A row's bits do not depend on the other rows, nor
    on the sharding where shards are multiples of 256 columns (the last one
    may be any).  Returns ``logprobs``."""
    status = (_module or _binding()).linear_logprobs(hidden, weights, tokens, logprobs, workspace, entropy, lse, vocab,
                                                     temperature, stream)
    if status:
        _dc._check(status)
    return logprobs


def linear_logprobs_backward(hidden, weights: Sequence, tokens, lse, grad_logprobs, grad_hidden, grad_weights,
                             workspace, entropy=None, grad_entropy=None, vocab: int | None = None,
                             temperature: float = 1.0, stream=None):
    """The gradient of :func:`linear_logprobs` with respect to the hidden rows
    and the head's weights: ``grad_hidden`` and ``grad_weights[r]`` (shaped and
    typed as ``hidden`` and ``weights[r]``; either may be None) receive that of
    ``sum(grad_logprobs * logprobs + grad_entropy * entropy)``.  ``lse`` and
    ``entropy`` are the forward call's outputs (``entropy`` only with
    ``grad_entropy``); the upstream gradients are float32 [rows], either may be
    None.

    The logits are computed again, up to 24576 columns at a time; their gradient is
    rounded to 16 bits before its products, but for the tokens' own elements; the
    sums are binary32, in an order that is fixed but, for the hidden rows' gradient,
    depends on the sharding.  Rows of the weights' gradient past ``vocab`` receive 0.
    A token past the vocabulary gives NaN.  A row without upstream gradients (padding) has none, but its hidden row has
    to be finite: the weights' gradient is a product with all of them.  ``workspace``:
    :func:`linear_logprobs_workspace` with ``backward``.  Returns
    ``(grad_hidden, grad_weights)``."""
    status = (_module or _binding()).linear_logprobs_backward(hidden, weights, tokens, lse, grad_logprobs, grad_hidden,
                                                              grad_weights, workspace, entropy, grad_entropy, vocab,
                                                              temperature, stream)
    if status:
        _dc._check(status)
    return grad_hidden, grad_weights


_linear_function = None


def linear_logprobs_and_entropy(hidden, weights: Sequence, tokens, vocab: int | None = None, temperature: float = 1.0):
    """``(logprobs, entropy)`` of :func:`linear_logprobs` as new tensors that
    autograd differentiates with respect to the hidden rows and every shard
    (through :func:`linear_logprobs_backward`), once: a second derivative
    raises.  Workspaces come from torch's allocator."""
    global _linear_function
    import torch

    if _linear_function is None:
        class LinearLogprobs(torch.autograd.Function):
            @staticmethod
            def forward(ctx, tokens, vocab, temperature, hidden, *weights):
                rows, size = hidden.shape
                logprobs, entropy, lse = (torch.empty(rows, dtype=torch.float32, device=hidden.device) for _ in range(3))
                ws = linear_logprobs_workspace(rows, size, sum(w.shape[0] for w in weights), device=hidden.device)
                linear_logprobs(hidden, weights, tokens, logprobs, ws, entropy=entropy, lse=lse, vocab=vocab,
                                temperature=temperature)
                ctx.set_materialize_grads(False)  # an output that is not used has no upstream gradient to read
                ctx.save_for_backward(tokens, lse, entropy, hidden, *weights)
                ctx.vocab, ctx.temperature = vocab, temperature
                return logprobs, entropy

            @staticmethod
            def backward(ctx, g, h):
                tokens, lse, entropy, hidden, *weights = ctx.saved_tensors
                want_hidden, want_weights = ctx.needs_input_grad[3], any(ctx.needs_input_grad[4:])
                if (g is None and h is None) or not (want_hidden or want_weights):
                    return (None,) * (4 + len(weights))
                grad_hidden = torch.empty_like(hidden, memory_format=torch.contiguous_format) if want_hidden else None
                grads = [torch.empty_like(w, memory_format=torch.contiguous_format) for w in weights] if want_weights else None
                # upstream gradients may be broadcast (a sum's is one number for all rows)
                g, h = (None if u is None else u.to(torch.float32).contiguous() for u in (g, h))
                ws = linear_logprobs_workspace(*hidden.shape, sum(w.shape[0] for w in weights), backward=True,
                                               device=hidden.device)
                linear_logprobs_backward(hidden, weights, tokens, lse, g, grad_hidden, grads, ws, entropy=entropy,
                                         grad_entropy=h, vocab=ctx.vocab, temperature=ctx.temperature)
                out = [x for x in (grad_hidden, *(grads or ())) if x is not None]
                if torch.is_grad_enabled():  # create_graph: the gradients leave a kernel, no graph holds them
                    out = list(_first_derivative("linear_logprobs_and_entropy").apply(
                        len(out), *out, hidden, *weights, *(u for u in (g, h) if u is not None)))
                grad_hidden = out.pop(0) if want_hidden else None
                return (None, None, None, grad_hidden, *(out if want_weights else (None,) * len(weights)))

        _linear_function = LinearLogprobs
    return _linear_function.apply(tokens, vocab, temperature, hidden, *weights)


def _aligned(t):
    """`t`, or a copy of it where it does not start at a multiple of 16 bytes."""
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _first_derivative(name: str):
    """A function that passes gradients on with the tensors that they depend on: their own derivative is refused."""
    import torch

    class FirstDerivative(torch.autograd.Function):
        @staticmethod
        def forward(ctx, count, *tensors):
            return tuple(t.detach() for t in tensors[:count])

        @staticmethod
        def backward(ctx, *_):
            raise RuntimeError(f"{name} has no second derivative: its gradients cannot be differentiated")

    return FirstDerivative


# ------------------------------------------------------------ paged cache ---

def kv_append(k, v, positions, seqs, page_table, k_cache, v_cache, q=None, q_out=None, cos_sin=None,
              interleaved: bool = False, stream=None, q_norm=None, k_norm=None, eps: float = 1e-6):
    """Puts the keys and values of new tokens ([tokens, kv_heads, dim]) into a
    paged cache ([pages, page_size, kv_heads, dim] tensors, or views of that
    shape with any strides), rotating the keys, and the queries ``q`` into
    ``q_out`` ([tokens, q_heads, dim]; ``q_out`` may be ``q``), to their
    positions.  Token i of sequence ``seqs[i]`` at ``positions[i]`` (int32)
    goes to slot ``positions[i] % page_size`` of page ``page_table[seqs[i],
    positions[i] // page_size]`` (int32).

    ``cos_sin`` (float32 [positions, rotary_dim]): the cosines of a position's
    rotary_dim/2 angles, then their sines; None: no rotation.  Pair j is
    elements j and j + rotary_dim/2, or 2j and 2j + 1 if ``interleaved``;
    elements past rotary_dim stay.

    ``k_norm`` (and ``q_norm`` where there are queries; [dim], float32 or the
    heads' type): keys and queries are normed per head before they are rotated,
    ``x * w / sqrt(mean(x * x) + eps)`` (dim up to 512).

    A negative position is padding and writes nothing.  A token whose
    sequence, position or page does not exist writes no cache; its queries
    become NaN.  Returns ``q_out``."""
    if q_norm is None and k_norm is None:
        status = (_module or _binding()).kv_append(k, v, positions, seqs, page_table, k_cache, v_cache, q, q_out, cos_sin,
                                                   interleaved, stream)
    else:
        status = (_module or _binding()).kv_append_norm(k, v, positions, seqs, page_table, k_cache, v_cache, q, q_out,
                                                        cos_sin, interleaved, stream, q_norm, k_norm, eps)
    if status:
        _dc._check(status)
    return q_out


def qk_norm_rotate(q, k, positions, cos_sin, q_norm, k_norm, q_out, k_out, eps: float = 1e-6, interleaved: bool = False,
                   stream=None):
    """The queries and keys ([tokens, heads, dim]; bfloat16, float16 or
    float32) of a training step, normed per head and rotated to ``positions``
    (int32 [tokens]) into ``q_out`` and ``k_out``, with the bits that
    :func:`kv_append` gives with ``q_norm`` and ``k_norm``; ``cos_sin`` and
    ``interleaved`` as there, dim up to 512.

    A negative position is padding: its rows are 0.  A position past
    ``cos_sin`` gives NaN.  Returns ``(q_out, k_out)``, which may be exactly
    ``q`` and ``k``."""
    status = (_module or _binding()).qk_norm_rotate(q, k, positions, cos_sin, q_norm, k_norm, q_out, k_out, eps, interleaved,
                                                    stream)
    if status:
        _dc._check(status)
    return q_out, k_out


def qk_norm_workspace(tokens: int, q_heads: int, kv_heads: int, dim: int, device=None):
    """A workspace tensor for :func:`qk_norm_rotate_backward`; its contents do
    not matter, and calls that may run at the same time need one each."""
    import torch

    n = dc_qk_norm_workspace_bytes(tokens, q_heads, kv_heads, dim)
    if n == 0:
        raise _dc.DCError(1, _dc.last_error() or "no such heads")
    return torch.empty(n, dtype=torch.uint8, device=device if device is not None else "cuda")


def qk_norm_rotate_backward(q, k, positions, cos_sin, q_norm, k_norm, grad_q_out, grad_k_out, grad_q, grad_k,
                            grad_q_norm=None, grad_k_norm=None, workspace=None, eps: float = 1e-6,
                            interleaved: bool = False, stream=None):
    """The gradient of :func:`qk_norm_rotate`: ``grad_q`` and ``grad_k``
    (which may be exactly ``grad_q_out`` and ``grad_k_out``), and, where given,
    those of the weights (typed as the weights; they need ``workspace``:
    :func:`qk_norm_workspace`), summed in binary32 in one fixed order.
    Padding has no gradient.  Returns ``(grad_q, grad_k)``."""
    status = (_module or _binding()).qk_norm_rotate_backward(q, k, positions, cos_sin, q_norm, k_norm, grad_q_out, grad_k_out,
                                                             grad_q, grad_k, grad_q_norm, grad_k_norm, workspace, eps,
                                                             interleaved, stream)
    if status:
        _dc._check(status)
    return grad_q, grad_k


_norm_function = None


def normed_queries_and_keys(q, k, positions, cos_sin, q_norm, k_norm, eps: float = 1e-6, interleaved: bool = False):
    """``(q_out, k_out)`` of :func:`qk_norm_rotate` as new tensors that
    autograd differentiates with respect to ``q``, ``k``, ``q_norm`` and
    ``k_norm`` (through :func:`qk_norm_rotate_backward`), once: a second
    derivative raises."""
    global _norm_function
    import torch

    if _norm_function is None:
        class NormRotate(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, q_norm, k_norm, positions, cos_sin, eps, interleaved):
                outs = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k)]
                qk_norm_rotate(q, k, positions, cos_sin, q_norm, k_norm, *outs, eps=eps, interleaved=interleaved)
                ctx.save_for_backward(q, k, q_norm, k_norm, positions, *([] if cos_sin is None else [cos_sin]))
                ctx.eps, ctx.interleaved = eps, interleaved
                return tuple(outs)

            @staticmethod
            def backward(ctx, gq, gk):
                q, k, q_norm, k_norm, positions, *rest = ctx.saved_tensors
                cos_sin = rest[0] if rest else None
                # upstream gradients may be broadcast, or laid out in a way that the kernel does not read
                gq, gk = (_aligned(g.to(t.dtype).contiguous()) for g, t in zip((gq, gk), (q, k)))
                grads = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k)]
                want = any(ctx.needs_input_grad[2:4])
                sums = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q_norm, k_norm)] if want else [None] * 2
                ws = qk_norm_workspace(q.shape[0], q.shape[1], k.shape[1], q.shape[2], q.device) if want else None
                qk_norm_rotate_backward(q, k, positions, cos_sin, q_norm, k_norm, gq, gk, *grads, *sums, workspace=ws,
                                        eps=ctx.eps, interleaved=ctx.interleaved)
                out = [g for g in (*grads, *sums) if g is not None]
                if torch.is_grad_enabled():  # create_graph: the gradients leave a kernel, no graph holds them
                    out = list(_first_derivative("normed_queries_and_keys").apply(len(out), *out, q, k, q_norm, k_norm, gq, gk))
                return (*out, *(() if want else (None, None)), None, None, None, None)

        _norm_function = NormRotate
    return _norm_function.apply(q, k, q_norm, k_norm, positions, cos_sin, eps, interleaved)


def attention_workspace(seqs: int, q_heads: int, kv_heads: int, dim: int, max_tokens: int, device=None):
    """A zeroed workspace tensor for :func:`paged_attention` with up to
    ``seqs`` sequences and page tables of up to ``max_tokens`` tokens a row
    (allocated by torch; the library itself allocates nothing).  Keep it: a
    call leaves it, and any part of it that starts where it does, ready for
    the next.  One workspace per stream."""
    import torch

    n = dc_attention_workspace_bytes(seqs, q_heads, kv_heads, dim, max_tokens)
    if n == 0:
        raise _dc.DCError(1, _dc.last_error() or "no such attention")
    return torch.zeros(n, dtype=torch.uint8, device=device if device is not None else "cuda")


def paged_attention(q, k_cache, v_cache, page_table, lengths, out, workspace, scale: float | None = None,
                    window: int = 0, lse=None, stream=None):
    """Attention of one new token per sequence over a paged cache.

    ``q``, ``out``: [sequences, q_heads, dim] (bfloat16 or float16; dim 64,
    96, 128, 192 or 256); caches as in :func:`kv_append`, q_heads a multiple
    of kv_heads; ``page_table`` int32 [sequences, pages], ``lengths`` int32
    [sequences]: sequence b attends to its first ``lengths[b]`` tokens, or to
    the last ``window`` of them.  ``scale``: default ``dim ** -0.5``.  ``lse``
    (float32 [sequences, q_heads]) receives the log of the normaliser, with
    which results over parts of a context can be joined.

    A length of 0 gives zeros (lse -inf).  A page number outside the cache, or
    a length past the table, gives NaN.  ``workspace``: see
    :func:`attention_workspace`.  Returns ``out``."""
    status = (_module or _binding()).paged_attention(q, k_cache, v_cache, page_table, lengths, out, workspace, scale, window,
                                                     lse, stream)
    if status:
        _dc._check(status)
    return out


def prefix_attention_workspace(seqs: int, prefixes: int, q_heads: int, kv_heads: int, dim: int, max_prefix_tokens: int,
                               max_tokens: int, device=None):
    """A zeroed workspace tensor for :func:`prefix_attention` with ``seqs``
    sequences behind ``prefixes`` prefixes, prefix tables of up to
    ``max_prefix_tokens`` and page tables of up to ``max_tokens`` tokens a row.
    Keep it: a call leaves it ready for the next.  One workspace per stream."""
    import torch

    n = dc_prefix_attention_workspace_bytes(seqs, prefixes, q_heads, kv_heads, dim, max_prefix_tokens, max_tokens)
    if n == 0:
        raise _dc.DCError(1, _dc.last_error() or "no such attention")
    return torch.zeros(n, dtype=torch.uint8, device=device if device is not None else "cuda")


def prefix_attention(q, k_cache, v_cache, prefix_table, prefix_lengths, page_table, lengths, out, workspace,
                     scale: float | None = None, lse=None, stream=None):
    """:func:`paged_attention` of sequences that share prefixes, whose keys and
    values are read once for all of a group: with P rows in ``prefix_table``
    (int32 [P, pages], pages of the same caches) sequences come in P groups of
    neighbours of one size, and a sequence attends to the first
    ``prefix_lengths[g]`` (int32 [P]) tokens of its group's prefix, then to its
    own ``lengths[b]`` tokens of ``page_table``.

    The other arguments are those of :func:`paged_attention` (no window).
    Either part may be empty; without any token the result is zeros (lse
    -inf).  A page number outside the cache, or a length past its table, gives
    NaN in the sequences that it belongs to.  A sequence's bits do not depend
    on the other sequences.  The prefix's weights are rounded to 16 bits before
    they meet the values, where :func:`paged_attention` rounds nothing but the
    output (error 2.4e-3 for 1.7e-3 in bfloat16, 2.9e-4 for 2.1e-4 in float16).
    ``workspace``: :func:`prefix_attention_workspace`.
    Returns ``out``."""
    status = (_module or _binding()).prefix_attention(q, k_cache, v_cache, page_table, lengths, out, workspace, scale, 0, lse,
                                                      stream, prefix_table, prefix_lengths)
    if status:
        _dc._check(status)
    return out
