"""Tokens from logits and their probabilities: mk_sample and mk_logprobs (include/mk.h), and a decode loop that samples.

`sample` and `logprobs` are the operators; `SampledLoop` runs a loaded model
with them, one token a sequence and step, every step on the device.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import LogprobStruct, MKError, SamplingStruct, _check, lib
from .pages import _DTYPE, _launch, _ptr

_SAMPLING = struct.Struct("Pq PPPPP PPP iiii")
_LOGPROB = struct.Struct("Pq PPPPPP iiiiii")
assert _SAMPLING.size == ctypes.sizeof(SamplingStruct) and _LOGPROB.size == ctypes.sizeof(LogprobStruct)


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None, return_details=False,
           stream=None):
    """One token a row of `logits` ([rows, vocab], float32, bfloat16 or float16) with the random numbers u (float32
    [rows], in [0, 1)).

    temperature, top_p, min_p: float32 [rows]; top_k: int32 [rows]; each may be None (1, no top-p, no min-p, no
    top-k). The filters apply in the order top-k, top-p, min-p; temperature <= 0 takes the largest logit. -inf masks
    a token; a row with a NaN, +inf or no unmasked token gives -1. Returns int32 tokens [rows] (`out`, when given),
    with return_details (tokens, the token's probability among the kept ones, how many were kept)."""
    dt = _DTYPE.get(logits.dtype)
    if dt is None or logits.dim() != 2 or not logits.is_cuda or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be a float32, bfloat16 or float16 CUDA tensor [rows, vocab] with contiguous rows, "
                         f"got {logits.dtype} {tuple(logits.shape)} strides {logits.stride()} on {logits.device}")
    R, V = logits.shape
    dev, n = logits.device, logits.shape[:1]
    if u is None:
        raise ValueError("u is required")
    args = (_ptr(u, "u", n, torch.float32, dev),
            0 if temperature is None else _ptr(temperature, "temperature", n, torch.float32, dev),
            0 if top_k is None else _ptr(top_k, "top_k", n, torch.int32, dev),
            0 if top_p is None else _ptr(top_p, "top_p", n, torch.float32, dev),
            0 if min_p is None else _ptr(min_p, "min_p", n, torch.float32, dev))
    if out is not None:
        _ptr(out, "out", n, torch.int32, dev)
    return _launch(dev, stream, _sample, (logits, args, out, return_details, n, R, V, dt))


def _sample(h, logits, args, out, details, n, R, V, dt):
    dev = logits.device
    tokens = torch.empty(n, dtype=torch.int32, device=dev) if out is None else out
    probs = torch.empty(n, dtype=torch.float32, device=dev) if details else None
    kept = torch.empty(n, dtype=torch.int32, device=dev) if details else None
    if R:
        a = _SAMPLING.pack(logits.data_ptr(), logits.stride(0), *args, tokens.data_ptr(),
                           probs.data_ptr() if details else 0, kept.data_ptr() if details else 0, R, V, dt, 0)
        rc = lib().mk_sample(a, h)
        if rc:
            _check(rc)
    return (tokens, probs, kept) if details else tokens


def logprobs(logits, tokens, top=0, temperature=None, stream=None):
    """Log probabilities of given tokens under `logits` ([rows, vocab], float32, bfloat16 or float16), divided by
    `temperature` (float32 [rows]) when given.

    tokens: int32 [rows] or [rows, given], or None; top: how many of the most probable tokens to name (at most 64).
    Returns (log probabilities, float32 shaped as tokens, or None; entropies, float32 [rows]; the top tokens, int32
    [rows, top], by descending logit, the lower id first where logits are equal; their log probabilities, float32
    [rows, top]). An id outside the vocabulary gets NaN. -inf masks a token; a row with a NaN, +inf, no unmasked token
    or a temperature that is not above 2^-120 gives NaN throughout, and ids -1."""
    dt = _DTYPE.get(logits.dtype)
    if dt is None or logits.dim() != 2 or not logits.is_cuda or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be a float32, bfloat16 or float16 CUDA tensor [rows, vocab] with contiguous rows, "
                         f"got {logits.dtype} {tuple(logits.shape)} strides {logits.stride()} on {logits.device}")
    dev, n = logits.device, logits.shape[:1]
    given = 0
    if tokens is not None:
        if tokens.dim() not in (1, 2):
            raise ValueError(f"tokens must be [rows] or [rows, given], got {tuple(tokens.shape)}")
        _ptr(tokens, "tokens", n + tokens.shape[1:], torch.int32, dev)
        given = tokens.shape[1] if tokens.dim() == 2 else 1
    t = 0 if temperature is None else _ptr(temperature, "temperature", n, torch.float32, dev)
    if not 0 <= top <= logits.shape[1]:
        raise ValueError(f"top must be between 0 and the vocabulary's {logits.shape[1]}, got {top}")
    return _launch(dev, stream, _logprobs, (logits, tokens, given, top, t, dt))


def _logprobs(h, logits, tokens, given, top, t, dt):
    dev, (R, V) = logits.device, logits.shape
    out = None if tokens is None else torch.empty(tokens.shape, dtype=torch.float32, device=dev)
    entropy = torch.empty((R,), dtype=torch.float32, device=dev)
    ids = torch.empty((R, top), dtype=torch.int32, device=dev)
    best = torch.empty((R, top), dtype=torch.float32, device=dev)
    if R:
        a = _LOGPROB.pack(logits.data_ptr(), logits.stride(0), t, tokens.data_ptr() if given else 0,
                          out.data_ptr() if given else 0, entropy.data_ptr(), ids.data_ptr() if top else 0,
                          best.data_ptr() if top else 0, R, V, dt, given, top, 0)
        rc = lib().mk_logprobs(a, h)
        if rc:
            _check(rc)
    return out, entropy, ids, best


class SampledLoop:
    """Sampled decoding of `batch` sequences, one token each a step.

    model, kv: a loaded `Model` and its `KVCache`; first_tokens[b] is the last token known of sequence b, to be
    written at positions[b]. generator: a torch.Generator of the device (the random numbers), or None for torch's
    own. temperature, top_k, top_p, min_p: a number for all sequences, one a sequence, or None. The drawn tokens
    feed the next step on the device; the host reads them when `tokens()` is called. logprobs: with a number, every
    step also keeps its tokens' log probabilities under the model's own logits, and as many alternatives (0: none)."""

    def __init__(self, model, kv, first_tokens, positions, vocab, temperature=None, top_k=None, top_p=None, min_p=None,
                 generator=None, device="cuda", logprobs=None):
        B = len(first_tokens)
        if len(positions) != B or B < 1:
            raise ValueError("one position per sequence")
        if int(vocab) != model.config.vocab:  # the step writes rows of the model's size
            raise ValueError(f"vocab {vocab}, but the model's is {model.config.vocab}")

        def ints(v):
            return torch.as_tensor(v, dtype=torch.int32).to(device)

        def each(v, dtype):
            if v is None:
                return None
            v = torch.as_tensor(v, dtype=dtype)
            if v.dim() > 1 or (v.dim() == 1 and v.shape[0] != B):
                raise ValueError("a setting is one number, or one a sequence")
            return v.expand(B).contiguous().to(device)

        self.model, self.kv, self.B, self.generator = model, kv, B, generator
        self.tok = ints(first_tokens).reshape(B, 1).contiguous()
        self.pos = ints(positions)
        self.logits = torch.empty((B, int(vocab)), dtype=torch.float32, device=device)
        self.u = torch.empty((B,), dtype=torch.float32, device=device)
        self.settings = dict(temperature=each(temperature, torch.float32), top_k=each(top_k, torch.int32),
                             top_p=each(top_p, torch.float32), min_p=each(min_p, torch.float32))
        if logprobs is not None and not 0 <= logprobs <= min(64, int(vocab)):
            raise ValueError(f"logprobs must be None or a number of alternatives up to {min(64, int(vocab))}, got {logprobs}")
        self.emitted = []
        self.top, self.scored = logprobs, []
        self.failed = None  # the error of a step, from then on

    def step(self):
        """One decode step and one draw a sequence; returns the tokens (int32 [batch], on the device)."""
        if self.failed:
            raise self.failed
        self.model.decode_step(self.kv, self.tok, self.pos, self.logits)
        self.u.uniform_(generator=self.generator)
        drawn = sample(self.logits, self.u, **self.settings)
        self.tok = drawn.reshape(self.B, 1)
        self.pos = self.pos + 1
        self.emitted.append(drawn)
        if self.top is not None:
            self.scored.append(logprobs(self.logits, drawn, top=self.top))
        return drawn

    def tokens(self):
        """The tokens drawn so far, [batch][steps], after checking the steps' device status. After a failed step (a row
        without a distribution, whose token -1 the next step refuses, or a position past the cache) it raises, and so
        do later calls: what was drawn from there on came from old logits."""
        self._settle()
        return torch.stack(self.emitted, dim=1).cpu().tolist() if self.emitted else [[] for _ in range(self.B)]

    def logprobs(self):
        """What the steps so far kept of their tokens' probabilities (a loop made with `logprobs`): (log probabilities
        [batch, steps], entropies [batch, steps], alternatives [batch, steps, n], their log probabilities), tensors on
        the host. Fails as `tokens()` does."""
        if self.top is None:
            raise ValueError("the loop was made without logprobs")
        self._settle()
        if not self.scored:
            return (torch.empty((self.B, 0)), torch.empty((self.B, 0)),
                    torch.empty((self.B, 0, self.top), dtype=torch.int32), torch.empty((self.B, 0, self.top)))
        return tuple(torch.stack(x, dim=1).cpu() for x in zip(*self.scored))

    def _settle(self):
        if not self.failed:
            try:
                self.model.check()
            except MKError as e:
                self.failed = e
        if self.failed:
            raise self.failed
