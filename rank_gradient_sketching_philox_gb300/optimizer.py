"""AdamW for the tensors that are not sketched: norm weights, biases,
embeddings, a dense head; and clipping by the global norm of any gradients or
sketches.

The optimizer is bound to its tensors and their gradient buffers once and keeps
their states, in 32 bits or in 8; a step is one call of the library for all of
them.  Gradient buffers are fixed, like the sketches C that the layers
accumulate into: a backward pass writes or adds to them in place
(``layer_norm_backward``'s dgamma, ``cross_entropy_backward``'s dW).
"""
import torch

from . import binding

STATE_BLOCK = 256  # values of an 8-bit state that share a scale


class AdamW:
    """AdamW over the tensors ``params`` (BF16, stochastically rounded, or fp32)
    with gradients in ``grads`` (BF16 or fp32).

    state_bits: 32 (fp32 moments) or 8 (E4M3 codes of m and sqrt(v) with an fp32
    scale per 256 values: 2.03 bytes a value instead of 8).  ``state``: states
    to go on from, as ``state_dict()`` returns them (lists m, v, or m, u,
    m_scale, u_scale); zeros when not given.  ``layers``: the Philox counter word
    of each tensor's rounding stream, its index by default; tensors that share
    (seed, layer) with a sketched layer share that layer's rounding bits.
    """

    def __init__(self, params, grads, state_bits=32, state=None, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                 seed=0, layers=None):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32, got %r" % (state_bits,))
        self.params, self.grads = list(params), list(grads)
        self.state_bits, self.betas, self.eps, self.weight_decay, self.seed = state_bits, betas, eps, weight_decay, seed
        if not self.params:
            raise ValueError("no tensors")
        names = ("m", "v") if state_bits == 32 else ("m", "u", "m_scale", "u_scale")
        if state is None:
            state = {name: [self._zeros(p, name) for p in self.params] for name in names}
        if set(state) != set(names):
            raise ValueError("the states of %d bits are %s, got %s" % (state_bits, names, tuple(state)))
        self._state = {name: list(state[name]) for name in names}
        s = self._state
        self._problems = binding.adamw_problems(self.params, self.grads, s["m"], s[names[1]], s.get("m_scale"),
                                                s.get("u_scale"), layers)
        self._device = self.params[0].device

    def _zeros(self, p, name):
        if name.endswith("scale"):
            return torch.zeros((p.numel() + STATE_BLOCK - 1) // STATE_BLOCK, dtype=torch.float32, device=p.device)
        dtype = torch.float32 if self.state_bits == 32 else torch.float8_e4m3fn
        return torch.zeros(p.numel(), dtype=dtype, device=p.device)

    def state_dict(self):
        """The states themselves (not copies), a list per name."""
        return {name: list(ts) for name, ts in self._state.items()}

    def step(self, lr, step, grad_scale=None, stream=None):
        """Update every tensor with its gradient buffer; ``step`` counts from 0.
        grad_scale: a one-element fp32 device tensor that multiplies the
        gradients, or None."""
        binding.adamw_batched(self._problems, lr, self.betas, self.eps, self.weight_decay, self.seed, step,
                              grad_scale, self._device, stream)


class GradClip:
    """Clipping of the gradients (or sketches) ``grads`` by their global norm.

    ``step()`` writes ``norm`` = sqrt(sum of squares over all tensors) and ``scale`` =
    1 where norm <= max_norm, else max_norm / norm, one-element fp32 tensors that
    the host does not wait for: ``AdamW.step(..., grad_scale=clip.scale)``.  With
    ``outs`` (tensors of the same sizes and types, or the gradients themselves) it
    also writes the scaled gradients there; none of them overlaps another, or another's
    gradient.  Before the first step norm and scale hold nothing.  The object is bound to its tensors
    and keeps the call's workspace, so its steps are ordered on one stream.  Building it checks
    every tensor, which takes the host some 2.4 us for each (0.3 ms for 114, a step 9 us): gradients
    that are new tensors in every step (``zero_grad(set_to_none=True)``) need a new object each
    time, gradients that stay where they are, as sketches do, one for all steps.
    """

    def __init__(self, grads, max_norm, outs=None):
        self.grads = list(grads)
        self.outs = None if outs is None else list(outs)
        self.max_norm = float(max_norm)
        if not 0.0 < self.max_norm < float("inf"):
            raise ValueError("max_norm must be finite and > 0, got %r" % (max_norm,))
        self._problems = binding.grad_problems(self.grads, self.outs)
        if self.outs is not None and self._problems.written_twice:
            raise ValueError("a tensor of outs overlaps another one, or another's gradient")
        dev = self.grads[0].device
        self.norm = torch.empty(1, dtype=torch.float32, device=dev)
        self.scale = torch.empty(1, dtype=torch.float32, device=dev)
        self._ws = torch.empty(binding.workspace_bytes(binding.OP_GRAD_NORM, len(self.grads)), dtype=torch.uint8,
                               device=dev)

    def step(self, stream=None):
        """Measure the gradients, and scale them where there are ``outs``; returns the scale."""
        binding.grad_norm_batched(self._problems, self.norm, self.scale, self.max_norm, ws=self._ws, stream=stream)
        if self.outs is not None:
            binding.grad_scale_batched(self._problems, self.scale, stream=stream)
        return self.scale
