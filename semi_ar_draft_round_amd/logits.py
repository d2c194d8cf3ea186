"""What the requests of a serving process ask of the target's logits.

Conditions owns the device buffers of include/dspark_logits.h for `slots`
requests (the token history, the penalties, the biases) and calls the entry
points in a round's order:

    conditions.prompt(tokens, start, count)       # new requests
    conditions.apply(d.target, ell, d.gamma, d.x0, d.x, mask=mask)   # after the target's pass
    conditions.commit(ell, d.n_acc, d.x0, d.x)    # after dspark_verify

device_round.run_round_cached does the last two.  The tensors `repetition`,
`presence`, `frequency` [slots], `bias_tok` and `bias` [slots][biases] are the
caller's to fill (a bias_tok of -1 is none); they start without effect.
Nothing is allocated after construction except what fork needs for a moment,
so a round can be captured in a HIP graph.  All calls run on the current
stream.
"""

from __future__ import annotations

import torch

from . import binding as B


class Conditions:
    def __init__(self, slots: int, vocab: int, biases: int = 0, device="cuda:0"):
        if slots < 1 or vocab < 2 or biases < 0:
            raise ValueError(f"no conditions of {slots} slots, {vocab} tokens, {biases} biases")
        dev = torch.device(device)
        f32 = dict(dtype=torch.float32, device=dev)
        self.state = torch.zeros((slots, vocab), dtype=torch.int16, device=dev)
        self.repetition, self.presence, self.frequency = (torch.full((slots,), x, **f32) for x in (1.0, 0.0, 0.0))
        self.bias_tok = torch.full((slots, biases), -1, dtype=torch.int32, device=dev) if biases else None
        self.bias = torch.zeros((slots, biases), **f32) if biases else None

    def prompt(self, tokens, start, count):
        """Slot r starts over with the prompt tokens[start[r]] .. of count[r]
        tokens (count[r] < 0: goes on as it is)."""
        B.dspark_logits_prompt(self.state, tokens, start, count)

    def apply(self, logits, ell, gamma: int, x0, x=None, *, row0=None, mask=None, out=None):
        """The rows' logits under every request's conditions, in place unless
        `out` is given."""
        return B.dspark_logits(logits, self.state, ell, gamma, x0, x, row0=row0, repetition=self.repetition,
                               presence=self.presence, frequency=self.frequency, bias_tok=self.bias_tok,
                               bias=self.bias, mask=mask, out=logits if out is None else out)

    def commit(self, ell, n_acc, x0, x=None):
        """The anchor and the accepted drafts of every request that had rows."""
        B.dspark_logits_commit(self.state, ell, n_acc, x0, x)

    def fork(self, parent):
        """Slot r goes on from parent[r]'s history and conditions (r: its own;
        -1: an empty history; values outside [-1, slots) leave r alone)."""
        from .cache import rows_of_parents
        if parent.shape != self.state.shape[:1] or parent.dtype not in (torch.int32, torch.int64) or (
                parent.device != self.state.device):
            raise ValueError(f"parent must be [{self.state.shape[0]}] int32 on {self.state.device}, not "
                             f"{list(parent.shape)} {parent.dtype} on {parent.device}")
        for t in (self.state, self.repetition, self.presence, self.frequency, self.bias_tok, self.bias):
            if t is not None:
                t.copy_(rows_of_parents(t, parent, empty=t is self.state))
