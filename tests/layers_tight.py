"""Limits on the layers' operators' errors taken together, beside layers_oracle's for each element.

Those bound the worst case: every rounding of a long sum at its most and of one sign.  At real widths they are so far
above what happens that a result may lack a part of a sum and keep them.  These are for the root mean square over many
elements of random inputs, where roundings add up as independent ones:

- A rounding to BF16 is off by at most 2^-8 of the value, evenly spread: 2^-8 / sqrt(3) root mean square at most.
  Experts round w h and y: 2^-8 sqrt(2 / 3).  A prompt's outputs round the weights of a chunk, the state they read
  and themselves; weights and state make a part of the output each: 2^-8 sqrt(2 / 3) as well.
- A state's keys are exact to FP32, its factors off by some units of 2^-24.  Each of a chunk's 12 products cuts the sum off
  below its 24th bit: 2^-24 of it on average, 7.2e-7 in all where a state holds the last chunk's tokens mostly.  (With the
  keys in two BF16 numbers, cut off, they are off by 2^-17 on average; one less cuts off 8 bits more.)
"""
from __future__ import annotations

import torch

EXPERTS = 2.0 ** -8 * (2 / 3) ** 0.5 * 1.05  # (5% for the sample, of 500 elements and more)
OUTPUTS = 2.0 ** -8 * (2 / 3) ** 0.5 * 1.05
STATES = 1e-6


def rms(got, want):
    """The error's root mean square, relative to that of the values."""
    got, want = got.detach().cpu().double(), want.double()
    return float((got - want).pow(2).sum().sqrt() / want.pow(2).sum().sqrt())


def cut_keys(k, f, numbers):
    """k times its factors f (FP64), as the sum of `numbers` BF16 numbers cut off after 8 bits each."""
    rest = (k.float() * f.float())
    total = torch.zeros(rest.shape, dtype=torch.float64)
    for _ in range(numbers):
        part = (rest.view(torch.int32) & -65536).view(torch.float32)
        total += part.double()
        rest = rest - part
    return total
