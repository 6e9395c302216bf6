"""Limits of the layers' operators that are checked on the host, far beyond them.  No kernel is launched."""
from __future__ import annotations

import pytest

from test_layers_abi import lib, prompt, step  # noqa: F401  (lib is a fixture)


@pytest.mark.parametrize("B", [1 << 25, 1 << 28, 1 << 60, 1 << 61, (1 << 61) + 1, 1 << 62, (1 << 63) - 1])
def test_more_sequences_than_a_step_takes(lib, B):  # noqa: F811
    """8 heads each: the product passes 64 bits, and comes to 0 or little again."""
    assert step(lib, B=B) == 2
    assert prompt(lib, B=B) == 2
