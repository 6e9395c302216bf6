"""Shared pytest configuration.

Tests marked ``gpu`` need a GB300 and the built CUDA library; everything else
runs on a CPU-only machine (``pytest -m "not gpu"``).
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103) and the built library")


def pytest_runtest_setup(item):
    """Tests for a CPU-only machine may end a call that passes every check at the missing device.
    Where there is one, such a call would launch a kernel on pointers that are made up."""
    import pytest
    import torch

    made_up = ("test_norm_accepts", "test_append_accepts", "test_attention_accepts")
    if item.path.name == "test_decode_abi.py" and item.name in made_up and torch.cuda.is_available():
        pytest.skip("for a machine without a GPU: the pointers are made up")
