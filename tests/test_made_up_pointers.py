"""Calls on made-up pointers that would pass every check are made on machines without a GPU only."""
from __future__ import annotations

import os
import re
import types

import pytest
import torch

import conftest

HERE = os.path.dirname(os.path.abspath(__file__))


def skipped(file, name):
    try:
        conftest.pytest_runtest_setup(types.SimpleNamespace(path=types.SimpleNamespace(name=file), name=name))
    except pytest.skip.Exception:
        return True
    return False


@pytest.mark.parametrize("gpu", [True, False])
def test_they_are_skipped_where_there_is_a_gpu(monkeypatch, gpu):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    text = open(os.path.join(HERE, "test_decode_abi.py")).read()
    names = re.findall(r"^def (test_\w+)", text, flags=re.M)
    body = dict(zip(names, re.split(r"^def test_\w+", text, flags=re.M)[1:]))
    # those that expect a call to come as far as the device
    assert {n for n in names if skipped("test_decode_abi.py", n)} == ({n for n in names if "OK_OR_DEVICE" in body[n]} if gpu else set())
    assert not skipped("test_other.py", "test_norm_accepts")
