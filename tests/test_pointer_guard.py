"""Tests that hand made-up pointers to the C entry points do not run where a
kernel could be launched on them."""
import types

import pytest
import torch

import conftest
import test_serving_abi


def items():
    return [types.SimpleNamespace(function=f, marks=[], name=n) for n, f in vars(test_serving_abi).items() if n.startswith("test_")]


@pytest.mark.parametrize("device", [False, True])
def test_only_without_a_device(device, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: device)
    every = items()
    for x in every:
        x.add_marker = x.marks.append
    conftest.pytest_collection_modifyitems(every)
    skipped = {x.name for x in every if x.marks}
    wanted = {"test_valid_arguments_reach_the_device", "test_rope_refusals", "test_append_refusals",
              "test_append_rows_that_would_overlap_are_refused", "test_decode_refusals", "test_decode_limit_of_steps"}
    assert skipped == (wanted if device else set())
