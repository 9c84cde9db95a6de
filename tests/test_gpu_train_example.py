"""examples/train_rows.py: the dense operators together with the coded table."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_rows.py")


def test_training_lowers_the_loss_and_the_coded_rows_read_out_alike():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    spec = importlib.util.spec_from_file_location("train_rows", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, difference, square = example.train(rows=1000, tokens=512, steps=30)
    assert all(a == a for a in losses) and losses[-1] < 0.8 * losses[0], losses
    # two bits a value: the trellis leaves about a sixteenth of a Gaussian row's square, the norm and product pass it on
    assert difference < 0.25 * square, (difference, square)
    again, _, _ = example.train(rows=1000, tokens=512, steps=30)
    assert losses == again  # nothing depends on how the GPU schedules the work
