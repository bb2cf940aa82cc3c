"""The example that trains and searches a tied-vocabulary model with the vocabulary
operators and the fused loss (examples/tied_vocabulary.py)."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "tied_vocabulary.py")


def _module():
    spec = importlib.util.spec_from_file_location("tied_vocabulary", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_help_and_host_parts():
    r = subprocess.run([sys.executable, PATH, "--help"], capture_output=True, text=True)
    assert r.returncode == 0 and "--beams" in r.stdout
    m = _module()
    assert m.follow(torch.tensor([0, 1]), 3).tolist() == [[3, 18, 93], [8, 43, 24]]
    # the states' backward pass is their adjoint
    e, c = torch.randn(2, 5, 3, dtype=torch.float64), torch.randn(2, 5, 3, dtype=torch.float64)
    assert abs((m.states_of(e) * c).sum() - (e * m.states_backward(c)).sum()) < 1e-12


@pytest.mark.gpu
def test_learns_and_searches_the_rule():
    import __graft_entry__
    __graft_entry__.build()
    losses, right, errors = _module().main(["--steps", "300"])
    assert errors == (0, 0)
    # untrained: about ln 97 = 4.57; the rule has no uncertainty once it is learned
    assert losses[0] > 3.5 and losses[-1] < 0.1
    assert right == 1.0
