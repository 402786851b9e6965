"""The drafted-tree example: the tree evaluated in one pass gives what its paths give token by token, and the
example's command runs."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [aq.AQ_KV_BF16, aq.AQ_KV_E4M3], ids=["bf16", "e4m3"])
def test_tree_equals_its_paths(kind):
    """Row i of the tree against the hidden state that the same model gives its path alone, as a chain of single
    tokens over the prompt. Both run bf16 activations through two layers (about 2^-8 a rounding, a dozen roundings
    on the way, the sums in different orders): 3 % in the 2-norm."""
    import draft_tree_step as ex
    model = ex.Model(kind=kind)
    r = np.random.RandomState(3)
    prompt = [int(t) for t in r.randint(0, 4096, 70)]
    parent = [-1, -1, 0, 0, 1, 2]
    drafts = [int(t) for t in r.randint(0, 4096, len(parent))]
    hidden, path, token = ex.step(model, prompt, drafts, parent)
    assert all(parent[b] == a for a, b in zip([-1] + path[:-1], path)) and 0 <= token < 4096
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    table = torch.arange(16, dtype=torch.int32, device="cuda")[None]
    for node in range(len(parent)):
        line = [node]
        while parent[line[0]] >= 0:
            line.insert(0, parent[line[0]])
        tokens = prompt + [drafts[i] for i in line]
        state = None
        for i, t in enumerate(tokens):
            if i < len(prompt) - 1:
                continue      # the prompt's keys and values are in the cache, the tree's are written over
            state = model.forward(torch.tensor([t], device="cuda"), torch.tensor([i], dtype=torch.int32, device="cuda"), table, one, 1)
        got, want = hidden[node + 1].double(), state[0].double()
        assert float((got - want).norm() / want.norm()) < 0.03, node
    assert aq.aq_device_status() == aq.AQ_OK


def test_example_command_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "draft_tree_step.py")], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-2000:]
    assert "accepted" in r.stdout
