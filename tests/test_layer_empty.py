"""Calls of the training and serving operators over nothing: no tokens, no rows, no columns."""
import subprocess
import sys

import pytest
import torch


@pytest.mark.parametrize("query", ["qlora_forward_dropout_workspace_bytes", "qlora_backward_workspace_bytes",
                                   "mxfp4_forward_workspace_bytes", "mxfp4_backward_workspace_bytes"])
def test_workspace_of_no_tokens(query):
    # in a process of its own: a trap in the query would end this one
    code = f"from loftq_qlora_initialization_amd import binding as b\nprint([b.{query}(0, 64, c, r) for c in (0, 64, 8192) for r in (0, 8, 64)])"
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    assert len(run.stdout.split(",")) == 9


@pytest.mark.gpu
@pytest.mark.parametrize("r", [0, 8])
def test_serving_no_tokens(lib, r):
    W = torch.randn(64, 288, device="cuda")
    packed, scales = lib.loftq_mxfp4_quantize(W)
    X = torch.zeros(0, 288, dtype=torch.bfloat16, device="cuda")
    ad = dict(B=torch.randn(64, r, device="cuda"), A=torch.randn(r, 288, device="cuda")) if r else {}
    assert lib.loftq_mxfp4_forward(X, packed, scales, (64, 288), **ad).shape == (0, 64)
