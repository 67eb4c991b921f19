"""Corners of the operators of include/ar_ops.h that show without a GPU."""
import pytest
import torch

import tensor_decode_all_gb300 as tda


@pytest.fixture(scope="module", autouse=True)
def _built():
    tda.build()


@pytest.mark.parametrize("call", [tda.Kv4Workspace, tda.kv4_workspace, tda.kv4_workspaces])
def test_a_workspace_wants_a_cuda_device(call):
    with pytest.raises(ValueError, match="not a CUDA device"):
        call("cpu")
    with pytest.raises(ValueError, match="not a CUDA device"):
        call(torch.device("meta"))
