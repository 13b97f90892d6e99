"""What the expert operators' Python calls refuse before anything is launched (no GPU needed)."""
from types import SimpleNamespace

import pytest

import moe_expert_token_gb300 as moe
from moe_expert_token_gb300 import build as mbuild


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()


def test_a_stream_of_another_device_is_refused():
    """The call would run on the tensors' device, on a stream that the caller did not name."""
    import torch

    x = SimpleNamespace(device=torch.device("cuda", 0))
    stream = SimpleNamespace(device=torch.device("cuda", 1))
    for call, args in ((moe.moe_mx_quantize, (x,)), (moe.moe_mx_dequantize, (x, x)),
                       (moe.moe_mx_grouped_matmul, (x,) * 5), (moe.moe_few_token_layer, (x, x, x, x, 2))):
        with pytest.raises(ValueError, match="stream"):
            call(*args, stream=stream)


def test_no_state_is_shared_between_copies_of_the_library():
    """A variable that the loader makes one for all copies (a unique symbol) would say of one copy's kernels
    that their attributes are set when another's are."""
    import shutil
    import subprocess

    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("needs nm")
    out = subprocess.run([nm, "-C", mbuild.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert [line for line in out.splitlines() if " u " in line and ("moe_" in line or "mrr" in line or "tc::" in line)] == []
