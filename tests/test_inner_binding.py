"""The inner-step binding on the host (no GPU): sizes that do not fit the ABI's
arguments, what it passes on, and the autograd operation with the two norm
calls replaced by their formulas in torch."""
import pytest
import torch

import pseudo_grad_sync_gb300 as dl
from pseudo_grad_sync_gb300 import _build, inner


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()
    return dl.lib()


def test_widths_beyond_the_abi_are_refused():
    """A 32-bit width would be cut: 2^32 + 64 columns taken as 64."""
    for width in (2**31, 2**32 + 64):
        x, w = (torch.empty(s, dtype=torch.bfloat16, device="meta") for s in ((2, width), (width,)))
        r = torch.empty(2, device="meta")
        with pytest.raises(ValueError, match="at most 2\\^31 - 1"):
            dl.layernorm_forward(x, w)
        with pytest.raises(ValueError, match="at most 2\\^31 - 1"):
            dl.layernorm_backward(x, x, w, r, r)
        with pytest.raises(ValueError, match="at most 2\\^31 - 1"):
            dl.layer_norm(x, w)
    x, w = (torch.empty(s, dtype=torch.bfloat16, device="meta") for s in ((2, 2**31 - 1), (2**31 - 1,)))
    with pytest.raises(ValueError, match="CUDA device"):  # the widest that fits: the next check
        dl.layernorm_forward(x, w)
