"""Arguments of the attention block's calls that are no tensors of the expected
kind end in the library's own errors."""

import pytest
import torch

import sparse_convolution_hash_amd as spc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(4, 1, 0), (4, 2, 0), (4, 0, 16), (0, 1, 0)])
def test_heads_of_no_elements(shape):
    e = torch.zeros(*shape, device="cuda")
    with pytest.raises((ValueError, spc.SpcError)):
        spc.attention_fwd(e, e, e)


def test_out_that_is_no_tensor():
    x, f = torch.zeros(4, 2, 16, device="cuda"), torch.zeros(8, device="cuda")
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    for out in (3, x.cpu(), x.half()):
        with pytest.raises(TypeError):
            spc.rotary(x, pos, f, (8,), out=out)
        with pytest.raises(TypeError):
            spc.attention_fwd(x, x, x, out=out)
    with pytest.raises(ValueError):
        spc.rotary(x, pos, f, (8,), out=x[:2])
