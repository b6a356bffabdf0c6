"""The binding of the operators between tokens and singles, as far as it needs no GPU."""
import numpy as np
import pytest

import padding_free_pair_amd as nt

torch = pytest.importorskip("torch")

OF_TYPE = [nt.nt_token_loss_workspace_bytes, nt.nt_token_loss_backward_workspace_bytes]


@pytest.mark.parametrize("of", OF_TYPE)
def test_names_of_types(of):
    """A type by its torch or numpy dtype, its names or its code has the same workspace."""
    sizes = 400, 900, 128
    bf16, f32 = of(*sizes, nt.NT_BF16), of(*sizes, nt.NT_F32)
    assert bf16 != f32
    for dtype in (torch.bfloat16, "bf16", "bfloat16", "torch.bfloat16"):
        assert of(*sizes, dtype) == bf16, dtype
    for dtype in (torch.float32, "f32", "fp32", "float32", "torch.float32", np.float32,
                  np.dtype("float32")):
        assert of(*sizes, dtype) == f32, dtype


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, "half", "f16", "bfloat", "", None,
                                   np.float64, "float8_e4m3fn"])
def test_unknown_types(dtype):
    """A type that no operator takes is refused, not taken for float32."""
    for of in OF_TYPE:
        with pytest.raises(TypeError):
            of(400, 900, 128, dtype)
    with pytest.raises(TypeError):
        nt.nt_block_workspace_bytes(None, 384, 128, 512, dtype)
    with pytest.raises(TypeError):
        nt.nt_chain_workspace_bytes(None, 2, 384, 128, 512, dtype)
