"""What the compiled binding of the paged operators refuses before it looks at a tensor (no GPU)."""
import pytest
import torch

import block_sparse_streaming_b200 as bss


@pytest.fixture(scope="module", autouse=True)
def built():
    bss.build()


def test_parameter_structures_are_told_apart():
    """Params and RopeParams have the same size and, by their bytes alone, pass for each other."""
    x, pos = torch.zeros(2, 8, 64), torch.zeros(2, dtype=torch.int32)
    freq, window, rope = torch.zeros(32, dtype=torch.float64), bss.Params(1.0, 64, 0, 1), bss.RopeParams(64, 1, True)
    for bad in (window, bytes(rope), bytearray(bytes(rope)), torch.zeros(4).numpy(), None, 3):
        for call in (lambda: bss.loza_rope(x, pos, freq, bad), lambda: bss.loza_qk_norm_rope(x, x, pos, freq, bad),
                     lambda: bss.loza_qk_norm_rope_backward(x, x, x, x, pos, freq, bad)):
            with pytest.raises(TypeError, match="rope must be a RopeParams"):
                call()
    for bad in (rope, bytes(window), bytearray(bytes(window)), torch.zeros(4).numpy(), None, 3):
        with pytest.raises(TypeError, match="params must be a Params"):
            bss.loza_ssa_decode_paged_kv(x, x, x, pos.view(2, 1), pos, 1, bad)
