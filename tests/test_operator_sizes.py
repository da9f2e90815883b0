"""CPU checks of sizes that do not fit the C calls' integers."""
import pytest
import torch

from calibration_free_vector_b200 import nsn


@pytest.mark.parametrize("tokens", [2**31, 2**32, 2**32 + 1])
def test_readback_refuses_more_tokens_than_32_bits_hold(tokens):
    # 2**32 + 1 rows on top of each other would arrive in C as one
    cache = nsn.Cache(1, 1, 128, 128, 2, device="cpu")
    out = torch.empty((1, 1, 1, 128)).expand(1, tokens, 1, 128)
    with pytest.raises(ValueError, match="below 2"):
        nsn.nsn_dequantize_kv(cache, out, torch.empty((256, 8)))
