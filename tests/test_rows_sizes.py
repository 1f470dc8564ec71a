"""Sizes past 32 bits at the binding of the residual norm, the gated block and the log probabilities: refused, not taken for
what is left of them in 32 bits."""
import pytest
import torch

import bit_nf4_quantized_11_amd as Q
from helpers import log, require_gpu

WIDE = 1 << 32


def test_workspace_queries():
    assert Q.qlora_rms_norm_bwd_workspace(3, 64) > 0 and Q.qlora_gated_workspace(3, 64, 128, 8) > 0
    assert Q.qlora_token_logprob_workspace(3, 40000, 5) > 0
    for wide in (WIDE, -WIDE, 1 << 63, -(1 << 63)):
        assert Q.qlora_rms_norm_bwd_workspace(3, wide + 64) == 0
        assert Q.qlora_gated_workspace(3, 64, 128, wide + 8) == 0
        assert Q.qlora_token_logprob_workspace(3, 40000, wide + 5) == 0


@pytest.mark.gpu
def test_a_row_of_more_than_32_bits():
    """One row of 2^32 + 64 elements (8.6 GB) is none of 64."""
    require_gpu()
    log("rows of 2^32 + 64")
    x = torch.empty(1, WIDE + 64, dtype=torch.bfloat16, device="cuda")
    x[:, :64] = 1.0
    y = torch.zeros_like(x)
    with pytest.raises(Q.QLoRAError):
        Q.qlora_rms_norm(x, None, out=y)
    with pytest.raises(Q.QLoRAError):
        Q.qlora_rms_norm_bwd(x, x, None, dx=y)
    assert torch.all(y[:, :128] == 0)


@pytest.mark.gpu
def test_more_alternatives_than_logits():
    """Refused before anything of that size is allocated."""
    require_gpu()
    x, token = torch.zeros(1, 50, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    before = torch.cuda.max_memory_allocated()
    for top in (51, WIDE + 5, -WIDE + 5, 1 << 62):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_token_logprob(x, token, top=top)
    assert torch.cuda.max_memory_allocated() == before
    assert Q.qlora_token_logprob(x, token, top=32)[4].tolist() == [list(range(32))]
