"""The shape of the first tokens' outputs at the binding of the log probabilities (no GPU)."""
import pytest
import torch

from speculative_decoding_vocab_gb300 import binding as ssd


@pytest.mark.parametrize("shape", [(2, 3), (6,), (), (2, 3, 4, 1), (2, 4, 3), (3, 2, 4)])
@pytest.mark.parametrize("which", ["top_ids", "top_logprob"])
def test_first_tokens_of_another_shape(which, shape):
    dtype = torch.int32 if which == "top_ids" else torch.float32
    with pytest.raises(ValueError, match=which):
        ssd.ssd_token_logprobs(torch.zeros(2, 3, 16), 16, 1.0, status=torch.zeros(1, dtype=torch.int32),
                               **{which: torch.zeros(shape, dtype=dtype)})
