"""Calls of more rows than 32 bits count are refused, not cut."""
import pytest
import torch

import draft_verification_row_amd as sv

pytestmark = pytest.mark.gpu
ROWS = (1 << 32) + 3


def test_rows_past_32_bits_are_refused():
    """2^32 + 3 rows of one element each, which 32 bits take for three."""
    one = torch.zeros(ROWS, 1, dtype=torch.bfloat16, device="cuda")
    tok = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
    w = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda")
    kl = one.view(ROWS, 1, 1)
    for f in (lambda: sv.spec_token_logprobs(one, tok), lambda: sv.spec_linear(one, w),
              lambda: sv.spec_draft_kl(kl, kl), lambda: sv.spec_draft_kl(kl.view(1, ROWS, 1), kl[:1]),
              lambda: sv.spec_draft_kl(kl.view(1, ROWS, 1), kl.view(1, ROWS, 1))):
        with pytest.raises(sv.SpecVerifyError):
            f()
