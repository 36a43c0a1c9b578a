"""Host logic of the head operators' torch calls, without a GPU."""
import pytest

import draft_verification_row_amd as sv
from draft_verification_row_amd import heads


@pytest.mark.parametrize("wrap", [1 << 32, 3 << 32, 1 << 31])
def test_sizes_past_32_bits_are_refused(wrap):
    """Sizes that a 32-bit argument would take for small ones."""
    for query, sizes in (("spec_logprobs_workspace_bytes", [1, 6, 100, 5]),
                         ("spec_draft_kl_workspace_bytes", [1, 2, 3, 100]),
                         ("spec_linear_workspace_bytes", [1, 4, 8, 16]),
                         ("spec_linear_grad_workspace_bytes", [1, 4, 8, 16])):
        assert heads._workspace_bytes(query, *sizes) > 0
        for i in (1, 2, 3):
            with pytest.raises(sv.SpecVerifyError):
                heads._workspace_bytes(query, *(n + wrap * (j == i) for j, n in enumerate(sizes)))
                print("not refused:", query, i)
