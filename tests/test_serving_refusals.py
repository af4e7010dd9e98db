"""What the binding of the serving calls refuses before the library is called.  No GPU."""

import pytest
import torch

from gated_deltanet_linear_conv_gb300 import gdn


@pytest.mark.parametrize('rows,num_seqs,bounds', [(6, 3, None), (2, 1, None), (3, 3, [0, 2, 3, 3]), (3, 3, [0, 1, 2, 3])])
def test_verify_without_a_row_of_draft_probs(monkeypatch, rows, num_seqs, bounds):
    """draft_probs of no drafts are not the same as none: drafts would be judged by another rule."""
    monkeypatch.setattr(gdn, '_device', lambda t: t.get_device())
    monkeypatch.setattr(gdn, '_fn', lambda name: pytest.fail('called ' + name))
    cu = None if bounds is None else torch.tensor(bounds, dtype=torch.int32)
    with pytest.raises(ValueError, match='no drafts'):
        gdn.draft_verify(torch.rand(rows, 8), torch.zeros(rows, dtype=torch.int32), torch.rand(rows), torch.rand(num_seqs, 0, 8),
                         cu_seqlens=cu, num_seqs=num_seqs)
