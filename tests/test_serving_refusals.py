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


@pytest.mark.parametrize('D', [64, 128, 256])
def test_workspace_of_the_4_bit_attention(D):
    """What the header says: nothing for short tables, else 5.2 MB at most on 152 SMs, whatever the table."""
    from gated_deltanet_linear_conv_gb300 import _build
    _build.build()
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152
    sizes = {gdn.paged_kv4_attn_decode_workspace_size(D, n) for n in (513, 4096, 1 << 20, 1 << 40)}
    assert len(sizes) == 1 and 4e6 * sms / 152 < max(sizes) <= 5.2e6 * sms / 152
    assert gdn.paged_kv4_attn_decode_workspace_size(D, 0) == gdn.paged_kv4_attn_decode_workspace_size(D, 512) == 0
