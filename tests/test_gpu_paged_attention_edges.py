"""Paged softmax attention on the GPU: calls that the header allows or refuses at its edges."""

import math

import numpy as np
import pytest
import torch

import oracle.attn_oracle as A
from gated_deltanet_linear_conv_gb300 import gdn
from helpers import np64
from test_gpu_paged_attention import BF, F32, Cache, check_attn, close_attn, i32, rand, rope_table, run_attn

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the layer step refuses as a whole

def _misaligned(*shape):
    return torch.zeros(math.prod(shape) + 1, dtype=BF, device='cuda')[1:].view(*shape)


REFUSED = {
    'o of another shape': (dict(bufs=lambda: dict(o=torch.zeros(2, 4, 64, dtype=BF, device='cuda'))), 'o must'),
    'o of another type': (dict(out_dtype=torch.float16), 'dtype'),
    'o not aligned': (dict(bufs=lambda: dict(o=_misaligned(1, 4, 64))), 'o must'),
    'q buffer of another type': (dict(bufs=lambda: dict(q=torch.zeros(1, 4, 64, device='cuda'))), 'dtype'),
    'q buffer of another shape': (dict(bufs=lambda: dict(q=torch.zeros(1, 2, 64, dtype=BF, device='cuda'))), 'q buffer'),
    'workspace too small': (dict(bufs=lambda: dict(workspace=torch.zeros(64, dtype=torch.uint8, device='cuda'))), 'workspace'),
    'workspace not aligned': (dict(bufs=lambda: dict(workspace=torch.zeros(1 << 27, dtype=torch.uint8, device='cuda')[8:])), 'workspace'),
    'gate of another type': (dict(gate=lambda: torch.zeros(1, 4, 64, device='cuda')), 'gate'),
    'gate of another shape': (dict(gate=lambda: torch.zeros(1, 2, 64, dtype=BF, device='cuda')), 'gate'),
    'gate not aligned': (dict(gate=lambda: _misaligned(1, 4, 64)), 'gate'),
    'gate with odd strides': (dict(gate=lambda: torch.zeros(1, 4, 68, dtype=BF, device='cuda')[..., :64]), 'gate'),
    'gate transposed': (dict(gate=lambda: torch.zeros(1, 64, 4, dtype=BF, device='cuda').transpose(1, 2)), 'gate'),
    'gate on the host': (dict(gate=lambda: torch.zeros(1, 4, 64, dtype=BF)), 'gate'),
    'scale no number': (dict(scale='1'), None),
}


@pytest.mark.parametrize('what', REFUSED)
def test_layer_step_refuses_before_the_cache_changes(what):
    kw, word = REFUSED[what]
    c = Cache([4096], 2, 16, 64, BF)                 # a table long enough to need a workspace
    q, k = rand(1, 1, 4, 64), rand(2, 1, 2, 64)
    kw = {n: x() if callable(x) else x for n, x in kw.items()}
    with pytest.raises((ValueError, TypeError) if word else Exception, match=word):
        gdn.attention_decode(q, k, k, c.k, c.v, c.block_table, i32([3]), **kw)
    gdn.check_device_error()
    assert c.k.isnan().all() and c.v.isnan().all()


def test_layer_step_with_buffers_equals_its_two_calls():
    c, d = (Cache([4096, 100], 2, 16, 64, BF).fill([700, 33], 7) for _ in range(2))
    q, k, v, lens = rand(1, 2, 4, 64), rand(2, 2, 2, 64), rand(3, 2, 2, 64), i32([700, 33])
    gate = rand(4, 2, 4, 64)
    n = gdn.paged_attn_decode_workspace_size(2, 2, 4, 2, 64, BF, c.bt.shape[1] * 16)
    bufs = dict(q=torch.empty_like(q), o=torch.empty(2, 4, 64, device='cuda'),
                workspace=torch.empty(n, dtype=torch.uint8, device='cuda'))
    y = gdn.attention_decode(q, k, v, c.k, c.v, c.block_table, lens, gate=gate, scale=0.2, bufs=bufs)
    qr = gdn.paged_kv_append(k, v, d.k, d.v, d.block_table, lens, q=q)
    z = gdn.paged_attn_decode(qr, d.k, d.v, d.block_table, lens, 0.2, gate, out_dtype=F32)
    gdn.check_device_error()
    assert y.data_ptr() == bufs['o'].data_ptr() and torch.equal(bufs['q'], qr) and torch.equal(y, z)
    seen = ~d.k.isnan()
    assert torch.equal(c.k.isnan(), d.k.isnan()) and torch.equal(c.k[seen], d.k[seen])
    # one token: strides over its axis are never used
    g1 = torch.empty_strided((1, 4, 64), (3, 64, 1), dtype=BF, device='cuda').copy_(gate[:1])
    y1 = gdn.attention_decode(q[:1], k[:1], v[:1], c.k, c.v, c.block_table[:1], lens[:1], gate=g1, scale=0.2, out_dtype=F32)
    z1 = gdn.paged_attn_decode(q[:1], d.k, d.v, d.block_table[:1], lens[:1], 0.2, gate[:1], out_dtype=F32)
    gdn.check_device_error()
    assert torch.equal(y1, z1)
