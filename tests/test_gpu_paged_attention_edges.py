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


# ------------------------------------------------------------------ bad metadata: what the rest of the call holds

@pytest.mark.parametrize('dtype', [BF, F32])
@pytest.mark.parametrize('width', [3, 300])          # tables with and without a split over the length
def test_a_bad_page_reads_as_zeros(dtype, width):
    H, P, D, lens = 2, 16, 64, [40, 17, 48]
    c = Cache(lens, H, P, D, dtype).fill(lens, 201)
    q = rand(202, 3, 8, D, dtype=dtype)
    K, V = (np.concatenate([np64(x), np.zeros((1, H, P, D))]) for x in (c.k, c.v))
    bt = np.zeros((3, width), dtype=np.int64)
    bt[:, :3] = c.bt
    for s, p, bad in ((0, 0, -1), (0, 2, c.pages), (1, 1, 1 << 30), (2, 1, -2 ** 31)):
        given, zero = bt.copy(), bt.copy()
        given[s, p], zero[s, p] = bad, c.pages       # (the oracle's caches have a page of zeros at their end)
        y = gdn.paged_attn_decode(q, c.k, c.v, i32(given), i32(lens), out_dtype=dtype)
        with pytest.raises(RuntimeError, match='device error 3'):
            gdn.check_device_error()
        ref = A.attention(np64(q), K, V, zero, [0, 1, 2, 3], lens, 1 / math.sqrt(D))
        close_attn(y, ref, max(lens), D, dtype, dtype, (s, p, bad))


@pytest.mark.parametrize('dtype', [BF, F32])
@pytest.mark.parametrize('width', [3, 300])
def test_bad_bounds_leave_their_rows_and_the_others_are_right(dtype, width):
    """Sequences whose bounds pass the number of tokens, or end before they start, are skipped: their rows of every
    output stay as they were, and the consistent sequences get what they get in a good call."""
    H, G, P, D, T = 2, 4, 16, 64, 6
    lens = [40, 17, 48]
    tab = rope_table(64, 32)
    q, k, v = rand(211, T, H * G, D, dtype=dtype), rand(212, T, H, D, dtype=dtype), rand(213, T, H, D, dtype=dtype)
    bt = np.zeros((3, width), dtype=np.int64)
    for bad_cu, good_cu, kept in (([0, 3, 9, 6], [0, 3, 6, 6], [0, 1, 2]), ([0, 3, 2, 1], [0, 3, 6, 6], [0, 1, 2]),
                                  ([1, 3, 5, 6], [0, 3, 5, 6], [3, 4, 5]), ([0, -1, 2, 6], [0, 0, 2, 6], [2, 3, 4, 5])):
        rest = [t for t in range(T) if t not in kept]
        got = []
        for cu in (bad_cu, good_cu):
            c = Cache(lens, H, P, D, dtype).fill(lens, 214)
            bt[:, :3] = c.bt
            out = [torch.full((T, H * G, D), 7.0, dtype=dtype, device='cuda') for _ in range(3)]
            calls = [lambda: gdn.qk_norm_rope(q, cos_sin=tab, cu_seqlens=i32(cu), q_out=out[0]),
                     lambda: gdn.paged_kv_append(k, v, c.k, c.v, i32(bt), i32(lens), q, tab, cu_seqlens=i32(cu), q_out=out[1]),
                     lambda: gdn.paged_attn_decode(q, c.k, c.v, i32(bt), i32(lens), cu_seqlens=i32(cu), o=out[2])]
            for i, call in enumerate(calls):
                if i == 2:                           # attention over one and the same cache
                    c.fill(lens, 214)
                call()
                if cu is bad_cu:
                    with pytest.raises(RuntimeError, match='device error 1'):
                        gdn.check_device_error()
                else:
                    gdn.check_device_error()
            got.append(out)
        for y, z in zip(*got):
            assert torch.equal(y[kept], z[kept]), bad_cu
            assert (y[rest] == 7).all(), bad_cu


# ------------------------------------------------------------------ norm + rotation over its own input, slots written twice

@pytest.mark.parametrize('T,Nq,Nkv,D,rot,inter', [(1, 16, 2, 256, 64, False), (77, 6, 3, 64, 64, False),
                                                  (300, 32, 8, 128, 128, False), (41, 40, 1, 128, 96, True)])
@pytest.mark.parametrize('dtype', [BF, F32])
def test_norm_rope_in_place(T, Nq, Nkv, D, rot, inter, dtype):
    q, k, tab = rand(221, T, Nq, D, dtype=dtype), rand(222, T, Nkv, D, dtype=dtype), rope_table(T, rot)
    w = 1 + rand(223, D, dtype=F32, std=0.2)
    qo, ko = gdn.qk_norm_rope(q, k, tab, w, w, interleaved=inter, out_dtype=dtype)
    q1, k1, q2 = q.clone(), k.clone(), q.clone()
    gdn.qk_norm_rope(q1, k1, tab, w, w, interleaved=inter, q_out=q1, k_out=k1)
    assert torch.equal(q1, qo) and torch.equal(k1, ko)
    c = Cache([T], Nkv, 16, D, dtype)
    gdn.paged_kv_append(k, k, c.k, c.v, c.block_table, i32([T]), q2, tab, w, w, interleaved=inter, q_out=q2)
    gdn.check_device_error()
    assert torch.equal(q2, qo)


def test_two_sequences_that_append_to_one_slot():
    """What is left there is made of the two rows; nothing else is touched."""
    c = Cache([16] * 32, 2, 16, 128, BF)
    c.bt[:, 0] = c.bt[0, 0]
    k, v = rand(231, 32, 2, 128), rand(232, 32, 2, 128)
    gdn.paged_kv_append(k, v, c.k, c.v, i32(c.bt), i32([5] * 32))
    gdn.check_device_error()
    for x, y in ((c.k, k), (c.v, v)):
        row = x[int(c.bt[0, 0]), :, 4].reshape(2, 16, 1, 8)           # 16-byte pieces
        assert (row == y.reshape(32, 2, 16, 8).permute(1, 2, 0, 3)).all(-1).any(-1).all()
        assert int((~x.isnan()).sum()) == 2 * 128


# ------------------------------------------------------------------ caches in other orders

@pytest.mark.parametrize('order', [(1, 0, 2, 3), (2, 0, 1, 3), (2, 1, 0, 3), (1, 2, 0, 3)])
@pytest.mark.parametrize('dtype', [BF, F32])
@pytest.mark.parametrize('P', [16, 20])
def test_any_order_of_pages_heads_and_slots(order, dtype, P):
    """Memory in the given order of the axes page 0, head 1, slot 2."""
    H, D, lens = 3, 128, [150, 33, 0, 7]
    c = Cache(lens, H, P, D, dtype)
    shape = (c.pages, H, P, D)
    back = [order.index(i) for i in range(4)]
    c.k, c.v = (torch.full([shape[i] for i in order], float('nan'), dtype=dtype, device='cuda').permute(back)
                for _ in range(2))
    assert c.k.shape == shape
    k, v, T = rand(241, 190, H, D, dtype=dtype), rand(242, 190, H, D, dtype=dtype), 190
    cu = i32([0, 150, 183, 183, 190])
    gdn.paged_kv_append(k, v, c.k, c.v, c.block_table, i32(lens), cu_seqlens=cu)
    gdn.check_device_error()
    assert int((~c.k.isnan()).sum()) == k.numel() and int((~c.v.isnan()).sum()) == v.numel()
    q = rand(243, T, 2 * H, D, dtype=dtype)
    check_attn(c, q, lens, [150, 33, 0, 7], out_dtype=dtype)


# ------------------------------------------------------------------ one workspace, many calls

@pytest.mark.parametrize('dtype', [BF, F32])
@pytest.mark.parametrize('N,most', [(1, 9000), (20, 2000), (100, 900)])          # few cut units, some, many
def test_calls_in_flight_on_one_workspace(dtype, N, most):
    """Calls of other lengths, inputs and numbers of tokens one behind the other, without a wait between them: each
    gives what it gives alone with a workspace of its own."""
    H, G, D, P = 2, 4, 128, 16
    rng = np.random.default_rng(N)
    calls, width = [], (most + P - 1) // P
    for i, t in enumerate((1, 1, 2, 1, 4)):
        lens = [int(x) for x in rng.integers(most // 2, most, N)]
        c = Cache(lens, H, P, D, dtype, seed=i)
        c.k.copy_(rand(250 + i, *c.k.shape, dtype=dtype))
        c.v.copy_(rand(260 + i, *c.v.shape, dtype=dtype))
        bt = np.zeros((N, width), dtype=np.int64)
        bt[:, :c.bt.shape[1]] = c.bt
        calls.append((rand(270 + i, N * t, H * G, D, dtype=dtype), c.k, c.v, i32(bt), i32(lens)))
    alone = []
    for a in calls:
        alone.append(gdn.paged_attn_decode(*a, out_dtype=dtype))
        torch.cuda.synchronize()
    n = gdn.paged_attn_decode_workspace_size(N, N, H * G, H, D, dtype, width * P)
    ws = torch.full((n,), 255, dtype=torch.uint8, device='cuda')
    order = rng.integers(0, len(calls), 120).tolist()
    outs = [gdn.paged_attn_decode(*calls[i], out_dtype=dtype, workspace=ws) for i in order]
    gdn.check_device_error()
    for i, y in zip(order, outs):
        assert torch.equal(y, alone[i]), i


def test_a_gate_made_on_another_stream_beside_the_append():
    """Fork before the append, join before the attention; eager, and captured into a graph."""
    N, H, D = 8, 2, 128
    lens = [int(x) for x in np.random.default_rng(3).integers(1, 1000, N)]
    c = Cache([1000] * N, H, 16, D, BF).fill(lens, 281)
    q, k, v, src = rand(282, N, 8, D), rand(283, N, H, D), rand(284, N, H, D), rand(285, N, 8, D)
    gate, big, n = src.clone(), rand(286, 2048, 2048, dtype=F32), i32(lens)
    side, own = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x = big @ big                            # some time before the gate is there
            gate.copy_(src + 0 * x[:1, :1].to(BF))
        gdn.paged_kv_append(k, v, c.k, c.v, c.block_table, n)
        main.wait_stream(side)
        return gdn.paged_attn_decode(q, c.k, c.v, c.block_table, n, gate=gate)

    gdn.paged_kv_append(k, v, c.k, c.v, c.block_table, n)
    ref = gdn.paged_attn_decode(q, c.k, c.v, c.block_table, n, gate=gate)
    torch.cuda.synchronize()
    for _ in range(10):
        gate.zero_()
        assert torch.equal(step(), ref)
    torch.cuda.synchronize()
    with torch.cuda.stream(own):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=own):
        y = step()
    for _ in range(10):
        gate.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
    gdn.check_device_error()


# ------------------------------------------------------------------ long contexts, each tile's share

def position_values(n, D):
    """Values [n, D] of which a row names its place: token j has a one in column j D / n.  A column of the output
    then is the weight of its stretch of tokens, and a tile that is lost or counted twice changes it."""
    v = np.zeros((n, D))
    v[np.arange(n), np.arange(n) * D // n] = 1.0
    return v


def close_shares(y, ref, n, units, D, in_dtype, out_dtype, ctas, what=''):
    """With values >= 0 the mass is the output itself, so the bound is relative.  The longest chain of additions into one sum
    is a CTA's share of the tokens (rounded up to tiles of up to 64), then the pieces of a unit, at most one per CTA."""
    close_attn(y, ref, -(-n * units // ctas) + 64 + ctas, D, in_dtype, out_dtype, what)


@pytest.mark.parametrize('D,H,dtype,n,P', [(256, 2, BF, 131072, 64), (128, 1, BF, 100003, 20), (64, 3, BF, 65537, 16),
                                           (128, 1, F32, 40009, 24), (256, 1, F32, 30000, 64)])
def test_every_tile_of_a_long_context_counts_once(D, H, dtype, n, P):
    c = Cache([n], H, P, D, dtype)
    c.k.copy_(rand(291, *c.k.shape, dtype=dtype))
    v = np.zeros((c.bt.shape[1] * P, D))
    v[:n] = position_values(n, D)
    c.v[c.block_table[0].long()] = torch.tensor(v, dtype=dtype, device='cuda').reshape(-1, 1, P, D)
    q = rand(292, 1, 4 * H, D, dtype=dtype)
    y = run_attn(c, q, [n], [1], out_dtype=dtype, cu=False)
    ref = A.attention(np64(q), np64(c.k), np64(c.v), c.bt, [0, 1], [n], 1 / math.sqrt(D))
    ctas = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    close_shares(y, ref, n, H, D, dtype, dtype, ctas)
