"""CPU pins of the paged-attention oracle, and the host-side refusals of its calls."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.attn_oracle as A


def table(P, r, theta=1e4):
    ang = np.arange(P)[:, None] * theta ** (-2.0 * np.arange(r // 2) / r)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1)


@pytest.mark.parametrize('inter', [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance_only(inter):
    rng = np.random.default_rng(0)
    tab = table(64, 16)
    q, k = rng.standard_normal((2, 1, 1, 24))
    rot = lambda x, p: A.norm_rope(x, None, 0.0, tab, [p], inter)  # noqa: E731
    np.testing.assert_array_equal(rot(q, 0), q)
    np.testing.assert_array_equal(rot(q, 7)[..., 16:], q[..., 16:])
    assert np.linalg.norm(rot(q, 9)) == pytest.approx(np.linalg.norm(q), rel=1e-12)
    a = float((rot(q, 30) * rot(k, 21)).sum())
    assert a == pytest.approx(float((rot(q, 12) * rot(k, 3)).sum()), rel=1e-10)


def test_rotation_by_hand():
    # r = 4, one position with cosines (0, 1) and sines (1, 0): the first pair turns by 90 degrees
    row = np.array([0.0, 1.0, 1.0, 0.0])
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0])
    np.testing.assert_array_equal(A.norm_rope_row(x, None, 0, row, False), [-3, 2, 1, 4, 5])
    np.testing.assert_array_equal(A.norm_rope_row(x, None, 0, row, True), [-2, 1, 3, 4, 5])
    y = A.norm_rope_row(np.array([3.0, 4.0]), np.array([1.0, 2.0]), 0.0, None, False)
    np.testing.assert_allclose(y, np.array([3.0, 8.0]) / math.sqrt(12.5), rtol=1e-15)


def test_attention_closed_forms():
    # equal scores average the visible values; one token returns its own; an inactive sequence gives zeros
    k = np.zeros((3, 1, 4, 2))
    v = np.arange(24.0).reshape(3, 1, 4, 2)
    bt = np.array([[2, 0], [1, 1], [0, 0]])
    q = np.ones((4, 2, 2))
    y, mass, _ = A.attention(q, k, v, bt, [0, 2, 3, 4], [6, 1, 0], 1.0)
    idx = [v[2, 0, 0], v[2, 0, 1], v[2, 0, 2], v[2, 0, 3], v[0, 0, 0], v[0, 0, 1]]
    np.testing.assert_allclose(y[0, 0], np.mean(idx[:5], 0))
    np.testing.assert_allclose(y[1, 1], np.mean(idx, 0))
    np.testing.assert_allclose(y[2, 0], v[1, 0, 0])
    assert not y[3].any() and not mass[3].any()


def test_append_then_attention_equals_dense_causal_attention():
    rng = np.random.default_rng(1)
    T, H, G, D, P = 9, 2, 2, 8, 4
    q, k, v = rng.standard_normal((T, H * G, D)), rng.standard_normal((T, H, D)), rng.standard_normal((T, H, D))
    ck, cv = np.full((4, H, P, D), np.nan), np.full((4, H, P, D), np.nan)
    bt = [[3, 1, 0]]
    out = []
    for a, b in ((0, 4), (4, 5), (5, 9)):
        A.append(ck, cv, k[a:b], v[a:b], bt, [0, b - a], [b])
        out.append(A.attention(q[a:b], ck, cv, bt, [0, b - a], [b], 0.3)[0])
    sc = 0.3 * np.einsum('thd,shd->hts', q, k.repeat(G, 1))
    sc = np.where(np.tril(np.ones((T, T), bool)), sc, -np.inf)
    w = np.exp(sc - sc.max(-1, keepdims=True))
    ref = np.einsum('hts,shd->thd', w / w.sum(-1, keepdims=True), v.repeat(G, 1))
    np.testing.assert_allclose(np.concatenate(out), ref, rtol=1e-12, atol=1e-12)


# ---------------------------------------------------------------- refusals (no launch, no GPU)

@pytest.fixture(scope='module')
def gdn():
    from gated_deltanet_linear_conv_gb300 import _build, gdn as m
    _build.build()
    m.lib()
    return m


X = 0x10000          # stands for an aligned device address: never read, every call below is refused


def _args(gdn, **kw):
    a = dict(N=2, T=2, Nq=8, Nkv=2, D=128, cu=None, ts=1024, hs=128, dt=0, rot=64, inter=0, maxpos=16, tab=X, pos=None,
             qw=X, kw=X, k=X, v=X, ps=2 * 16 * 128, chs=16 * 128, ss=128, pages=4, psize=16, maxp=2, bt=X, lens=X,
             q=X, qout=X, cdt=0, odt=0, gate=None, ws=X, wsb=1 << 40, nr=True, cache=True)
    a.update(kw)
    H = gdn.gdn_heads
    d = gdn.gdn_attn_dims(a['N'], a['T'], a['Nq'], a['Nkv'], a['D'])
    h = H(a['q'], a['ts'], a['hs'])
    nr = gdn.gdn_norm_rope(a['qw'], a['kw'], 1e-6, a['rot'], a['inter'], a['maxpos'], a['tab'], a['pos']) if a['nr'] else None
    c = gdn.gdn_paged_cache(a['k'], a['v'], a['ps'], a['chs'], a['ss'], a['pages'], a['psize'], a['maxp'], a['bt'],
                            a['lens']) if a['cache'] else None
    return a, d, h, nr, c


def _append(gdn, **kw):
    a, d, h, nr, c = _args(gdn, **kw)
    kv = gdn.gdn_heads(X, 256, 128)
    return gdn.lib().gdn_paged_kv_append(d, a['cu'], h, kv, kv, a['dt'], nr, c, a['cdt'], a['qout'], a['odt'], None)


def _attn(gdn, **kw):
    a, d, h, _, c = _args(gdn, **kw)
    return gdn.lib().gdn_paged_attn_decode(d, a['cu'], h, a['gate'], a['dt'], c, 1.0, a['qout'], a['odt'], a['ws'],
                                           a['wsb'], None)


def _rope(gdn, **kw):
    a, d, h, nr, _ = _args(gdn, **kw)
    return gdn.lib().gdn_qk_norm_rope(d, a['cu'], h, None, a['dt'], nr, a['qout'], None, a['odt'], None)


BOTH = [(dict(Nq=9), 'INVALID', 'multiple'), (dict(N=0), 'INVALID', 'num_seqs'), (dict(T=-1), 'INVALID', 'total_tokens'),
        (dict(T=3), 'INVALID', 'cu_seqlens'), (dict(D=96), 'UNSUPPORTED', 'head dim'), (dict(dt=5), 'INVALID', 'dtype'),
        (dict(odt=2), 'INVALID', 'dtype'), (dict(q=X + 8), 'INVALID', 'aligned'), (dict(ts=1020), 'INVALID', 'strides'),
        (dict(hs=-128), 'INVALID', 'strides'), (dict(cu=X + 4), 'INVALID', 'aligned'), (dict(qout=None), 'INVALID', 'NULL'),
        (dict(Nkv=0), 'INVALID', 'head counts')]
CACHE = [(dict(cache=False), 'INVALID', 'cache'), (dict(k=None), 'INVALID', 'cache_k'), (dict(v=X + 2), 'INVALID', 'cache_v'),
         (dict(bt=None), 'INVALID', 'block_table'), (dict(lens=X + 4), 'INVALID', 'kv_lens'),
         (dict(pages=0), 'INVALID', 'num_pages'), (dict(psize=0), 'INVALID', 'page_size'), (dict(maxp=0), 'INVALID', 'max_pages'),
         (dict(ps=4095), 'INVALID', 'strides'), (dict(chs=0), 'INVALID', 'strides'), (dict(ss=120), 'INVALID', 'overlap'),
         (dict(chs=15 * 128), 'INVALID', 'overlap'), (dict(ps=16 * 128), 'INVALID', 'overlap'), (dict(ss=2 * 128, chs=64), 'INVALID', 'overlap'),
         (dict(ps=2 * 16 * 128 + 8), 'UNSUPPORTED', 'multiples'), (dict(psize=1 << 30, ps=1 << 38, pages=1 << 30), 'INVALID', 'overlap'),
         (dict(ps=1 << 39), 'INVALID', 'strides')]
NR = [(dict(rot=144), 'INVALID', 'rotary_dim'), (dict(rot=24), 'UNSUPPORTED', 'multiple of 16'),
      (dict(tab=None), 'INVALID', 'cos_sin'), (dict(maxpos=0), 'INVALID', 'max_positions'),
      (dict(inter=2), 'INVALID', 'interleaved'), (dict(pos=X + 4), 'INVALID', 'positions'), (dict(qw=X + 4), 'INVALID', 'q_norm_w')]


@pytest.mark.parametrize('call,kw,code,word',
                         [(f, *c) for f, cs in (('rope', BOTH + NR), ('append', BOTH + NR + CACHE), ('attn', BOTH + CACHE))
                          for c in cs])
def test_refusals(gdn, call, kw, code, word):
    st = {'rope': _rope, 'append': _append, 'attn': _attn}[call](gdn, **kw)
    assert st == getattr(gdn, 'GDN_ERR_%s%s' % (code, '_ARG' if code == 'INVALID' else ''))
    assert word in gdn.lib().gdn_last_error_string().decode(), gdn.lib().gdn_last_error_string()


def test_workspace_too_small_is_refused(gdn):
    big = dict(maxp=4096)                              # tables of 65536 entries
    assert _attn(gdn, wsb=16, **big) == _attn(gdn, ws=None, **big) == _attn(gdn, ws=X + 8, **big) == gdn.GDN_ERR_INVALID_ARG
    assert b'workspace' in gdn.lib().gdn_last_error_string()


@pytest.mark.parametrize('dtype', [torch.bfloat16, torch.float32])
def test_one_workspace_serves_any_number_of_tokens(gdn, dtype):
    """Calls pick their rows per pass by the tokens per sequence; the size has to be that of the most."""
    for Nq, Nkv, D in ((8, 2, 64), (8, 2, 128), (8, 1, 128), (16, 2, 256), (4, 4, 256)):
        sizes = {gdn.paged_attn_decode_workspace_size(n, n * t, Nq, Nkv, D, dtype, 1 << 20)
                 for n in (1, 7, 256) for t in range(1, 10)}
        assert len(sizes) == 1 and sizes.pop() > 0


def test_no_tokens_is_no_work(gdn):
    assert _rope(gdn, T=0) == _append(gdn, T=0) == _attn(gdn, T=0) == gdn.GDN_OK


def test_null_structs(gdn):
    L = gdn.lib()
    n = ctypes.c_size_t(0)
    size = L.gdn_paged_attn_decode_workspace_size
    d = gdn.gdn_attn_dims(3, 7, 8, 2, 128)
    assert size(None, 0, 64, n) == size(d, 0, 64, None) == size(d, 3, 64, n) == size(d, 0, -1, n) == gdn.GDN_ERR_INVALID_ARG
    assert size(gdn.gdn_attn_dims(3, 7, 8, 2, 96), 0, 64, n) == gdn.GDN_ERR_UNSUPPORTED
    assert size(d, 0, 64, n) == gdn.GDN_OK and n.value == 0           # short tables need none
    assert size(d, 0, 100000, n) == gdn.GDN_OK and n.value > 0
    short = n.value
    assert size(d, 0, 1 << 40, n) == gdn.GDN_OK and n.value == short
    assert L.gdn_paged_attn_decode(None, None, None, None, 0, None, 1.0, None, 0, None, 0, None) == gdn.GDN_ERR_INVALID_ARG
    assert _rope(gdn, nr=False) == gdn.GDN_ERR_INVALID_ARG


def test_packed_structs_have_the_c_layout(gdn):
    h = gdn.gdn_heads.from_buffer_copy(gdn._pack_heads(5, -6, 7))
    assert (h.data, h.token_stride, h.head_stride) == (5, -6, 7)
    vals = (1, 2, 0.5, 4, 5, 6, 7, 8)
    n = gdn.gdn_norm_rope.from_buffer_copy(gdn._pack_norm_rope(*vals))
    assert tuple(getattr(n, f) for f, _ in gdn.gdn_norm_rope._fields_) == vals
    vals = tuple(range(1, 11))
    c = gdn.gdn_paged_cache.from_buffer_copy(gdn._pack_cache(*vals))
    assert tuple(getattr(c, f) for f, _ in gdn.gdn_paged_cache._fields_) == vals
    d = gdn.gdn_attn_dims.from_buffer_copy(gdn._pack_dims(1, 2, 3, 4, 5))
    assert tuple(getattr(d, f) for f, _ in gdn.gdn_attn_dims._fields_) == (1, 2, 3, 4, 5)


def test_binding_refusals(gdn):
    bf = torch.bfloat16
    q, kc = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(3, 2, 16, 64, dtype=bf)
    bt, lens = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match='CUDA'):
        gdn.paged_attn_decode(q, kc, kc, bt, lens)                     # CPU tensors
    with pytest.raises(ValueError, match='dtype'):
        gdn.paged_attn_decode(q, kc.float(), kc.float(), bt, lens)
    with pytest.raises(ValueError, match='shape'):
        gdn._cache(kc, kc[:2], bt, lens, 2, 64, 2, -1)
    with pytest.raises(ValueError, match='heads'):
        gdn._cache(kc, kc, bt, lens, 4, 64, 2, -1)
    with pytest.raises(ValueError, match='contiguous'):
        gdn._cache(kc.transpose(2, 3).contiguous().transpose(2, 3), kc, bt, lens, 2, 64, 2, -1)
    with pytest.raises(ValueError, match='strides'):
        gdn._cache(kc, torch.zeros(3, 16, 2, 64, dtype=bf).transpose(1, 2), bt, lens, 2, 64, 2, -1)
    with pytest.raises(ValueError, match='block_table'):
        gdn._cache(kc, kc, bt, lens[:1], 2, 64, 2, -1)
    with pytest.raises(ValueError, match='int32'):
        gdn._cache(kc, kc, bt, lens.long(), 2, 64, 2, -1)
    with pytest.raises(ValueError, match='contiguous'):
        gdn._cache(kc, kc, torch.zeros(1, 2, dtype=torch.int32).T.expand(2, 2), lens, 2, 64, 2, -1)
    with pytest.raises(ValueError, match='contiguous'):
        gdn._heads(torch.zeros(2, 64, 8).transpose(1, 2), -1, 'q')
    with pytest.raises(ValueError, match='norm weight'):
        gdn._norm_rope(torch.zeros(32), None, 1e-6, None, None, False, 2, 64, -1)
    with pytest.raises(ValueError, match='share'):
        gdn.qk_norm_rope(q, q.float())


@pytest.mark.parametrize('pages,ps', [(1 << 26, 1 << 38), (1 << 30, 1 << 34), ((1 << 30) + 1, 1 << 34), (1 << 23, (1 << 38) + (1 << 20))])
@pytest.mark.parametrize('call', ['append', 'attn'])
def test_strides_that_span_more_than_any_memory_are_refused(gdn, call, pages, ps):
    """Also where the product of a stride and its extent passes 64 bits."""
    st = {'append': _append, 'attn': _attn}[call](gdn, pages=pages, ps=ps)
    assert st == gdn.GDN_ERR_INVALID_ARG
    assert b'span' in gdn.lib().gdn_last_error_string(), gdn.lib().gdn_last_error_string()


@pytest.mark.parametrize('n,D,dtype', [(131072, 256, torch.bfloat16), (65537, 64, torch.bfloat16), (40009, 128, torch.float32)])
def test_a_lost_or_doubled_tile_of_a_long_context_is_seen(n, D, dtype):
    """The GPU test of long contexts rejects an answer that lacks a tile, or a CTA's piece, or has it twice."""
    from test_gpu_paged_attention_edges import close_shares, position_values

    rng = np.random.default_rng(2)
    k, q, v = rng.standard_normal((n, D)), rng.standard_normal(D), position_values(n, D)
    x = k @ q / math.sqrt(D)
    w = np.exp(x - x.max())
    smax = (np.abs(k) @ np.abs(q)).max(keepdims=True) / math.sqrt(D)
    y = (w / w.sum()) @ v
    near = lambda z: close_shares(torch.tensor(z)[None].to(dtype), (y[None], y[None], smax), n, 2, D, dtype, dtype, 304)  # noqa: E731
    near(y)
    tile = 8192 // (D * dtype.itemsize)
    for length in (tile, 862 // tile * tile):
        for t0 in (0, 10 * tile, n // 2 // tile * tile, n - length):
            for times in (0.0, 2.0):
                z = w.copy()
                z[t0:t0 + length] *= times
                with pytest.raises(AssertionError):
                    near((z / z.sum()) @ v)
