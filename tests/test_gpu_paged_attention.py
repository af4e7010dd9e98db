"""Paged softmax attention on the GPU against the fp64 oracle: norm + rotation, append,
attention of the new tokens, and the three together.

Tolerances, per element.  A stored value is off by at most half a step of its type, h =
finfo.eps / 2, relative to itself.  Before that:
 - norm + rotation in float32: a sum of D squares in any order, its mean, root and two products are off by
   less than (8 + log2 D + 8) 2^-24 < 2^-19 relative to u, and a c - b s adds 3 roundings of at most
   |a| + |b|: 2^-19 (|a| + |b|) bounds it, with |a| + |b| at most 2 max |u| of the row's rotated part or of
   the element itself.
 - attention: a score is off by at most ds = (D + 4) 2^-23 smax, smax = scale sum |q_i k_i| (2^-23, a whole step,
   also covers accumulators that truncate), so each weight by a factor e^(2 ds) and a few steps of the
   exponential (8 2^-23); the sums over n tokens add n 2^-23; weights rounded to a pair of bf16 values for the
   tensor cores 2^-16.  All relative to the mass sum_j p_j |v_j|.
"""

import math

import numpy as np
import pytest
import torch

import oracle.attn_oracle as A
from gated_deltanet_linear_conv_gb300 import gdn
from helpers import np64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device='cuda')


def rand(seed, *shape, dtype=BF, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def rope_table(P, r, theta=1e6):
    ang = np.arange(P)[:, None] * theta ** (-2.0 * np.arange(r // 2) / r)
    return torch.tensor(np.concatenate([np.cos(ang), np.sin(ang)], 1), dtype=F32, device='cuda')


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close_rows(y, ref, u, dtype, what=''):
    """Norm + rotation: y against ref with u the oracle's row before the rotation (see above)."""
    y = np64(y)
    tol = half_step(dtype) * np.abs(ref) + 2.0 ** -18 * np.abs(u).max(-1, keepdims=True)
    bad = ~(np.abs(y - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist())


def close_attn(y, ref, n_max, D, in_dtype, out_dtype, what=''):
    y0, mass, smax = ref
    e = 2 * (D + 4) * 2.0 ** -23 * smax[..., None] + (8 + n_max) * 2.0 ** -23
    if in_dtype == BF:
        e = e + 2.0 ** -16
    tol = half_step(out_dtype) * np.abs(y0) + 1.01 * np.expm1(np.minimum(e, 50)) * mass + 1e-37
    y = np64(y)
    bad = ~(np.abs(y - y0) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.nanmax(np.abs(y - y0))))


def cuts(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).tolist()


# ------------------------------------------------------------------ norm + rotation

@pytest.mark.parametrize('D,rot,inter,norm', [(64, 64, False, True), (64, 16, True, False), (128, 128, False, True),
                                              (128, 96, False, False), (128, 32, True, True), (256, 64, False, True),
                                              (256, 256, True, True), (256, 240, False, True), (128, 0, False, True)])
@pytest.mark.parametrize('din,dout', [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_qk_norm_rope(D, rot, inter, norm, din, dout):
    lengths = [1, 0, 7, 30, 1]
    T, Nq, Nkv = sum(lengths), 6, 3
    q, k = rand(1, T, Nq, D, dtype=din, std=2.0), rand(2, T, Nkv, D, dtype=din, std=0.5)
    wq, wk = (1 + rand(3, D, dtype=F32, std=0.2), 1 + rand(4, D, dtype=F32, std=0.2)) if norm else (None, None)
    tab = rope_table(40, rot) if rot else None
    qo, ko = gdn.qk_norm_rope(q, k, tab, wq, wk, cu_seqlens=i32(cuts(lengths)), interleaved=inter, out_dtype=dout)
    pos = [i for n in lengths for i in range(n)]
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        ref = A.norm_rope(np64(x), np64(w), 1e-6, np64(tab), pos, inter)
        close_rows(y, ref, A.norm_rope(np64(x), np64(w), 1e-6, None, pos, inter), dout)
    gdn.check_device_error()


def test_qk_norm_rope_one_token_positions_slices_and_in_place():
    T, Nq, Nkv, D, rot = 5, 4, 2, 128, 64
    tab, w = rope_table(2000000, rot), 1 + rand(3, D, dtype=F32, std=0.2)
    joint = rand(5, T, 2 * Nq + 2 * Nkv, D)                  # a joint projection: q and k are slices of it
    q, k = joint[:, :2 * Nq:2], joint[:, 2 * Nq:2 * Nq + Nkv]
    pos = [0, 1999999, 17, 1048577, 3]                       # far positions come from the table as they are
    qr = A.norm_rope(np64(q), np64(w), 1e-6, np64(tab), pos, False)
    u = A.norm_rope(np64(q), np64(w), 1e-6, None, pos, False)
    kr = A.norm_rope(np64(k), None, 1e-6, np64(tab), pos, False)
    qo, ko = gdn.qk_norm_rope(q, k, tab, w, None, positions=i32(pos))
    close_rows(qo, qr, u, BF)
    close_rows(ko, kr, np64(k), BF)
    one = q[1:2].contiguous()
    y, none = gdn.qk_norm_rope(one, cos_sin=tab, q_norm_w=w, positions=i32(pos[1:2]), q_out=one)
    assert none is None and y.data_ptr() == one.data_ptr() and torch.equal(y, qo[1:2])
    # q alone with NaN in a row: only that row is NaN
    bad = q.contiguous().clone()
    bad[2, 1, 5] = float('nan')
    y, _ = gdn.qk_norm_rope(bad, cos_sin=tab, q_norm_w=w, positions=i32(pos))
    ok = torch.ones(T, Nq, dtype=torch.bool)
    ok[2, 1] = False
    assert torch.equal(y[ok.cuda()], qo[ok.cuda()]) and y[2, 1].isnan().all()


def test_qk_norm_rope_bad_positions_and_lengths():
    T, D = 6, 64
    q, tab = rand(6, T, 2, D), rope_table(4, 32)
    out = torch.full((T, 2, D), 7.0, dtype=BF, device='cuda')
    gdn.qk_norm_rope(q, cos_sin=tab, positions=i32([0, 4, 1, -1, 3, 2]), q_out=out)
    with pytest.raises(RuntimeError, match='device error 3'):
        gdn.check_device_error()
    assert (out[1] == 7).all() and (out[3] == 7).all() and not (out[[0, 2, 4, 5]] == 7).all(-1).any()
    out.fill_(7.0)
    gdn.qk_norm_rope(q, cos_sin=tab, cu_seqlens=i32([0, 3, 2, 6]), q_out=out)
    with pytest.raises(RuntimeError, match='device error 1'):
        gdn.check_device_error()
    gdn.check_device_error()


def test_qk_norm_rope_many_tokens():
    T, D = 5003, 128
    q, k, tab = rand(7, T, 9, D), rand(8, T, 3, D), rope_table(T, D)
    w = 1 + rand(3, D, dtype=F32, std=0.2)
    qo, ko = gdn.qk_norm_rope(q, k, tab, w, w)
    rows = [0, 1, 777, 4095, 4096, T - 1]
    for x, y in ((q, qo), (k, ko)):
        x = np64(x[rows])
        close_rows(y[rows], A.norm_rope(x, np64(w), 1e-6, np64(tab), rows, False),
                   A.norm_rope(x, np64(w), 1e-6, None, rows, False), BF)
    # every row equals the same row of a call of its own tokens only
    qs, _ = gdn.qk_norm_rope(q[2500:].contiguous(), cos_sin=tab, q_norm_w=w,
                             positions=torch.arange(2500, T, dtype=torch.int32, device='cuda'))
    assert torch.equal(qs, qo[2500:])


# ------------------------------------------------------------------ the cache

class Cache:
    """A cache of sequences of the given capacities with shuffled pages, filled with NaN."""

    def __init__(self, caps, H, P, D, dtype, seed=0, token_major=False, joint=False):
        need = [(c + P - 1) // P for c in caps]
        self.pages, self.P = sum(need) + 2, P
        ids = np.random.default_rng(seed).permutation(self.pages)
        width = max(1, max(need))
        self.bt = np.full((len(caps), width), -1)
        at = 0
        for s, n in enumerate(need):
            self.bt[s, :n] = ids[at:at + n]
            at += n
        shape = (self.pages, P, H, D) if token_major else (self.pages, H, P, D)
        if joint:                                    # k and v of a page side by side
            both = torch.full((self.pages, 2) + shape[1:], float('nan'), dtype=dtype, device='cuda')
            kv = both[:, 0], both[:, 1]
        else:
            kv = (torch.full(shape, float('nan'), dtype=dtype, device='cuda') for _ in range(2))
        self.k, self.v = (x.transpose(1, 2) if token_major else x for x in kv)
        self.block_table = i32(self.bt)

    def fill(self, lens, seed, k_std=1.0):
        """Random keys and values below each length; everything else stays NaN."""
        H, D = self.k.shape[1], self.k.shape[3]
        for s, n in enumerate(lens):
            for p in range((n + self.P - 1) // self.P):
                m = min(self.P, n - p * self.P)
                page = int(self.bt[s, p])
                self.k[page, :, :m] = rand(seed + 7919 * s + p, H, m, D, dtype=self.k.dtype, std=k_std)
                self.v[page, :, :m] = rand(seed + 7919 * s + p + 104729, H, m, D, dtype=self.k.dtype)
        return self


@pytest.mark.parametrize('D,H,P,din,dc,kw', [
    (64, 3, 16, BF, BF, {}), (128, 2, 7, BF, BF, dict(token_major=True)), (256, 1, 1, F32, F32, {}),
    (256, 2, 64, BF, BF, dict(joint=True)), (128, 8, 24, F32, BF, {}), (64, 1, 256, BF, F32, dict(token_major=True, joint=True))])
@pytest.mark.parametrize('with_q,rope', [(True, True), (False, True), (True, False)])
def test_append(D, H, P, din, dc, kw, with_q, rope):
    # ragged new tokens: one, none, many, an inactive slot, a whole sequence
    new, lens = [1, 0, 5, 2, 40], [33, 9, 70, 0, 40]
    T, Nq, cu = sum(new), 2 * H, cuts(new)
    c = Cache([n + 3 for n in lens], H, P, D, dc, **kw)
    q, k, v = (rand(s, T, h, D, dtype=din) for s, h in ((1, Nq), (2, H), (3, H)))
    tab, wq, wk = rope_table(80, 32), 1 + rand(3, D, dtype=F32, std=0.2), 1 + rand(4, D, dtype=F32, std=0.2)
    args = dict(cos_sin=tab, q_norm_w=wq, k_norm_w=wk) if rope else {}
    q_out = torch.full((T, Nq, D), 7.0, dtype=din, device='cuda') if with_q else None
    r = gdn.paged_kv_append(k, v, c.k, c.v, c.block_table, i32(lens), q=q if with_q else None, cu_seqlens=i32(cu),
                            q_out=q_out, **args)
    gdn.check_device_error()
    assert r is q_out
    idx = [p for _, p in A.new_token_indices(cu, lens)]
    act = [t for t, p in enumerate(idx) if p is not None]
    pos = [idx[t] for t in act]

    def expect(x, w):
        x = np64(x)[act]
        return (A.norm_rope(x, np64(w), 1e-6, np64(tab), pos, False), A.norm_rope(x, np64(w), 1e-6, None, pos, False)) \
            if rope else (x, x)

    K, V = np64(c.k), np64(c.v)
    kr, ku = expect(k, wk)
    seen = np.zeros((c.pages, P), bool)
    rows = A.new_token_indices(cu, lens)
    for n, t in enumerate(act):
        page, slot = c.bt[rows[t][0]][rows[t][1] // P], rows[t][1] % P
        seen[page, slot] = True
        close_rows(torch.tensor(K[page, :, slot]), kr[n], ku[n], dc)
        assert np.array_equal(V[page, :, slot], np64(v[t].to(dc)))
    assert np.isnan(K.transpose(0, 2, 1, 3)[~seen]).all() and np.isnan(V.transpose(0, 2, 1, 3)[~seen]).all()
    if with_q:
        qr, qu = expect(q, wq)
        close_rows(q_out[act], qr, qu, din)
        rest = [t for t in range(T) if t not in act]
        assert (q_out[rest] == 7).all()              # an inactive sequence: nothing written


def test_append_positions_apart_from_cache_indices():
    """A cache that dropped its oldest tokens: positions run ahead of the cache index."""
    c = Cache([40], 2, 16, 64, F32)
    k, v, tab = rand(1, 2, 2, 64, dtype=F32), rand(2, 2, 2, 64, dtype=F32), rope_table(1000, 64)
    gdn.paged_kv_append(k, v, c.k, c.v, c.block_table, i32([20]), cos_sin=tab, positions=i32([998, 999]), interleaved=True)
    ref = A.norm_rope(np64(k), None, 0, np64(tab), [998, 999], True)
    for i, p in enumerate((18, 19)):
        close_rows(c.k[int(c.bt[0, p // 16]), :, p % 16], ref[i], np64(k)[i], F32)


def test_append_bad_metadata_writes_nothing_there():
    P, H, D = 16, 2, 64
    k, v = rand(1, 4, H, D), rand(2, 4, H, D)
    # too long for its row of the table; a page id out of range; fewer cached than new; below zero; then a good one
    for lens, edit, bad in (([33, 8, 8, 8], None, 0), ([8, 8, 8, 8], (1, -2), 1), ([8, 8, 8, 8], (2, 99), 2), ([8, 8, 8, -1], None, 3)):
        c = Cache([32] * 4, H, P, D, BF)
        if edit:
            c.bt[edit[0], 0] = edit[1]
            c.block_table = i32(c.bt)
        gdn.paged_kv_append(k, v, c.k, c.v, c.block_table, i32(lens))
        with pytest.raises(RuntimeError, match='device error 3'):
            gdn.check_device_error()
        for s in range(4):
            if s != bad:
                assert torch.equal(c.k[int(c.bt[s, 0]), :, 7], k[s]) and torch.equal(c.v[int(c.bt[s, 0]), :, 7], v[s])
        assert int((~c.k.isnan()).sum()) == 3 * H * D
    c = Cache([32] * 2, H, P, D, BF)
    gdn.paged_kv_append(k, v, c.k, c.v, c.block_table, i32([1, 8]))           # two new tokens, one cached
    with pytest.raises(RuntimeError, match='device error 3'):
        gdn.check_device_error()
    assert int((~c.k.isnan()).sum()) == 2 * H * D


# ------------------------------------------------------------------ attention

def run_attn(c, q, lens, new, gate=None, out_dtype=BF, scale=None, cu=True, **kw):
    y = gdn.paged_attn_decode(q, c.k, c.v, c.block_table, i32(lens), scale, gate, i32(cuts(new)) if cu else None,
                              out_dtype=out_dtype, **kw)
    gdn.check_device_error()
    return y


def check_attn(c, q, lens, new, gate=None, out_dtype=BF, scale=None, cu=True, what=''):
    D = q.shape[2]
    y = run_attn(c, q, lens, new, gate, out_dtype, scale, cu)
    # unused slots are NaN: the oracle reads only the visible ones
    ref = A.attention(np64(q), np64(c.k), np64(c.v), c.bt, cuts(new), lens, scale or 1 / math.sqrt(D), np64(gate))
    close_attn(y, ref, max(lens), D, q.dtype, out_dtype, what)
    return y


LENS = [1, 2, 15, 16, 17, 0, 31, 33, 63, 64, 65, 127, 129, 200]


@pytest.mark.parametrize('D', [64, 128, 256])
@pytest.mark.parametrize('dtype', [BF, F32])
@pytest.mark.parametrize('H,G', [(1, 1), (2, 3), (3, 8), (1, 12), (2, 16), (4, 5)])
def test_attention_head_layouts(D, dtype, H, G):
    c = Cache(LENS, H, 16, D, dtype).fill(LENS, 11)
    q = rand(12, len(LENS), H * G, D, dtype=dtype, std=2.0)
    check_attn(c, q, LENS, [1] * len(LENS), out_dtype=dtype, cu=False)


@pytest.mark.parametrize('P', [1, 3, 8, 20, 24, 32, 48, 64, 128, 256, 100])
@pytest.mark.parametrize('D,dtype', [(64, BF), (128, BF), (256, BF), (128, F32), (256, F32), (64, F32)])
def test_attention_page_sizes(P, D, dtype):
    c = Cache(LENS, 2, P, D, dtype, token_major=P % 3 == 0, joint=P % 2 == 0).fill(LENS, 21)
    q, gate = rand(22, len(LENS), 8, D, dtype=dtype), rand(23, len(LENS), 8, D, dtype=dtype, std=3.0)
    check_attn(c, q, LENS, [1] * len(LENS), gate, out_dtype=F32)


@pytest.mark.parametrize('D,dtype,G', [(64, BF, 8), (128, BF, 4), (256, BF, 8), (256, BF, 16), (128, F32, 8), (64, F32, 3), (64, F32, 8), (128, F32, 3), (256, F32, 4),
                                       (256, F32, 6), (64, F32, 12)])
def test_attention_several_new_tokens(D, dtype, G):
    """Draft + verify with ragged counts, an inactive slot, no tokens, and a whole prompt at once."""
    new, lens = [1, 4, 0, 3, 2, 37, 8], [50, 4, 30, 66, 0, 37, 300]
    c = Cache(lens, 2, 16, D, dtype).fill(lens, 31)
    q, gate = rand(32, sum(new), 2 * G, D, dtype=dtype), rand(33, sum(new), 2 * G, D, dtype=dtype)
    check_attn(c, q, lens, new, gate, out_dtype=dtype)


@pytest.mark.parametrize('P', [20, 12, 3])
@pytest.mark.parametrize('D,G,n', [(64, 3, 4), (64, 8, 6), (128, 4, 4), (128, 4, 5), (128, 8, 2), (256, 4, 2), (256, 8, 3)])
@pytest.mark.parametrize('dtype', [BF, F32])
def test_several_new_tokens_in_tiles_that_are_not_full(P, D, G, n, dtype):
    """Every count of octets per pass, with a last pass that is not full, over whole and cut units."""
    lens = [n, 19, 20, 21, 61, 333, 1200]
    c = Cache(lens, 1, P, D, dtype).fill(lens, 35)
    q = rand(36, n * len(lens), G, D, dtype=dtype)
    check_attn(c, q, lens, [n] * len(lens), out_dtype=dtype)
    new = [n] * len(lens)
    new[1], new[4] = n - 1, n + 1
    check_attn(c, q, lens, new, out_dtype=dtype)


@pytest.mark.parametrize('dtype', [BF, F32])
def test_one_workspace_for_calls_of_any_number_of_tokens(dtype):
    lens = [1200, 333, 700]
    c = Cache(lens, 1, 16, 128, dtype).fill(lens, 37)
    n = gdn.paged_attn_decode_workspace_size(3, 3 * 9, 4, 1, 128, dtype, c.bt.shape[1] * c.P)
    ws = torch.full((n,), 255, dtype=torch.uint8, device='cuda')
    for t in range(1, 10):
        q = rand(38 + t, 3 * t, 4, 128, dtype=dtype)
        y = run_attn(c, q, lens, [t] * 3, out_dtype=dtype, workspace=ws)
        assert torch.equal(y, check_attn(c, q, lens, [t] * 3, out_dtype=dtype))


@pytest.mark.parametrize('D,dtype', [(64, BF), (128, BF), (256, BF), (64, F32), (128, F32), (256, F32)])
def test_later_tokens_never_reach_a_row(D, dtype):
    """NaN and infinities in a later new token's key and value leave the earlier rows as they are."""
    new, lens = [4, 3], [77, 35]
    c = Cache(lens, 1, 16, D, dtype).fill(lens, 41)
    q = rand(42, 7, 4, D, dtype=dtype)
    y = check_attn(c, q, lens, new, out_dtype=dtype)
    for s, bad in ((0, float('nan')), (1, float('inf'))):
        p = lens[s] - 1
        c.k[int(c.bt[s, p // 16]), :, p % 16] = bad
        c.v[int(c.bt[s, p // 16]), :, p % 16] = bad
    z = run_attn(c, q, lens, new, out_dtype=dtype)
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(z[keep], y[keep])
    assert z[3].isnan().all() and z[6].isnan().any()


@pytest.mark.parametrize('D,H,G,dtype,n', [(128, 2, 8, BF, 20011), (256, 1, 8, BF, 40000), (64, 8, 1, BF, 9999), (128, 1, 4, F32, 30001)])
def test_one_long_sequence(D, H, G, dtype, n):
    c = Cache([n], H, 64, D, dtype)
    c.k.copy_(rand(51, *c.k.shape, dtype=dtype))
    c.v.copy_(rand(52, *c.v.shape, dtype=dtype))
    check_attn(c, rand(53, 2, H * G, D, dtype=dtype, std=2.0), [n], [2], out_dtype=dtype)


def test_many_sequences_of_mixed_lengths():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    lens[13], lens[500] = 5000, 2500
    c = Cache(lens, 2, 32, 128, BF)
    c.k.copy_(rand(61, *c.k.shape))
    c.v.copy_(rand(62, *c.v.shape))
    check_attn(c, rand(63, 700, 16, 128), lens, [1] * 700)


@pytest.mark.parametrize('dtype', [BF, F32])
def test_extreme_scores(dtype):
    """Far apart, all equal, all hugely negative, and -inf scores beside finite ones."""
    D, n = 128, 300
    c = Cache([n] * 4, 1, 16, D, dtype).fill([n] * 4, 71)
    q = rand(72, 4, 8, D, dtype=dtype)
    q[0] *= 200.0                                     # one token takes all the weight
    q[1] = 0.0                                        # equal weights
    for p in range(n):
        c.k[int(c.bt[2, p // 16]), :, p % 16] = 1e18  # scores near -1e38 and equal
    q[2] = -1e18
    y = check_attn(c, q, [n] * 4, [1] * 4, out_dtype=dtype, cu=False)
    V = np64(c.v)[c.bt[2][np.arange(n) // 16], 0, np.arange(n) % 16]     # rows 1 and 2: plain averages
    tol = half_step(dtype) * np.abs(V.mean(0)) + (n + 8) * 2.0 ** -23 * np.abs(V).mean(0) + 2.0 ** -16 * np.abs(V).mean(0)
    assert (np.abs(np64(y[2]) - V.mean(0)) <= tol).all()
    page, slot = int(c.bt[3, 5]), 3                   # a key of -inf: its score is -inf, its weight 0
    c.k[page, :, slot, 0] = float('-inf')
    q[3, :, 0] = 1.0
    y = run_attn(c, q, [n] * 4, [1] * 4, out_dtype=dtype, cu=False)
    j = [p for p in range(n) if p != 83]
    pages = c.bt[3][np.array(j) // 16]
    K, V = np64(c.k)[pages, 0, np.array(j) % 16], np64(c.v)[pages, 0, np.array(j) % 16]
    x = np64(q)[3] @ K.T / math.sqrt(D)
    w = np.exp(x - x.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    smax = (np.abs(np64(q)[3]) @ np.abs(K).T).max(-1) / math.sqrt(D)
    close_attn(y[3], (w @ V, w @ np.abs(V), smax), n, D, dtype, dtype)


@pytest.mark.parametrize('dtype', [BF, F32])
def test_values_of_inf_reach_their_rows_only(dtype):
    """(As inf, or as NaN where a weight is held as the sum of two.)"""
    lens = [40, 40]
    c = Cache(lens, 2, 16, 64, dtype).fill(lens, 75)
    q = rand(76, 2, 8, 64, dtype=dtype)
    y = run_attn(c, q, lens, [1, 1], out_dtype=dtype)
    c.v[int(c.bt[0, 1]), 1, 2, 9] = float('inf')      # sequence 0, kv head 1, column 9
    z = run_attn(c, q, lens, [1, 1], out_dtype=dtype)
    hit = torch.zeros(2, 8, 64, dtype=torch.bool, device='cuda')
    hit[0, 4:, 9] = True
    assert torch.equal(z[~hit], y[~hit]) and not z[hit].isfinite().any()


def test_attention_bad_metadata():
    H, P, D = 2, 16, 64
    for dtype in (BF, F32):
        good = [20, 20, 20, 20]
        q = rand(81, 4, 8, D, dtype=dtype)
        c = Cache(good, H, P, D, dtype).fill(good, 82)
        y = run_attn(c, q, good, [1] * 4, out_dtype=dtype)
        for lens, edit, s in (([20, 20, 33, 20], None, 2), ([20, -3, 20, 20], None, 1), (good, (3, -1), 3), (good, (0, 1 << 20), 0)):
            bt = c.bt.copy()
            if edit:
                bt[edit[0], 0] = edit[1]
            z = gdn.paged_attn_decode(q, c.k, c.v, i32(bt), i32(lens), out_dtype=dtype)
            with pytest.raises(RuntimeError, match='device error 3'):
                gdn.check_device_error()
            keep = [x for x in range(4) if x != s]
            assert torch.equal(z[keep], y[keep])
            assert not z[s].any() if edit is None else z[s].isfinite().all()
        gdn.paged_attn_decode(q, c.k, c.v, c.block_table, i32(good), cu_seqlens=i32([0, 2, 1, 3, 4]), out_dtype=dtype)
        with pytest.raises(RuntimeError, match='device error 1'):
            gdn.check_device_error()


@pytest.mark.parametrize('dtype', [BF, F32])
def test_offsets_past_32_bits(dtype):
    """A cache of more than 2^32 elements whose used pages lie at its end; append, then attention."""
    H, P, D, n = 2, 64, 128, 150
    pages = (1 << 32) // (H * P * D) + 5
    k = torch.zeros(pages, H, P, D, dtype=dtype, device='cuda')
    v = torch.zeros(pages, H, P, D, dtype=dtype, device='cuda')
    bt = np.array([[pages - 1, pages - 3, pages - 2]])
    kk, vv, q = rand(1, n, H, D, dtype=dtype), rand(2, n, H, D, dtype=dtype), rand(3, n, 8, D, dtype=dtype)
    gdn.paged_kv_append(kk, vv, k, v, i32(bt), i32([n]))
    y = gdn.paged_attn_decode(q[-1:].contiguous(), k, v, i32(bt), i32([n]), out_dtype=dtype)
    gdn.check_device_error()
    assert torch.equal(k[pages - 3, :, 5], kk[64 + 5]) and torch.equal(v[pages - 2, 1, 21], vv[149, 1])
    ref = A.attention(np64(q[-1:]), np64(k[-3:]), np64(v[-3:]), bt - (pages - 3), [0, 1], [n], 1 / math.sqrt(D))
    close_attn(y, ref, n, D, dtype, dtype)


# ------------------------------------------------------------------ as they are used together

def _layer(seed, N, T_cap, H=2, G=4, D=128, rot=64, P=16):
    c = Cache([T_cap] * N, H, P, D, BF, seed=seed)
    return dict(c=c, tab=rope_table(T_cap, rot), wq=1 + rand(3, D, dtype=F32, std=0.2), wk=1 + rand(4, D, dtype=F32, std=0.2),
                H=H, G=G, D=D)


def _step_inputs(L, seed, T):
    joint = rand(seed, T, 2 * L['H'] * L['G'] + 2 * L['H'], L['D'])    # [q | gate per head, k, v]
    Nq = L['H'] * L['G']
    return joint, joint[:, 0:2 * Nq:2], joint[:, 1:2 * Nq:2], joint[:, 2 * Nq:2 * Nq + L['H']], joint[:, 2 * Nq + L['H']:]


def _step(L, x, lens, cu=None, **kw):
    _, q, gate, k, v = x
    return gdn.attention_decode(q, k, v, L['c'].k, L['c'].v, L['c'].block_table, lens, L['tab'], L['wq'], L['wk'], gate,
                                cu_seqlens=cu, **kw)


def _check_step(L, x, y, lens, cu):
    """The step's rows against the oracle, from the rows that the cache and q really hold (each rounded to bf16)."""
    _, q, gate, k, v = x
    rows = A.new_token_indices(cu, lens)
    pos = [0 if p is None else p for _, p in rows]
    c, H = L['c'], L['H']
    kr = A.norm_rope(np64(k), np64(L['wk']), 1e-6, np64(L['tab']), pos, False)
    ku = A.norm_rope(np64(k), np64(L['wk']), 1e-6, None, pos, False)
    K = np64(c.k)
    for t, (s, p) in enumerate(rows):
        if p is not None:
            page, slot = c.bt[s][p // c.P], p % c.P
            close_rows(torch.tensor(K[page, :, slot]), kr[t], ku[t], BF)
    qr = A.norm_rope(np64(q), np64(L['wq']), 1e-6, np64(L['tab']), pos, False)
    y0, mass, smax = A.attention(qr, K, np64(c.v), c.bt, cu, lens, 1 / math.sqrt(L['D']), np64(gate))
    # q enters the products rounded to bf16: each score is off by at most 2^-8 smax more
    e = 2 * (2.0 ** -8 + (L['D'] + 4) * 2.0 ** -23) * smax[..., None] + 2.0 ** -15
    tol = half_step(BF) * np.abs(y0) + 1.01 * np.expm1(np.minimum(e, 50)) * mass
    d = np.abs(np64(y) - y0)
    assert (d <= tol).all(), float((d - tol).max())
    assert np.linalg.norm(d) <= 1e-2 * np.linalg.norm(y0)              # and the tensor as a whole


def test_prompt_then_decode_steps():
    """Prompts of three sequences, four decode steps, then a verify step, with an empty slot throughout."""
    N, cap = 4, 64
    L = _layer(1, N, cap)
    lens, step = np.array([0, 0, 0, 0]), 0
    for new in ([20, 7, 0, 33], [1] * 4, [1] * 4, [1] * 4, [1] * 4, [3, 3, 3, 3]):
        lens = lens + np.array(new)
        lens[2] = 0
        x = _step_inputs(L, 100 + step, sum(new))
        cu = cuts(new)
        y = _step(L, x, i32(lens), i32(cu) if step % 2 == 0 else (i32(cu) if len(set(new)) > 1 else None))
        gdn.check_device_error()
        _check_step(L, x, y, lens.tolist(), cu)
        step += 1


def test_decode_step_in_a_graph_on_a_side_stream_beside_another():
    """Two captured steps, each with a workspace of its own, replayed at the same time on two streams with
    new inputs and growing lengths."""
    N, cap = 5, 700
    Ls, xs, lens, ys, graphs = [], [], [], [], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    start = [[3, 600, 64, 17, 0], [640, 1, 5, 300, 31]]
    for i in range(2):
        L = _layer(10 + i, N, cap)
        L['c'].k.copy_(rand(20 + i, *L['c'].k.shape))
        L['c'].v.copy_(rand(30 + i, *L['c'].v.shape))
        x, n, out = _step_inputs(L, 40 + i, N), i32(start[i]), torch.zeros(N, 8, 128, dtype=BF, device='cuda')
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[i]):
            _step(L, x, n)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            _step(L, x, n, bufs=dict(o=out))
        Ls.append(L), xs.append(x), lens.append(n), ys.append(out), graphs.append(g)
    for rep in range(3):
        for i in range(2):
            lens[i].copy_(i32([n + 1 + rep if n else 0 for n in start[i]]))
            xs[i][0].copy_(rand(60 + 2 * rep + i, *xs[i][0].shape))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            _check_step(Ls[i], xs[i], ys[i], lens[i].tolist(), list(range(N + 1)))
    gdn.check_device_error()


def test_same_call_twice_is_bit_equal():
    lens = [5000, 17, 900, 0, 64]
    c = Cache(lens, 2, 16, 128, BF)
    c.k.copy_(rand(91, *c.k.shape))
    c.v.copy_(rand(92, *c.v.shape))
    q = rand(93, 5, 16, 128)
    y = run_attn(c, q, lens, [1] * 5)
    n = gdn.paged_attn_decode_workspace_size(5, 5, 16, 2, 128, BF, c.bt.shape[1] * c.P)
    ws = torch.full((n,), 255, dtype=torch.uint8, device='cuda')
    for _ in range(5):
        assert torch.equal(run_attn(c, q, lens, [1] * 5, workspace=ws), y)


def test_sequences_that_share_pages():
    """A common prefix: rows of the block table that name the same pages."""
    c = Cache([48, 48], 2, 16, 64, BF).fill([48, 48], 95)
    c.bt[1, :2] = c.bt[0, :2]
    c.block_table = i32(c.bt)
    check_attn(c, rand(96, 2, 8, 64), [40, 45], [1, 1])


@pytest.mark.parametrize('D,H,dtype', [(256, 2, BF), (128, 2, BF), (64, 2, BF), (256, 1, F32), (128, 1, F32)])
def test_long_contexts_back_to_back(D, H, dtype):
    """Many calls in flight on two caches, warps running ahead of one another over long ranges: every output is
    the first one's, bit for bit, and the first is right."""
    n = 131072 if dtype == BF else 30000
    cs = [Cache([n], H, 64, D, dtype, seed=s) for s in (1, 2)]
    for s, c in enumerate(cs):
        g = torch.Generator(device='cuda').manual_seed(s)
        c.k.normal_(generator=g)
        c.v.normal_(generator=g)
    q = rand(1, 1, 8 * H, D, dtype=dtype)
    first = [check_attn(c, q, [n], [1], out_dtype=dtype, cu=False) for c in cs]
    outs = [run_attn_async(c, q, n, dtype) for _ in range(100) for c in cs]
    gdn.check_device_error()
    for i, y in enumerate(outs):
        assert torch.equal(y, first[i % 2]), i


def run_attn_async(c, q, n, dtype):
    return gdn.paged_attn_decode(q, c.k, c.v, c.block_table, i32([n]), out_dtype=dtype)


def test_padded_strides():
    """Slots and heads apart by more than they hold, in both orders; what lies between is left as it was."""
    for order in ((0, 1, 2, 3), (0, 2, 1, 3)):                       # [page, head, slot, D] or [page, slot, head, D]
        H, P, D, lens = 2, 16, 64, [40, 17]
        c = Cache(lens, H, P, D, BF)
        shape = [c.pages, H, P, D]
        dims = [shape[i] for i in order]
        views = []
        for _ in range(2):
            raw = torch.full((dims[0], dims[1] + 1, dims[2] + 1, D + 8), float('nan'), dtype=BF, device='cuda')
            views.append((raw, raw[:, :dims[1], :dims[2], :D].permute(*order)))
        (kr, c.k), (vr, c.v) = views
        k, v, q = rand(1, 57, H, D), rand(2, 57, H, D), rand(3, 57, 8, D)
        gdn.paged_kv_append(k, v, c.k, c.v, c.block_table, i32(lens), cu_seqlens=i32([0, 40, 57]))
        check_attn(c, q, lens, lens)
        for raw, x in ((kr, k), (vr, v)):
            assert int((~raw.isnan()).sum()) == x.numel()


def test_nothing_to_attend_at_all():
    for n, width in ((1, 2), (5, 100)):
        c = Cache([width * 16] * n, 2, 16, 128, BF)
        o = torch.full((2 * n, 8, 128), 7.0, dtype=BF, device='cuda')
        gdn.paged_attn_decode(rand(1, 2 * n, 8, 128), c.k, c.v, c.block_table, i32([0] * n), o=o)
        gdn.check_device_error()
        assert not o.any()


def test_fewer_cached_than_new_and_negative_lengths():
    for dtype in (BF, F32):
        lens = [20, 20, 20]
        q = rand(81, 6, 4, 64, dtype=dtype)
        c = Cache(lens, 2, 16, 64, dtype).fill(lens, 82)
        y = run_attn(c, q, lens, [2] * 3, out_dtype=dtype)
        for bad in (1, -5):
            z = gdn.paged_attn_decode(q, c.k, c.v, c.block_table, i32([20, bad, 20]), out_dtype=dtype)
            with pytest.raises(RuntimeError, match='device error 3'):
                gdn.check_device_error()
            assert torch.equal(z[:2], y[:2]) and torch.equal(z[4:], y[4:]) and not z[2:4].any()


def test_no_tokens():
    c = Cache([16], 2, 16, 64, BF)
    e = torch.empty(0, 4, 64, dtype=BF, device='cuda')
    assert gdn.paged_attn_decode(e, c.k, c.v, c.block_table, i32([3])).shape == e.shape
    assert gdn.qk_norm_rope(e, e[:, :2])[0].shape == e.shape
    assert gdn.paged_kv_append(e[:, :2], e[:, :2], c.k, c.v, c.block_table, i32([3])) is None
    gdn.check_device_error()
    assert c.k.isnan().all()


def test_a_gate_of_another_type_is_refused_before_the_cache_changes():
    c = Cache([16], 2, 16, 64, BF)
    q, k = rand(1, 1, 4, 64, dtype=F32), rand(2, 1, 2, 64, dtype=F32)
    with pytest.raises(ValueError, match='gate'):
        gdn.attention_decode(q, k, k, c.k, c.v, c.block_table, i32([3]), gate=q)
    assert c.k.isnan().all()


@pytest.mark.parametrize('N', [161, 1000, 5000])
def test_more_sequences_than_threads(N):
    """Every sequence of a large batch of one-token rows returns its only value."""
    lens = [1 if s % 3 else 0 for s in range(N)]
    c = Cache([1] * N, 1, 8, 64, BF)
    v = rand(7, N, 1, 64)
    gdn.paged_kv_append(v, v, c.k, c.v, c.block_table, i32(lens))
    y = gdn.paged_attn_decode(rand(8, N, 2, 64), c.k, c.v, c.block_table, i32(lens))
    gdn.check_device_error()
    live = torch.tensor(lens, device='cuda').bool()
    assert torch.equal(y[live], v[live].expand(-1, 2, -1)) and not y[~live].any()
