"""Measured cases of the paged-attention operators: plain torch forms and the library's calls.

A case is one call: "op" says which operator, the rest are sizes.  ``own`` is set from outside:
false computes the plain form, true calls the library.  Sizes: 4096-token prefill, 256-sequence
decode, 16 sequences of 512..8192 tokens and a 131072-token context are the workloads of
inputs.py; head counts and head widths are generic.

Layouts: q [T, Nq, D], k and v [T, Nkv, D], caches [pages, Nkv, page, D], block_table [N, pages per
sequence] int32, kv_lens [N] int32 (cached tokens including the call's own), cos_sin [positions, r]
float32 (r/2 cosines, then r/2 sines).  New token i of n of a sequence has cache index
kv_len - n + i and sees the indices up to its own.
"""

import math
import random

import torch

own = False


# ------------------------------------------------------------------------------- the cases

def _rope(name, T, seqs, nq, nkv, d, rot, inter, norm, dtype):
    c = dict(op='rope', T=T, seqs=seqs, nq=nq, nkv=nkv, d=d, rot=rot, inter=inter, norm=norm, dtype=dtype)
    return dict(c, name=name) if name else c


def _append(name, seqs, lo, hi, new, nq, nkv, d, rot, inter, norm, page, dtype, len_seed):
    c = dict(op='append', seqs=seqs, lo=lo, hi=hi, new=new, nq=nq, nkv=nkv, d=d, rot=rot, inter=inter, norm=norm,
             page=page, dtype=dtype, len_seed=len_seed)
    return dict(c, name=name) if name else c


def _attn(name, seqs, lo, hi, new, nq, nkv, d, page, gate, dtype, len_seed):
    c = dict(op='attn', seqs=seqs, lo=lo, hi=hi, new=new, nq=nq, nkv=nkv, d=d, page=page, gate=gate, dtype=dtype,
             len_seed=len_seed)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence's decode step in a layer with partial rotation: latency of the smallest call
        _rope('rope_t1_d256', 1, 1, 16, 2, 256, 64, False, True, 'bf16'),
        # one 4096-token prompt, full rotation of 128-wide heads
        _rope('rope_t4096_d128', 4096, 1, 32, 8, 128, 128, False, True, 'bf16'),
        # a packed batch of odd lengths kept in float32, adjacent pairs rotated
        _rope('rope_varlen_f32', 1003, 5, 12, 4, 64, 32, True, True, 'f32'),
        # the decode step of 256 sequences: one new token each, q beside it
        _append('append_decode_b256', 256, 1, 128, 1, 16, 2, 256, 64, False, True, 64, 'bf16', 1),
        # the prompts of 16 sequences (ragged, new = 0: all of each sequence is new) into small pages
        _append('append_prompts_16seq', 16, 64, 512, 0, 32, 8, 128, 128, False, True, 16, 'bf16', 2),
        # draft + verify, three tokens of seven sequences, float32, pages of an odd size, no norm
        _append('append_verify_f32', 7, 3, 200, 3, 8, 4, 64, 64, True, False, 24, 'f32', 3),
        # one short chat turn: latency
        _attn('attn_b1_short', 1, 77, 77, 1, 16, 2, 256, 16, True, 'bf16', 4),
        # 256 sequences of ordinary lengths: the throughput case, about 4.5 GB of cache
        _attn('attn_b256', 256, 512, 8192, 1, 32, 8, 128, 64, False, 'bf16', 5),
        # one 131072-token context, two kv heads: everything hangs on the split over the length
        _attn('attn_b1_131072', 1, 131072, 131072, 1, 16, 2, 256, 64, True, 'bf16', 6),
        # draft + verify: four new tokens of 16 sequences
        _attn('attn_verify_16seq', 16, 512, 8192, 4, 16, 2, 256, 64, True, 'bf16', 7),
        # many short, ragged sequences, empty slots of a padded batch among them, three query heads to a kv head
        _attn('attn_ragged_short', 64, 0, 300, 1, 24, 8, 64, 16, False, 'bf16', 8),
        # float32 cache with pages that do not divide any tile
        _attn('attn_f32', 32, 100, 4000, 1, 8, 2, 128, 24, False, 'f32', 9),
    ]


_MOST = 256 * 8192 * 8 * 128          # cache elements (padded to the longest sequence) of attn_b256


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(['rope', 'append', 'attn', 'attn'])
    d = rng.choice([64, 128, 256])
    nkv = rng.choice([1, 2, 3, 4, 8])
    nq = nkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
    dtype = rng.choice(['bf16', 'bf16', 'bf16', 'f32'])
    rot = rng.choice([x for x in (0, 16, 32, 64, 96, 128, 256) if x <= d])
    inter, norm = rng.random() < 0.3, rng.random() < 0.8
    page = rng.choice([8, 16, 20, 32, 48, 64, 128, 256])
    if op == 'rope':
        T = _log_int(rng, 1, 4096)
        if not norm and rot == 0:
            norm = True
        return _rope(None, T, min(T, _log_int(rng, 1, 64)), nq, nkv, d, rot, inter, norm, dtype)
    if op == 'append':
        seqs = _log_int(rng, 1, 256)
        new = rng.choice([1, 1, 2, 3, 5, 0])
        hi = _log_int(rng, 8, 512 if seqs <= 16 else 128)
        return _append(None, seqs, max(1, new), hi, new, nq, nkv, d, rot, inter, norm, page, dtype, rng.randrange(1 << 20))
    seqs = _log_int(rng, 1, 256)
    new = rng.choice([1, 1, 1, 2, 3, 4, 6])
    most = min(131072, _MOST // (seqs * nkv * d * (2 if dtype == 'f32' else 1)) // max(1, nq * new // (8 * nkv)))
    hi = max(new, _log_int(rng, 16, max(16, most)))
    lo = rng.choice([0, hi // 16, hi])
    return _attn(None, seqs, lo, hi, new, nq, nkv, d, page, rng.random() < 0.5, dtype, rng.randrange(1 << 20))


# ------------------------------------------------------------------------------- the inputs

_DT = {'bf16': torch.bfloat16, 'f32': torch.float32}


def _lens(case):
    """Cached lengths (the call's tokens included); a drawn length below the new tokens' count is an empty slot."""
    r = random.Random(case['len_seed'])
    n = [r.randint(case['lo'], case['hi']) for _ in range(case['seqs'])]
    return [x if x >= case['new'] else 0 for x in n]


def _cuts(case):
    """Bounds of the packed sequences of a rope case."""
    r = random.Random(case['T'] * 131 + case['seqs'])
    inner = sorted(r.sample(range(1, case['T']), case['seqs'] - 1)) if case['seqs'] > 1 else []
    return [0] + inner + [case['T']]


def _table(positions, rot, device):
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * (1e6 ** (-2.0 * i / rot))
    return torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32)


def _norm_w(gen, case, dev):
    if not case['norm']:
        return None, None
    w = 1.0 + 0.1 * torch.randn(2, case['d'], generator=gen, device=dev)
    return w[0].contiguous(), w[1].contiguous()


def prepare(case, seed):
    dev = torch.device('cuda')
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[case['dtype']]

    def normal(*shape, std=1.0):
        x = torch.randn(*shape, generator=gen, device=dev, dtype=dt)
        return x if std == 1.0 else x.mul_(std)

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    nq, nkv, d = case['nq'], case['nkv'], case['d']
    st = dict(case=case, dt=dt)
    if case['op'] == 'rope':
        T, cuts = case['T'], _cuts(case)
        st.update(q=normal(T, nq, d, std=2.0), k=normal(T, nkv, d, std=2.0), cu=i32(cuts) if case['seqs'] > 1 else None)
        st['q_w'], st['k_w'] = _norm_w(gen, case, dev)
        st['table'] = _table(case['T'], case['rot'], dev) if case['rot'] else None
        return st
    lens = _lens(case)
    P = case['page']
    width = max(1, max((n + P - 1) // P for n in lens))
    used = sum((n + P - 1) // P for n in lens)
    pages = used + 3
    ids = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    at, rows = 0, []
    for n in lens:
        m = (n + P - 1) // P
        rows.append(torch.nn.functional.pad(ids[at:at + m], (0, width - m)))
        at += m
    st.update(kc=normal(pages, nkv, P, d), vc=normal(pages, nkv, P, d), bt=torch.stack(rows), lens=i32(lens))
    if case['op'] == 'append':
        new = [case['new'] or n for n in lens]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        T = cu[-1]
        st.update(q=normal(T, nq, d, std=2.0), k=normal(T, nkv, d, std=2.0), v=normal(T, nkv, d),
                  cu=None if case['new'] else i32(cu), table=_table(max(lens), case['rot'], dev) if case['rot'] else None)
        st['q_w'], st['k_w'] = _norm_w(gen, case, dev)
        return st
    T = case['seqs'] * case['new']
    st.update(q=normal(T, nq, d, std=1.5), gate=normal(T, nq, d) if case['gate'] else None)
    return st


# ------------------------------------------------------------------------------- one pass

def _norm_rope_plain(x, w, cs, inter):
    """x [T, H, D] -> float32; w [D] or None; cs [T, r] or None (the table rows of the tokens)."""
    u = x.float()
    if w is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-6) * w
    if cs is None:
        return u
    r = cs.shape[1]
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    if inter:
        a, b = u[..., 0:r:2], u[..., 1:r:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = u[..., :r // 2], u[..., r // 2:r]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, u[..., r:]], -1)


def _seq_of(cu, seqs, T):
    """Sequence and index within it of each of T packed tokens."""
    t = torch.arange(T, device='cuda')
    if cu is None:
        n = T // seqs
        return t // n, t % n
    s = torch.searchsorted(cu, t, right=True) - 1
    return s, t - cu[s]


def _rope_plain(st):
    case, dt = st['case'], st['dt']
    cs = None
    if st['table'] is not None:
        _, i = _seq_of(st['cu'], case['seqs'], case['T'])
        cs = st['table'][i]
    return (_norm_rope_plain(st['q'], st['q_w'], cs, case['inter']).to(dt),
            _norm_rope_plain(st['k'], st['k_w'], cs, case['inter']).to(dt))


def _append_plain(st):
    case, dt = st['case'], st['dt']
    s, i = _seq_of(st['cu'], case['seqs'], st['q'].shape[0])
    new = case['new'] or st['lens'][s]
    pos = (st['lens'][s] - new + i).long()
    cs = st['table'][pos] if st['table'] is not None else None
    page = st['bt'][s, pos // case['page']].long()
    st['kc'][page, :, pos % case['page']] = _norm_rope_plain(st['k'], st['k_w'], cs, case['inter']).to(dt)
    st['vc'][page, :, pos % case['page']] = st['v']
    return _norm_rope_plain(st['q'], st['q_w'], cs, case['inter']).to(dt), st['kc'], st['vc']


def _attn_plain(st):
    case = st['case']
    N, n, nkv, d, P = case['seqs'], case['new'], case['nkv'], case['d'], case['page']
    G = case['nq'] // nkv
    L = st['bt'].shape[1] * P
    bt = st['bt'].long()
    K = st['kc'][bt].transpose(1, 2).reshape(N, nkv, L, d).float()
    q = st['q'].float().reshape(N, n, nkv, G, d).transpose(1, 2).reshape(N, nkv, n * G, d)
    sc = (q @ K.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).reshape(N, nkv, n, G, L)
    del K
    # token i of n sees the cache indices up to len - n + i
    limit = st['lens'][:, None] - n + torch.arange(n, device='cuda')
    seen = torch.arange(L, device='cuda') <= limit[..., None]
    sc.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True).clamp_min(-1e30)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    V = st['vc'][bt].transpose(1, 2).reshape(N, nkv, L, d).float()
    o = p.reshape(N, nkv, n * G, L) @ V
    del V
    o = o.reshape(N, nkv, n, G, d) / l.clamp_min(1e-30)
    o = o.transpose(1, 2).reshape(N * n, nkv * G, d)
    if st['gate'] is not None:
        o = o * torch.sigmoid(st['gate'].float())
    return o.to(st['dt'])


def run(st):
    case = st['case']
    if own:
        from gated_deltanet_linear_conv_gb300 import gdn
        if case['op'] == 'rope':
            return gdn.qk_norm_rope(st['q'], st['k'], cos_sin=st['table'], q_norm_w=st['q_w'], k_norm_w=st['k_w'],
                                    cu_seqlens=st['cu'], interleaved=case['inter'], out_dtype=st['dt'])
        if case['op'] == 'append':
            q = gdn.paged_kv_append(st['k'], st['v'], st['kc'], st['vc'], st['bt'], st['lens'], q=st['q'],
                                    cos_sin=st['table'], q_norm_w=st['q_w'], k_norm_w=st['k_w'], cu_seqlens=st['cu'],
                                    interleaved=case['inter'], out_dtype=st['dt'])
            return q, st['kc'], st['vc']
        return gdn.paged_attn_decode(st['q'], st['kc'], st['vc'], st['bt'], st['lens'], gate=st['gate'],
                                     out_dtype=st['dt'])
    return {'rope': _rope_plain, 'append': _append_plain, 'attn': _attn_plain}[case['op']](st)


# ------------------------------------------------------------------------------- work and 64-bit values

def work(case):
    es = 2 if case['dtype'] == 'bf16' else 4
    nq, nkv, d = case['nq'], case['nkv'], case['d']
    if case['op'] == 'rope':
        T = case['T']
        return dict(bytes=2 * T * (nq + nkv) * d * es + 4 * max(b - a for a, b in zip(_cuts(case), _cuts(case)[1:])) * case['rot'],
                    flops=10.0 * T * (nq + nkv) * d)
    lens = _lens(case)
    if case['op'] == 'append':
        T = sum(case['new'] or n for n in lens)
        return dict(bytes=2 * T * (nq + 2 * nkv) * d * es + 4 * min(T, max(lens)) * case['rot'] + 4 * T,
                    flops=10.0 * T * (nq + nkv) * d)
    T = case['seqs'] * case['new']
    return dict(bytes=2 * sum(lens) * nkv * d * es + (3 if case['gate'] else 2) * T * nq * d * es + 4 * sum(lens) // case['page'],
                flops=4.0 * sum(lens) * case['new'] * nq * d)


def _exact_rows(x, w, pos, table, inter):
    """One row set in 64 bits: complex multiplication by cos + i sin of each pair."""
    u = x.double()
    if w is not None:
        u = u / (u.pow(2).sum(-1, keepdim=True) / u.shape[-1] + 1e-6).sqrt() * w.double()
    if table is None:
        return u
    h = table.shape[1] // 2
    rot = torch.complex(table[pos, :h].double(), table[pos, h:].double()).unsqueeze(1)
    out = u.clone()
    if inter:
        z = torch.view_as_complex(u[..., :2 * h].reshape(*u.shape[:-1], h, 2).contiguous()) * rot
        out[..., :2 * h] = torch.view_as_real(z).reshape(*u.shape[:-1], 2 * h)
    else:
        z = torch.complex(u[..., :h], u[..., h:2 * h]) * rot
        out[..., :h], out[..., h:2 * h] = z.real, z.imag
    return out


def exact(case, seed):
    if case['op'] == 'attn' and work(case)['flops'] > 4e12:
        return None                                   # over 20 seconds of 64-bit products
    st = prepare(case, seed)
    if case['op'] == 'rope':
        cuts = _cuts(case)
        pos = torch.tensor([i for a, b in zip(cuts, cuts[1:]) for i in range(b - a)], device='cuda')
        return tuple(_exact_rows(st[x], st[x + '_w'], pos, st['table'], case['inter']) for x in 'qk')
    lens, P = _lens(case), case['page']
    bt = st['bt'].tolist()
    if case['op'] == 'append':
        where = [(s, p) for s, n in enumerate(lens) for p in range(n - (case['new'] or n), n)]
        pos = torch.tensor([p for _, p in where], device='cuda')
        page = torch.tensor([bt[s][p // P] for s, p in where], device='cuda')
        q, k = (_exact_rows(st[x], st[x + '_w'], pos, st['table'], case['inter']) for x in 'qk')
        kc, vc = st['kc'].double(), st['vc'].double()
        kc[page, :, pos % P] = k
        vc[page, :, pos % P] = st['v'].double()
        return q, kc, vc
    n, G, d = case['new'], case['nq'] // case['nkv'], case['d']
    out = torch.zeros(case['seqs'] * n, case['nq'], d, dtype=torch.float64, device='cuda')
    for s, L in enumerate(lens):
        if L == 0:
            continue
        pages = st['bt'][s, :(L + P - 1) // P].long()
        for h in range(case['nkv']):
            K = st['kc'][pages, h].reshape(-1, d)[:L].double()
            V = st['vc'][pages, h].reshape(-1, d)[:L].double()
            for i in range(n):
                e = L - n + i + 1
                q = st['q'][s * n + i, h * G:(h + 1) * G].double()
                a = torch.softmax(q @ K[:e].T / math.sqrt(d), -1)
                out[s * n + i, h * G:(h + 1) * G] = a @ V[:e]
    if st['gate'] is not None:
        out = out / (1.0 + torch.exp(-st['gate'].double()))
    return out
