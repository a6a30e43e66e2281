"""The cache calls on the GPU against plain 64-bit forms: plan, norm and rotation,
append, attention, and whole rounds of them with the verify calls.

Tolerances.  A bf16 result is rounded once: half a step, 2^-8 of its value.
Norm and rotation in f32: the mean of squares carries at most 13 roundings,
halved by the root; rsqrt, the products, the reduced angle (pi 2^-24 + 2^-23) and
the rotation's sum bring the total below 2^-19 of |a| + |b|.  Attention: a score is
a sum of D + 8 f32 products or less, so it is off by at most
(D + 8) 2^-23 scale sum|q||k| (twice the half step, for truncating sums); the probabilities are rounded to f16
(2^-11) before the second product; the output's error is at most that relative
error of each probability times sum p|v|, plus the final rounding.  f16 has no
steps below 2^-24: with the keys' value scales s_j, the kernel rounds
P_j = 2^11 p_j s_j / max(p s) (or more), so below f16's normal numbers p_j s_j is
off by up to 2^-25 / 2^11 of max(p s); the sum over keys of that times
|v_j| / s_j is 2^-36 max(p s) sum |v| / s.  And a query (and a key that is not yet
in 8 bits) may be held as two e4m3 rows: exact but for its elements below 2^-9 of its
largest, which are rounded at 2^-10 of e4m3's scale; the products of that with
the other side are added to a score's error.
"""
import math

import numpy as np
import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def spec(cuda_device):
    import speculative_decoding_verify_temperature_b200 as s
    return s


def gpu(x):
    return torch.as_tensor(x).cuda()


def flagged(spec, ws):
    return bool(spec.spec_read_device_status(ws) & (1 << 4))


def workspace(spec, B=1, N=1, Hq=8, D=128):
    ws = torch.empty(spec.spec_cache_workspace_bytes(B, N, Hq, D), dtype=torch.uint8, device="cuda")
    spec.spec_workspace_init(ws)
    return ws


# ----------------------------------------------------------------------------- plan

@pytest.mark.parametrize("B,N,depth,back", [(1, 1, 0, 8), (3, 2, 64, 8), (5, 31, 64, 3), (4, 32, 64, 8), (4, 33, 64, 1),
                                            (7, 64, 16, 8), (2, 65, 64, 1), (2, 255, 64, 8), (130, 256, 64, 30)])
def test_plan_matches_the_climb(spec, B, N, depth, back):
    rs = np.random.RandomState(B * 1000 + N)
    parents = ref.random_parents(B, N, rs, depth, back)
    lengths = rs.randint(0, 100000, size=B).astype(np.int32)
    lengths[B // 2] = -1 if B > 2 else 0
    pos, words = spec.spec_tree_plan(gpu(parents), gpu(lengths), depth)
    epos, ewords = ref.plan(parents, lengths)
    assert np.array_equal(pos.cpu().numpy(), epos)
    assert np.array_equal(words.cpu().numpy(), ewords)


@pytest.mark.parametrize("N", [1, 6, 33, 256])
def test_plan_of_chains(spec, N):
    lengths = gpu(np.array([0, 7, -1], dtype=np.int32))
    pos, words = spec.spec_tree_plan(None, lengths, 0, N=N)
    chain = np.tile(np.arange(-1, N - 1, dtype=np.int32), (3, 1))
    epos, ewords = ref.plan(chain, [0, 7, -1])
    assert np.array_equal(pos.cpu().numpy(), epos) and np.array_equal(words.cpu().numpy(), ewords)


def test_plan_rejects_malformed_trees(spec):
    base = np.tile(np.arange(-1, 7, dtype=np.int32), (7, 1))
    base[1, 0] = 0                      # root with a parent
    base[2, 3] = 3                      # its own parent
    base[3, 4] = 6                      # a later node
    base[4, 5] = -1                     # a second root
    base[5, 2] = 1 << 30
    lengths = np.array([5, 5, 5, 5, 5, 5, 1 << 30], dtype=np.int32)
    ws = workspace(spec)
    pos, words = spec.spec_tree_plan(gpu(base), gpu(lengths), 7, workspace=ws)
    assert (pos[1:] == -1).all() and (words[1:] == 0).all() and flagged(spec, ws)
    assert pos[0].tolist() == list(range(5, 13))
    pos, _ = spec.spec_tree_plan(gpu(base[:1]), gpu(lengths[:1]), 6, workspace=ws)
    assert (pos == -1).all() and flagged(spec, ws)          # deeper than max_depth
    spec.spec_tree_plan(gpu(base[:1]), gpu(lengths[:1]), 7, workspace=ws)
    assert not flagged(spec, ws)


# ----------------------------------------------------------------------------- norm + rotation

NR = [  # B, N, Hq, Hk, D, rot, dtype, interleaved, weights
    (1, 1, 32, 8, 128, 128, BF, False, True), (2, 6, 7, 1, 64, 64, BF, False, True),
    (3, 33, 24, 6, 96, 48, torch.float32, True, False), (2, 5, 12, 4, 96, 96, BF, False, True),
    (1, 9, 3, 3, 256, 128, BF, True, True), (5, 2, 1, 1, 8, 0, torch.float32, False, True),
    (2, 3, 5, 5, 16, 16, torch.float32, False, True), (1, 4, 70, 10, 128, 64, torch.float32, False, True),
    (2, 3, 2, 2, 48, 32, BF, False, False), (700, 2, 4, 1, 128, 128, BF, False, True)]


def check_norm_rope(x, y, pos, freq, w, eps, inter):
    e, mag = ref.norm_rope(x.cpu(), pos.cpu(), None if freq is None else freq.cpu(), None if w is None else w.cpu(), eps,
                           inter)
    e = torch.where((pos.cpu() < 0)[..., None, None], torch.zeros_like(e), e)
    tol = e.abs() * (2.0 ** -8 if x.dtype == BF else 2.0 ** -24) + mag * 2.0 ** -19 + 1e-37
    assert ((y.cpu().double() - e).abs() <= tol).all()


@pytest.mark.parametrize("B,N,Hq,Hk,D,rot,dt,inter,weights", NR)
def test_norm_rope(spec, B, N, Hq, Hk, D, rot, dt, inter, weights):
    g = torch.Generator("cuda").manual_seed(B * 100 + N)
    q = torch.randn((B, N, Hq, D), generator=g, device="cuda").to(dt)
    k = (torch.randn((B, N, Hk, D), generator=g, device="cuda") * 30).to(dt)
    pos = torch.randint(0, 1 << 20, (B, N), generator=g, device="cuda", dtype=torch.int32)
    pos.view(-1)[0] = 0
    pos.view(-1)[-1] = (1 << 30) if B * N > 1 else 0
    if B > 1:
        pos[1] = -1
    freq = gpu(ref.inv_freq(rot)) if rot else None
    qw = torch.randn((D,), generator=g, device="cuda").to(dt) if weights else None
    kw = torch.randn((D,), generator=g, device="cuda").to(dt) if weights else None
    a, b = spec.spec_qk_norm_rope(q, k, pos, freq, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter)
    check_norm_rope(q, a, pos, freq, qw, 1e-5, inter)
    check_norm_rope(k, b, pos, freq, kw, 1e-5, inter)
    # one weight only, of the other type
    other = None if qw is None else qw.float()
    a2, b2 = spec.spec_qk_norm_rope(q, k, pos, freq, q_weight=other, eps=1e-5, interleaved=inter)
    check_norm_rope(q, a2, pos, freq, other, 1e-5, inter)
    check_norm_rope(k, b2, pos, freq, None, 1e-5, inter)


def test_norm_rope_strided_in_place(spec):
    """Rows inside a packed projection, written back where they lie: what is between them stays."""
    B, N, Hq, Hk, D = 3, 5, 6, 2, 64
    qkv = torch.randn((B, N, (Hq + 2 * Hk) * D), device="cuda").to(BF)
    was = qkv.clone()
    view = lambda t: (t[..., :Hq * D].unflatten(-1, (Hq, D)), t[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)))  # noqa: E731
    q, k = view(qkv)
    pos = torch.randint(0, 5000, (B, N), device="cuda", dtype=torch.int32)
    freq, w = gpu(ref.inv_freq(D)), torch.rand((D,), device="cuda").to(BF)
    e = spec.spec_qk_norm_rope(*view(was), pos, freq, q_weight=w, k_weight=w)
    a = spec.spec_qk_norm_rope(q, k, pos, freq, q_weight=w, k_weight=w, q_out=q, k_out=k)
    assert a[0] is q and torch.equal(q, e[0]) and torch.equal(k, e[1])
    assert torch.equal(qkv[..., (Hq + Hk) * D:], was[..., (Hq + Hk) * D:])
    # head-major tensors (transposed views) give the same
    qt, kt = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in view(was))
    b = spec.spec_qk_norm_rope(qt, kt, pos, freq, q_weight=w, k_weight=w)
    assert torch.equal(b[0], e[0]) and torch.equal(b[1], e[1])


def test_norm_rope_large_and_tiny_rows(spec):
    """A row of zeros stays zero; NaN stays in its head row."""
    D = 128
    q = torch.randn((1, 2, 4, D), device="cuda").to(BF)
    q[0, 0, 1] = 0
    q[0, 1, 2, 5] = float("nan")
    k = (torch.randn((1, 2, 1, D), device="cuda") * 1e-20).to(BF)
    pos = torch.tensor([[3, 4]], dtype=torch.int32, device="cuda")
    w = torch.ones(D, device="cuda", dtype=BF)
    a, b = spec.spec_qk_norm_rope(q, k, pos, gpu(ref.inv_freq(D)), q_weight=w, k_weight=w)
    assert (a[0, 0, 1] == 0).all() and torch.isnan(a[0, 1, 2]).all()
    ok = torch.ones((1, 2, 4), dtype=torch.bool)
    ok[0, 1, 2] = False
    assert torch.isfinite(a[ok.cuda()]).all() and torch.isfinite(b).all()


# ----------------------------------------------------------------------------- append

def make_cache(spec, B, Hkv, D, page, blocks, rs, slots=None, extra=3):
    P = B * blocks + extra
    ids = rs.permutation(P)[:B * blocks].astype(np.int32).reshape(B, blocks)
    ns = None
    if slots is not None:
        ns, slots = B + 4, gpu(np.asarray(slots, dtype=np.int32))
    return spec.KvCache.allocate(P, Hkv, page, D, gpu(ids), torch.zeros(B, dtype=torch.int32, device="cuda"), slots, ns)


def same_cache(c, r, exact=True):
    """The GPU cache holds what the CPU one says, byte for byte."""
    lengths, table = c.lengths.cpu().tolist(), c.page_table.cpu().long()
    slots = range(c.B) if c.slots is None else c.slots.cpu().tolist()
    for b in range(c.B):
        assert lengths[b] == r.length(b)
        n = lengths[b] // c.page_size
        for which, (pages, scale, ring) in enumerate(((c.k_pages, c.k_scale, c.k_open), (c.v_pages, c.v_scale, c.v_open))):
            eb, es = r.blocks(b, which)
            assert torch.equal(pages.view(torch.uint8).cpu()[table[b, :n]], eb)
            assert torch.equal(scale.cpu()[table[b, :n]].double(), es)
            at = torch.arange(n * c.page_size, lengths[b]) % (2 * c.page_size)
            assert torch.equal(ring.view(torch.int16).cpu()[slots[b]][:, at].transpose(0, 1),
                               r.open_rows(b, which).view(torch.int16))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", [BF, torch.float32])
def test_append_rows_any_split(spec, page, D, dt):
    """Prompts, single rows, accepted paths, block borders: the cache is what the rows are, however they came."""
    B, Hkv, rs = 5, 3, np.random.RandomState(page + D)
    c = make_cache(spec, B, Hkv, D, page, 9, rs, slots=[4, 0, 8, 2, 5])
    r = ref.Cache(B, Hkv, D, page)
    ws = workspace(spec)
    for step, T in enumerate([1, page - 1, 2, 3 * page + 1, 17, page, page + 1, 5, 2 * page - 1]):
        k = (torch.randn((B, T, Hkv, D)) * torch.exp(3 * torch.randn(B, 1, Hkv, 1))).to(dt)
        v = torch.randn((B, T, Hkv, D)).to(dt)
        if step == 4:
            k[0], v[1] = 0, 0                                     # blocks that may hold nothing but zeros
        count = np.array([T, T, rs.randint(0, T + 1), 0, rs.randint(0, T + 1)], dtype=np.int32)
        room = [9 * page + page - 1 - r.length(b) for b in range(B)]
        count = np.minimum(count, room).astype(np.int32)
        index = None
        if step % 2:
            index = np.full((B, T), -7, dtype=np.int32)           # entries past the count are not read
            for b in range(B):
                index[b, :count[b]] = rs.permutation(T)[:count[b]]
        spec.spec_kv_append(k.cuda(), v.cuda(), gpu(count - 1), c, accept_index=None if index is None else gpu(index),
                            workspace=ws)
        for b in range(B):
            i = np.arange(count[b]) if index is None else index[b, :count[b]]
            r.append(b, k[b, i], v[b, i])
        same_cache(c, r)
    assert not flagged(spec, ws)


@pytest.mark.parametrize("page,D,rot,inter,weights,dt", [(16, 128, 128, False, True, BF), (64, 64, 32, False, True, torch.float32),
                                                         (128, 128, 128, True, False, BF), (32, 64, 64, True, True, BF),
                                                         (128, 128, 64, False, False, torch.float32)])
def test_append_norms_and_rotates(spec, page, D, rot, inter, weights, dt):
    """Raw keys, normed and rotated on the way: within the roundings to bf16 and e4m3 of the formula."""
    B, Hkv, T = 3, 2, 2 * page + 7
    c = make_cache(spec, B, Hkv, D, page, 4, np.random.RandomState(1))
    start = [0, page - 1, 5]
    w = (torch.rand(D) + 0.5).to(dt) if weights else None
    freq = ref.inv_freq(rot)
    rows = [[], []]
    for n, first in ((max(start), True), (T, False)):
        k, v = (torch.randn(B, n, Hkv, D) * 2).to(dt), torch.randn(B, n, Hkv, D).to(dt)
        cnt = start if first else [T] * B
        before = [0] * B if first else start
        spec.spec_kv_append(k.cuda(), v.cuda(), gpu(np.array(cnt, dtype=np.int32) - 1), c, inv_freq=freq.cuda(),
                            k_weight=None if w is None else w.cuda(), eps=1e-6, interleaved=inter)
        rows[0].append([ref.norm_rope(k[b, :cnt[b]], torch.arange(before[b], before[b] + cnt[b]), freq, w, 1e-6, inter)
                        for b in range(B)])
        rows[1].append([(v[b, :cnt[b]].double(), v[b, :cnt[b]].double().abs()) for b in range(B)])
    for b in range(B):
        total = start[b] + T
        assert int(c.lengths[b]) == total
        n = total // page
        for which, (pages, scale, ring) in enumerate(((c.k_pages, c.k_scale, c.k_open), (c.v_pages, c.v_scale, c.v_open))):
            e = torch.cat([rows[which][i][b][0] for i in range(2)])
            mag = torch.cat([rows[which][i][b][1] for i in range(2)])
            bf = e.abs() * 2.0 ** -8 + mag * 2.0 ** -19
            at = torch.arange(n * page, total) % (2 * page)
            assert ((ring[b][:, at].transpose(0, 1).cpu().double() - e[n * page:]).abs() <= bf[n * page:]).all()
            ids = c.page_table[b, :n].long().cpu()
            s = scale.cpu()[ids].double()
            got = pages.view(torch.uint8).cpu()[ids].view(F8).double() * s[..., None, None]
            e, bf = (x[:n * page].view(n, page, Hkv, D).transpose(1, 2) for x in (e, bf))
            assert ((got - e).abs() <= (e.abs() + bf) * 2.0 ** -4 + bf + s[..., None, None] * 2.0 ** -10).all()
            amax = e.abs().amax((2, 3))
            slack = 1 + 2.0 ** -7
            assert (amax <= 448 * s * slack).all() and (amax * slack > 224 * s).all()
            assert torch.equal(torch.frexp(s)[0], torch.full_like(s, 0.5))


def test_append_leaves_bad_sequences_alone(spec):
    """Bad pages, slots, rows, counts and lengths: that sequence keeps its cache and gets length -1."""
    B, Hkv, D, page = 9, 2, 64, 16
    c = make_cache(spec, B, Hkv, D, page, 2, np.random.RandomState(0), slots=list(range(B)))
    k = torch.randn(B, 20, Hkv, D).to(BF)
    ws = workspace(spec)
    c.lengths.copy_(gpu(np.array([3, 3, 3, 3, 3, 30, -5, 3, 1 << 30], dtype=np.int32)))
    c.page_table[1, 0] = c.k_pages.shape[0]
    c.page_table[2, 0] = -1
    c.slots[3] = B + 4
    index = np.tile(np.arange(20, dtype=np.int32), (B, 1))
    index[4, 13] = 20
    num = np.full(B, 14, dtype=np.int32)
    num[5] = 18                          # 30 + 19 tokens: above 2 pages and an open block
    num[7] = 20                          # more rows than the path has
    before = [t.clone() for t in (c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8), c.k_scale, c.v_scale, c.k_open,
                                  c.v_open)]
    out = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    spec.spec_kv_append(k.cuda(), k.cuda(), gpu(num), c, accept_index=gpu(index), out_lengths=out, workspace=ws)
    assert out.tolist() == [18, -1, -1, -1, -1, -1, -5, -1, -1] and flagged(spec, ws)
    after = (c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8), c.k_scale, c.v_scale, c.k_open, c.v_open)
    mine = int(c.page_table[0, 0])
    for i, (x, y) in enumerate(zip(before, after)):
        keep = torch.ones(x.shape[0], dtype=torch.bool, device="cuda")
        keep[mine if i < 4 else 0] = False
        assert torch.equal(x[keep], y[keep])
    # nothing to append: lengths as they were, no flag
    out = spec.spec_kv_append(k.cuda(), k.cuda(), torch.full((B,), -1, dtype=torch.int32, device="cuda"),
                              c.batch(c.page_table, torch.arange(B, dtype=torch.int32, device="cuda"), gpu(np.arange(B, dtype=np.int32))),
                              workspace=ws)
    assert out.tolist() == list(range(B)) and not flagged(spec, ws)


def test_append_non_finite(spec):
    """NaN and infinities stay what they are in the ring and become NaN in a page; the scale is the finite values'."""
    k = torch.randn(1, 20, 1, 64).to(BF)
    k[0, 3, 0, 5], k[0, 4, 0, 6], k[0, 18, 0, 1] = float("inf"), float("nan"), float("-inf")
    v = torch.full((1, 20, 1, 64), float("nan"), dtype=BF)
    c = make_cache(spec, 1, 1, 64, 16, 2, np.random.RandomState(0))
    spec.spec_kv_append(k.cuda(), v.cuda(), None, c)
    r = ref.Cache(1, 1, 64, 16)
    r.append(0, k[0], v[0])
    pid = int(c.page_table[0, 0])
    e, s = r.blocks(0, 0)
    assert torch.equal(c.k_pages[pid].view(torch.uint8).cpu() & 0x7F, e[0] & 0x7F) and float(c.k_scale[pid, 0]) == float(s[0, 0])
    assert (c.v_pages[pid].view(torch.uint8) & 0x7F == 0x7F).all() and float(c.v_scale[pid, 0]) == 1.0
    assert float(c.k_open[0, 0, 18, 1]) == -math.inf and torch.isnan(c.v_open[0, 0, 16:20]).all()


def test_append_tiny_and_huge_blocks(spec):
    """Magnitudes at both ends of bf16: scales stay normal f32 numbers."""
    c = make_cache(spec, 4, 1, 64, 16, 1, np.random.RandomState(0))
    k = torch.randn(4, 16, 1, 64)
    k = torch.stack([k[0] * 2.0 ** -128, k[1] * 1e38 / k[1].abs().max() * 3, k[2] * 2.0 ** -120, k[3]]).to(BF)
    spec.spec_kv_append(k.cuda(), k.cuda(), None, c)
    r = ref.Cache(4, 1, 64, 16)
    for b in range(4):
        r.append(b, k[b], k[b])
    same_cache(c, r)


# ----------------------------------------------------------------------------- attention

def attention_inputs(spec, B, N, Hq, Hkv, D, page, lengths, seed, slots=None, kscale=1.0, tree=True):
    g = torch.Generator().manual_seed(seed)
    rs = np.random.RandomState(seed)
    blocks = max(max(lengths) // page, 0)
    c = make_cache(spec, B, Hkv, D, page, blocks, rs, slots=slots)
    r = ref.Cache(B, Hkv, D, page)
    T = max(max(lengths), 1)
    k = (torch.randn((B, T, Hkv, D), generator=g) * torch.exp(torch.randn((B, T, Hkv, 1), generator=g)) * kscale).to(BF)
    v = (torch.randn((B, T, Hkv, D), generator=g) * torch.exp(2 * torch.randn((B, T, Hkv, 1), generator=g))).to(BF)
    spec.spec_kv_append(k.cuda(), v.cuda(), gpu(np.maximum(lengths, 0).astype(np.int32) - 1), c)
    c.lengths.copy_(gpu(np.array(lengths, dtype=np.int32)))
    for b in range(B):
        r.append(b, k[b, :max(lengths[b], 0)], v[b, :max(lengths[b], 0)])
    q = torch.randn((B, N, Hq, D), generator=g).to(BF)
    nk, nv = torch.randn((B, N, Hkv, D), generator=g).to(BF), torch.randn((B, N, Hkv, D), generator=g).to(BF)
    parents = ref.random_parents(B, N, rs) if tree else np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1))
    mask = ref.unpack(torch.from_numpy(ref.plan(parents, np.zeros(B, dtype=np.int32))[1]), N)
    return c, r, q, nk, nv, mask


def check_attention(r, lengths, q, k, v, mask, out, lse, scale):
    out, lse = out.cpu().double(), lse.cpu().double()
    for b in range(q.shape[0]):
        if lengths[b] < 0:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        side, vscale = [], None
        for which in range(2):
            e, s = r.blocks(b, which)
            vscale = torch.cat((s.repeat_interleave(r.page, 0), ref.row_scale(r.open_rows(b, which).double())))
            full = (e.view(F8).double() * s[..., None, None]).transpose(1, 2).reshape(-1, r.H, r.D)
            side.append(torch.cat((full, r.open_rows(b, which).double())))
        full = max(lengths[b], 0) // r.page * r.page
        e, el, pv, mag, small, lost = ref.attention(q[b].double(), k[b].double(), v[b].double(), *side, mask[b], scale, vscale, full)
        ds = (r.D + 8) * 2.0 ** -23 * mag + lost
        # the probabilities' own rounding, the scores' (in numerator and sum), the exponentials' (2^-21)
        rel = 2.0 ** -11 + 2 * ds + 2.0 ** -20
        tol = e.abs() * 2.0 ** -8 + pv * rel[..., None] + small * 2.0 ** -36 + 1e-38
        assert ((out[b] - e).abs() <= tol).all(), float(((out[b] - e).abs() / tol).max())
        empty = el == -math.inf
        assert torch.equal(lse[b] == -math.inf, empty)
        assert ((lse[b] - el)[~empty].abs() <= (ds + 2.0 ** -20 * (1 + el.abs()))[~empty]).all()


ATT = [  # B, N, Hq, Hkv, D, page, lengths
    (1, 1, 1, 1, 64, 16, [0]), (1, 1, 8, 1, 128, 16, [1]), (3, 1, 32, 8, 128, 16, [15, 16, 17]),
    (4, 1, 7, 1, 128, 64, [1000, 64, 63, 129]), (2, 1, 16, 16, 64, 32, [257, 31]),
    (3, 6, 8, 1, 128, 16, [127, 128, 300]), (2, 6, 24, 8, 64, 128, [128, 500]), (2, 17, 3, 3, 128, 32, [33, 0]),
    (5, 3, 10, 2, 128, 64, [-1, 0, 200, -1, 64]), (2, 33, 8, 2, 128, 16, [129, 16]), (1, 64, 16, 2, 128, 32, [513]),
    (2, 32, 8, 2, 64, 128, [1023, 1]), (1, 64, 5, 1, 64, 16, [100]), (1, 256, 2, 1, 128, 64, [130]),
    (1, 129, 2, 2, 128, 128, [127]), (1, 31, 64, 2, 128, 64, [333]), (3, 43, 3, 1, 128, 16, [0, 47, 1]),
    (1, 2, 64, 1, 128, 16, [2050]), (1, 1, 129, 1, 64, 16, [40]), (2, 256, 8, 4, 64, 32, [65, 31]),
    (40, 6, 64, 8, 128, 16, [(i * 397) % 1501 for i in range(40)]),      # many tiles and items per CTA
    (24, 33, 64, 8, 128, 32, [(i * 211) % 900 for i in range(24)]), (20, 32, 32, 8, 64, 128, [(i * 533) % 2000 for i in range(20)]),
    (48, 2, 40, 8, 64, 64, [(i * 97) % 700 - 20 for i in range(48)]), (60, 1, 32, 8, 128, 16, [(i * 397) % 3001 for i in range(60)]),
    (70, 1, 7, 1, 128, 16, [(i * 397) % 3001 for i in range(70)]), (30, 7, 15, 5, 64, 32, [(i * 211) % 900 for i in range(30)]),
    (9, 5, 12, 4, 128, 16, [5, 4000, 17, 1, 90, 2222, 0, 64, 800])]


@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,lengths", ATT)
def test_attention(spec, B, N, Hq, Hkv, D, page, lengths):
    c, r, q, k, v, mask = attention_inputs(spec, B, N, Hq, Hkv, D, page, lengths, 100 * B + N)
    ws = workspace(spec, B, N, Hq, D)
    for scale in (None, 0.5):
        out, lse = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda(), scale=scale,
                                            return_lse=True, workspace=ws)
        check_attention(r, lengths, q, k, v, mask, out, lse, 1 / math.sqrt(D) if scale is None else scale)
    assert not flagged(spec, ws)
    again, lse2 = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda(), scale=0.5,
                                           return_lse=True, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)      # the same bits every time


@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,lengths", [
    (48, 6, 64, 8, 128, 16, [(i * 397) % 701 for i in range(48)]), (100, 20, 8, 4, 64, 16, [i % 40 - 1 for i in range(100)]),
    (12, 256, 4, 2, 128, 32, [(i * 37) % 300 for i in range(12)]), (40, 3, 8, 1, 128, 128, [(i * 131) % 1200 for i in range(40)]),
    (1, 40, 32, 4, 128, 64, [9000]), (150, 1, 8, 2, 128, 16, [(i * 29) % 90 for i in range(150)])])
def test_attention_waits_end(spec, B, N, Hq, Hkv, D, page, lengths):
    """Many short items, tails only, items cut over many blocks: no wait gives up (the status word stays 0), call after call."""
    c, r, q, k, v, mask = attention_inputs(spec, B, N, Hq, Hkv, D, page, lengths, 7 * B + N)
    ws = workspace(spec, B, N, Hq, D)
    args = (q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda())
    outs = [spec.spec_tree_attention(*args, return_lse=True, workspace=ws) for _ in range(20)]
    assert spec.spec_read_device_status(ws) == 0
    check_attention(r, lengths, q, k, v, mask, *outs[0], 1 / math.sqrt(D))
    assert all(torch.equal(o, outs[0][0]) and torch.equal(e, outs[0][1]) for o, e in outs)


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 8, 2, 128), (6, 4, 2, 64), (40, 8, 2, 128), (130, 2, 1, 128)])
def test_attention_any_mask(spec, N, Hq, Hkv, D):
    """Arbitrary masks, rows without any key among them, chains without a mask, slots in another order."""
    lengths = [0, 50, 0, 200]
    c, r, q, k, v, _ = attention_inputs(spec, 4, N, Hq, Hkv, D, 16, lengths, N, slots=[6, 1, 7, 0])
    mask = torch.rand(4, N, N, generator=torch.Generator().manual_seed(N)) < 0.3
    mask[0, N // 2] = False
    mask[1, 0] = False
    mask[2] = False
    out, lse = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda(), return_lse=True)
    check_attention(r, lengths, q, k, v, mask, out, lse, 1 / math.sqrt(D))
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()
    # bits past the last node are not read
    if N % 32:
        junk = ref.pack(mask)
        junk[..., -1] |= torch.tensor(-(1 << (N % 32)), dtype=torch.int32)
        out2 = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, junk.cuda())
        assert torch.equal(out, out2)
    chain = torch.tril(torch.ones(N, N, dtype=torch.bool)).expand(4, N, N)
    out, lse = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, None, return_lse=True)
    check_attention(r, lengths, q, k, v, chain, out, lse, 1 / math.sqrt(D))
    out2 = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(chain).cuda())
    assert torch.equal(out, out2)


@pytest.mark.parametrize("qs,ks", [(30.0, 1.0), (1.0, 100.0), (1e-6, 1.0), (0.0, 1.0), (2.0 ** 60, 2.0 ** -60), (2.0 ** -70, 2.0 ** 70)])
@pytest.mark.parametrize("N,Hq", [(1, 4), (20, 8), (64, 16)])
def test_attention_magnitudes(spec, qs, ks, N, Hq):
    """Sharp, flat and far-scaled scores."""
    lengths = [300, 90]
    c, r, q, k, v, mask = attention_inputs(spec, 2, N, Hq, 2, 128, 16, lengths, 5, kscale=ks)
    q, k = (q.float() * qs).to(BF), (k.float() * ks).to(BF)
    out, lse = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda(), return_lse=True)
    check_attention(r, lengths, q, k, v, mask, out, lse, 1 / math.sqrt(128))


@pytest.mark.parametrize("vs", [2.0 ** -100, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("N,Hq", [(1, 4), (20, 8)])
def test_attention_value_magnitudes(spec, vs, N, Hq):
    """Values far from 1, and blocks whose scales differ by many powers of two."""
    lengths = [300]
    c, r, q, k, v, mask = attention_inputs(spec, 1, N, Hq, 2, 64, 16, lengths, 6)
    rows = r.rows[1][0].float() * vs
    rows[64:80] *= 2.0 ** -20
    r.rows[1][0] = rows.to(BF)
    d = spec.KvCache.allocate(c.k_pages.shape[0], 2, 16, 64, c.page_table, torch.zeros(1, dtype=torch.int32, device="cuda"))
    spec.spec_kv_append(r.rows[0][0][None].cuda(), r.rows[1][0][None].cuda(), None, d)
    v = (v.float() * vs).to(BF)
    out, lse = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), d, ref.pack(mask).cuda(), return_lse=True)
    check_attention(r, lengths, q, k, v, mask, out, lse, 1 / 8)


@pytest.mark.parametrize("N,Hq,Hkv,D", [(6, 4, 2, 128), (6, 4, 2, 64), (40, 8, 2, 128)])
def test_attention_non_finite_nodes_stay_masked(spec, N, Hq, Hkv, D):
    """A node with NaN or infinite keys or values reaches the rows whose mask holds it, and no other."""
    c, r, q, k, v, mask = attention_inputs(spec, 2, N, Hq, Hkv, D, 16, [100, 5], 3)
    clean = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda())
    k, v = k.clone(), v.clone()
    k[0, 2], v[1, 3] = float("nan"), float("inf")
    v[0, 4, 0, 7], k[1, 1, 0, 0], k[1, 5] = float("nan"), float("inf"), float("-inf")
    out = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda())
    hit = torch.stack([mask[0, :, 2] | mask[0, :, 4], mask[1, :, 3] | mask[1, :, 1] | mask[1, :, 5]])
    assert hit.any() and not hit.all()
    assert torch.equal(out[~hit.cuda()], clean[~hit.cuda()])
    assert torch.isnan(out[0][mask[0, :, 2].cuda()]).all()
    both = mask[0, :, 4] & ~mask[0, :, 2]
    G = Hq // Hkv
    assert torch.isnan(out[0][both.cuda()][:, :G, 7]).all()
    rest = out[0][both.cuda()].clone()
    rest[:, :G, 7] = 0
    assert torch.isfinite(rest).all()
    only = mask[1, :, 3] & ~mask[1, :, 1] & ~mask[1, :, 5]
    assert (out[1][only.cuda()] == math.inf).all()


@pytest.mark.parametrize("N,Hq", [(1, 8), (6, 8), (40, 8)])
def test_attention_flags_bad_pages(spec, N, Hq):
    """A page id, slot or length out of range: NaN for that sequence, the others as without it."""
    lengths = [40, 100, 64, 33, 20, 70]
    c, r, q, k, v, mask = attention_inputs(spec, 6, N, Hq, 2, 64, 16, lengths, 8, slots=[0, 1, 2, 3, 4, 5])
    args = (q.cuda(), k.cuda(), v.cuda())
    clean, clean_lse = spec.spec_tree_attention(*args, c, ref.pack(mask).cuda(), return_lse=True)
    ws = workspace(spec, 6, N, Hq, 64)
    c.page_table[1, 3], c.page_table[2, 0] = c.k_pages.shape[0], -3
    c.page_table[0, 2] = -9                                       # past the last full block: not read
    c.slots[3] = 99
    c.lengths[4] = 16 * c.page_table.shape[1] + 16
    out, lse = spec.spec_tree_attention(*args, c, ref.pack(mask).cuda(), return_lse=True, workspace=ws)
    assert flagged(spec, ws)
    for b in (1, 2, 3, 4):
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
    for b in (0, 5):
        assert torch.equal(out[b], clean[b]) and torch.equal(lse[b], clean_lse[b])


@pytest.mark.parametrize("N", [1, 40])
def test_attention_strides_and_shared_pages(spec, N):
    """Packed projections and transposed views give the contiguous result; two sequences share a prefix's pages."""
    B, Hq, Hkv, D, page = 3, 8, 2, 64, 16
    c, r, q, k, v, mask = attention_inputs(spec, B, N, Hq, Hkv, D, page, [70, 70, 33], 4)
    anc = ref.pack(mask).cuda()
    e = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, anc)
    qkv = torch.cat((q.flatten(2), k.flatten(2), v.flatten(2)), -1).cuda()
    pq, pk, pv = qkv.split((Hq * D, Hkv * D, Hkv * D), -1)
    assert torch.equal(spec.spec_tree_attention(pq.unflatten(-1, (Hq, D)), pk.unflatten(-1, (Hkv, D)),
                                                pv.unflatten(-1, (Hkv, D)), c, anc), e)
    t = [x.transpose(1, 2).contiguous().transpose(1, 2).cuda() for x in (q, k, v)]
    assert torch.equal(spec.spec_tree_attention(*t, c, anc), e)
    q2, k2, v2 = (x[:1].expand(B, -1, -1, -1).cuda() for x in (q, k, v))          # stride 0 over the batch
    c.page_table[1] = c.page_table[0]
    c.k_open[1], c.v_open[1] = c.k_open[0], c.v_open[0]
    out = spec.spec_tree_attention(q2, k2, v2, c, anc[:1].expand(B, -1, -1).contiguous())
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], e[0])
    # a page table that is a slice of a wider one
    wide = torch.full((B, c.page_table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.page_table.shape[1]] = c.page_table
    d = c.batch(wide[:, :c.page_table.shape[1]], c.lengths)
    assert torch.equal(spec.spec_tree_attention(q2, k2, v2, d, anc[:1].expand(B, -1, -1).contiguous()), out)


def test_empty_batch(spec):
    c = spec.KvCache.allocate(1, 2, 16, 64, torch.zeros((0, 1), dtype=torch.int32, device="cuda"),
                              torch.zeros(0, dtype=torch.int32, device="cuda"))
    z = lambda h: torch.zeros((0, 3, h, 64), dtype=BF, device="cuda")  # noqa: E731
    assert spec.spec_tree_attention(z(4), z(2), z(2), c).shape == (0, 3, 4, 64)
    assert spec.spec_kv_append(z(2), z(2), None, c).shape == (0,)
    pos, anc = spec.spec_tree_plan(torch.zeros((0, 3), dtype=torch.int32, device="cuda"), c.lengths)
    assert pos.shape == (0, 3)
    assert spec.spec_qk_norm_rope(z(4), z(2), pos, None)[0].shape == (0, 3, 4, 64)


# ----------------------------------------------------------------------------- rounds

def _round(spec, w, c, tokens, parents, emb, freq, depth, **kw):
    """One verify round of a one-layer model: returns the verify call's outputs."""
    B, N = tokens.shape
    x = emb[tokens.long().clamp(min=0)]
    q, k, v = (torch.matmul(x, m).unflatten(-1, (-1, c.head_dim)) for m in (w["q"], w["k"], w["v"]))
    pos, anc = spec.spec_tree_plan(parents, c.lengths, depth, **kw)
    q, k = spec.spec_qk_norm_rope(q, k, pos, freq, q_weight=w["qn"], k_weight=w["kn"])
    out = spec.spec_tree_attention(q, k, v, c, anc, **kw)
    logits = torch.matmul(out.flatten(2), w["o"])
    index, toks, num = spec.spec_verify_tree_greedy(logits, tokens, parents, depth)
    spec.spec_kv_append(k, v, num, c, accept_index=index, **kw)
    return index, toks, num


def _model(V=64, Hq=8, Hkv=2, D=64, dim=128, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda") / math.sqrt(s[0])  # noqa: E731
    w = dict(q=r(dim, Hq * D), k=r(dim, Hkv * D), v=r(dim, Hkv * D), o=r(Hq * D, V))
    w = {n: m.to(BF) for n, m in w.items()}
    w["qn"], w["kn"] = (torch.rand(D, generator=g, device="cuda") + 0.5).to(BF), (torch.rand(D, generator=g, device="cuda") + 0.5).to(BF)
    return w, (torch.randn((V, dim), generator=g, device="cuda")).to(BF), gpu(ref.inv_freq(D))


def test_rounds_decode_like_single_tokens(spec):
    """Tree rounds whose drafts are partly right emit the greedy tokens that one-token rounds emit, and
    leave the same cache."""
    B, Hkv, D, page, V = 3, 2, 64, 16, 64
    w, emb, freq = _model()
    one, tree = (make_cache(spec, B, Hkv, D, page, 8, np.random.RandomState(2)) for _ in range(2))
    prompt = torch.randint(0, V, (B, 21), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x = emb[prompt]
    k, v = (torch.matmul(x, w[n]).unflatten(-1, (-1, D)) for n in "kv")
    num = gpu(np.array([20, 15, 9], dtype=np.int32))
    for c in (one, tree):
        spec.spec_kv_append(k, v, num, c, inv_freq=freq, k_weight=w["kn"])
    start = c.lengths.clone()
    root = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    steps = 60
    cur, text = root[:, None], []
    single = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        _, toks, num1 = _round(spec, w, one, cur, single, emb, freq, 0)
        assert (num1 == 0).all()
        text.append(toks[:, :1])
        cur = toks[:, :1].contiguous()
    text = torch.cat(text, 1).cpu()
    rs = np.random.RandomState(3)
    done = [0] * B
    last = root.cpu().clone()
    longest = 0
    while min(done) < steps - 8:
        N = int(rs.randint(2, 20))
        parents = ref.random_parents(B, N, rs, 6, 5)
        tokens = rs.randint(0, V, (B, N)).astype(np.int32)
        depth = np.zeros((B, N), dtype=int)
        for b in range(B):
            tokens[b, 0] = last[b]
            for n in range(1, N):
                depth[b, n] = depth[b, parents[b, n]] + 1
                if rs.rand() < 0.7 and done[b] + depth[b, n] - 1 < steps:
                    tokens[b, n] = text[b, done[b] + depth[b, n] - 1]
        _, toks, num = _round(spec, w, tree, gpu(tokens), gpu(parents), emb, freq, 6)
        toks, num = toks.cpu(), num.cpu()
        for b in range(B):
            n = int(num[b]) + 1
            longest = max(longest, n)
            m = min(n, steps - done[b])
            assert torch.equal(toks[b, :m], text[b, done[b]:done[b] + m])
            done[b] += n
            last[b] = toks[b, n - 1]
        if max(done) > steps:
            break
    assert longest >= 3
    # both caches hold the same tokens' rows, up to the shorter one's full blocks and the bits of its open block
    for b in range(B):
        n = min(int(one.lengths[b]), int(tree.lengths[b]))
        assert n > int(start[b]) + 8
        full = n // page
        a, t = one.page_table[b, :full].long(), tree.page_table[b, :full].long()
        for x, y in ((one.k_pages, tree.k_pages), (one.v_pages, tree.v_pages)):
            d = (x.view(torch.uint8)[a] != y.view(torch.uint8)[t]).float().mean()
            assert d < 0.02            # the products before may round a key by their batch's shape


def test_round_in_a_graph(spec):
    """A captured round, replayed over changing drafts, leaves what eager rounds leave; the workspace is the graph's own."""
    B, N, D, page = 2, 8, 64, 16
    w, emb, freq = _model(seed=4)
    eager, graphed = (make_cache(spec, B, 2, D, page, 8, np.random.RandomState(2)) for _ in range(2))
    rs = np.random.RandomState(5)
    parents = gpu(ref.random_parents(B, N, rs, 6))
    tokens = gpu(rs.randint(0, 64, (B, N)).astype(np.int32))
    scratch = make_cache(spec, B, 2, D, page, 8, np.random.RandomState(2))
    _round(spec, w, scratch, tokens, parents, emb, freq, 6)                # libraries warm up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _round(spec, w, graphed, tokens, parents, emb, freq, 6)
    assert (graphed.lengths == 0).all()
    for _ in range(9):
        tokens.copy_(gpu(rs.randint(0, 64, (B, N)).astype(np.int32)))
        graph.replay()
        e = _round(spec, w, eager, tokens, parents, emb, freq, 6)
        assert all(torch.equal(a, b) for a, b in zip(outs, e))
    assert torch.equal(eager.lengths, graphed.lengths) and int(eager.lengths.min()) >= 9
    for name in ("k_pages", "v_pages", "k_scale", "v_scale", "k_open", "v_open"):
        a, b = getattr(eager, name), getattr(graphed, name)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("N,Hq,lengths", [(1, 8, [3000, 2900]), (16, 16, [3000, 100])])
def test_two_graphs_and_streams_at_once(spec, N, Hq, lengths):
    """Two captured calls replayed on two streams, and eager calls on two streams, do not disturb each other."""
    sides = [attention_inputs(spec, 2, N, Hq, 2, 128, 16, lengths, s) for s in (1, 2)]
    want, graphs, outs = [], [], []
    for c, r, q, k, v, mask in sides:
        args = (q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda())
        want.append(spec.spec_tree_attention(*args))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(spec.spec_tree_attention(*args))
        graphs.append((g, args))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, e) for o, e in zip(outs, want))
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(spec.spec_tree_attention(*graphs[i][1], stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


def test_one_workspace_serves_every_size(spec):
    """Calls of different sizes, in turn, on one workspace."""
    ws = workspace(spec, 16, 64, 32, 128)
    for i, (B, N, Hq, lengths) in enumerate([(2, 64, 16, [900, 30]), (1, 1, 4, [2000]), (9, 3, 8, [70] * 9),
                                             (1, 40, 32, [1500]), (2, 64, 16, [33, 1200])]):
        c, r, q, k, v, mask = attention_inputs(spec, B, N, Hq, 2, 128, 16, lengths, 20 + i)
        out, lse = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda(), return_lse=True,
                                            workspace=ws)
        spec.spec_tree_plan(None, c.lengths, 0, N=5, workspace=ws)
        check_attention(r, lengths, q, k, v, mask, out, lse, 1 / math.sqrt(128))
        room = gpu(np.zeros(B, dtype=np.int32))
        spec.spec_kv_append(k.cuda(), v.cuda(), room - 1, c, workspace=ws)
        assert c.lengths.tolist() == lengths
