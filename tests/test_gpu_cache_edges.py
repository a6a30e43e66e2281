"""The cache calls at the edges of what their documentation allows.  Tolerances as in test_gpu_cache.py, whose
inputs and checks are used."""
import math
import os
import re
import types

import numpy as np
import pytest
import torch

import cache_ref as ref
from test_gpu_cache import BF, attention_inputs, check_attention, flagged, gpu, make_cache, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spec(cuda_device):
    import speculative_decoding_verify_temperature_b200 as s
    return s


# ----------------------------------------------------------------------------- values of any magnitude

def far_values(spec, N, Hq, Hkv, D, page, length, blocks, tail, nodes, seed=0):
    """One sequence whose cached values are multiplied by powers of two: 2^blocks[i mod n] in block i, 2^tail in the open
    block, 2^nodes[i mod n] in node i."""
    g = torch.Generator().manual_seed(seed)
    c = make_cache(spec, 1, Hkv, D, page, max(length // page, 1), np.random.RandomState(seed))
    r = ref.Cache(1, Hkv, D, page)
    full = length // page * page
    e = [blocks[t // page % len(blocks)] if t < full else tail for t in range(length)]
    scale = torch.exp2(torch.tensor(e, dtype=torch.float64))[:, None, None]
    k = torch.randn((length, Hkv, D), generator=g).to(BF)
    v = (torch.randn((length, Hkv, D), generator=g).double() * scale).to(BF)
    if length:
        spec.spec_kv_append(k[None].cuda(), v[None].cuda(), None, c)
        r.append(0, k, v)
    q, nk = torch.randn((1, N, Hq, D), generator=g).to(BF), torch.randn((1, N, Hkv, D), generator=g).to(BF)
    ne = torch.exp2(torch.tensor([nodes[i % len(nodes)] for i in range(N)], dtype=torch.float64))
    nv = (torch.randn((1, N, Hkv, D), generator=g).double() * ne[None, :, None, None]).to(BF)
    return c, r, q, nk, nv


FAR = [  # cached, exponents of the full blocks, of the open block, of the nodes
    (0, [0], 0, [-117]), (0, [0], 0, [-126, -118]), (1, [0], -119, [-119]), (300, [-118], -118, [-118]),
    (300, [-126, -110], -100, [-122]), (300, [-125, 20], 10, [15, -120]), (300, [20, -125, -125, -125], -125, [-125]),
    (300, [110, -120], -126, [100, -118]), (300, [118], 118, [118]), (333, [0, -118], -118, [0]), (9000, [-118, 30], 0, [-117]),
    (9000, [-118], -118, [-118]), (20000, [-60, -120, 60], 3, [1, -1, 90])]


@pytest.mark.parametrize("N,Hq,Hkv,D,page", [(1, 8, 2, 128, 16), (3, 8, 2, 64, 32), (5, 6, 2, 128, 64), (20, 8, 2, 128, 128),
                                             (33, 8, 2, 64, 16), (70, 4, 1, 128, 32)])
@pytest.mark.parametrize("length,blocks,tail,nodes", FAR)
def test_attention_of_far_values(spec, N, Hq, Hkv, D, page, length, blocks, tail, nodes):
    """Values of any magnitude that bf16 and the pages' scales hold, in one row's reach: neither the log-sum-exp, which has
    nothing to do with the values, nor the outputs lose a key."""
    c, r, q, k, v = far_values(spec, N, Hq, Hkv, D, page, length, blocks, tail, nodes)
    mask = torch.tril(torch.ones(N, N, dtype=torch.bool))[None]
    ws = workspace(spec, 1, N, Hq, D)
    out, lse = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda(), return_lse=True, workspace=ws)
    check_attention(r, [length], q, k, v, mask, out, lse, 1 / math.sqrt(D))
    assert spec.spec_read_device_status(ws) == 0


@pytest.mark.parametrize("length", [0, 7, 40])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 4, 2, 128), (1, 16, 1, 64), (5, 8, 2, 128), (30, 8, 2, 128), (40, 8, 1, 64)])
def test_attention_of_small_elements_of_open_values(spec, N, Hq, Hkv, D, length):
    """A value row that is not in a page yet is rounded at 2^-25 of its largest element at worst (half of f16's smallest step,
    2^-24, of a row that was brought to [1, 2)); the probabilities' weights sum to 1, so the outputs are off by no more than
    that of the largest row, beside what the other tests allow."""
    g = torch.Generator().manual_seed(N + length)
    page, full = 32, length // 32 * 32
    c, r = make_cache(spec, 1, Hkv, D, page, 2, np.random.RandomState(0)), ref.Cache(1, Hkv, D, page)
    rows = lambda n, h: torch.randn((1, n, h, D), generator=g)  # noqa: E731

    def values(n):
        v = rows(n, Hkv) * torch.exp2(-29 * torch.rand((1, n, Hkv, D), generator=g))
        v[..., 0] = 1.5
        return v.to(BF)

    if length:
        k, v = rows(length, Hkv).to(BF), torch.cat((rows(full, Hkv).to(BF) * 0, values(length - full)), 1)
        spec.spec_kv_append(k.cuda(), v.cuda(), None, c)
        r.append(0, k[0], v[0])
    q, k, v = (rows(N, Hq) * 4).to(BF), rows(N, Hkv).to(BF), values(N)
    mask = torch.tril(torch.ones(N, N, dtype=torch.bool))[None]
    out = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda())[0].cpu().double()
    cached = [torch.cat(((b.view(torch.float8_e4m3fn).double() * s[..., None, None]).transpose(1, 2).reshape(-1, Hkv, D),
                         r.open_rows(0, i).double())) for i in range(2) for b, s in [r.blocks(0, i)]]
    scales = torch.cat((torch.ones(full, Hkv), ref.row_scale(r.open_rows(0, 1).double())))
    e, _, pv, mag, small, lost = ref.attention(q[0].double(), k[0].double(), v[0].double(), *cached, mask[0], 1 / math.sqrt(D), scales,
                                               full)
    ds = (D + 8) * 2.0 ** -23 * mag + lost
    tol = e.abs() * 2.0 ** -8 + pv * (2.0 ** -11 + 2 * ds + 2.0 ** -20)[..., None] + small * 2.0 ** -36
    largest = max(float(x.abs().max()) for x in (v, r.open_rows(0, 1)) if x.numel())
    assert ((out - e).abs() <= tol + largest * 2.0 ** -25).all()


# ----------------------------------------------------------------------------- append

@pytest.mark.parametrize("rot", range(0, 129, 16))
@pytest.mark.parametrize("dt", [torch.float32, BF])
def test_append_every_rotated_width(spec, rot, dt):
    """Every width of rotation at the largest page and head: what a call needs of shared memory it asks for itself."""
    D = page = 128
    k, v = torch.randn(1, page + 3, 1, D).to(dt), torch.randn(1, page + 3, 1, D).to(dt)
    c = make_cache(spec, 1, 1, D, page, 1, np.random.RandomState(rot))
    freq = ref.inv_freq(rot) if rot else None
    spec.spec_kv_append(k.cuda(), v.cuda(), None, c, inv_freq=None if freq is None else freq.cuda())
    assert c.lengths.tolist() == [page + 3]
    e, mag = ref.norm_rope(k[0], torch.arange(page + 3), freq, None, 1e-6, False)
    got = c.k_open[0][:, page:page + 3].transpose(0, 1).cpu().double()
    assert ((got - e[page:]).abs() <= e[page:].abs() * 2.0 ** -8 + mag[page:] * 2.0 ** -19).all()


@pytest.mark.parametrize("D,page,rot,inter,weights,dt", [(128, 64, 128, False, True, BF), (128, 128, 128, False, True, BF),
                                                         (64, 16, 32, False, True, torch.float32), (128, 32, 96, True, False, BF),
                                                         (64, 128, 64, True, True, torch.float32), (128, 16, 128, False, False, BF)])
def test_append_rotates_as_the_norm_and_rotation_call_does(spec, D, page, rot, inter, weights, dt):
    """Raw keys appended with a norm and a rotation leave what that call's output leaves, bit for bit: bf16 keys, which it rounds
    as the append does."""
    B, Hkv, first, T = 3, 4, 1000, 2 * page + 41
    g = torch.Generator("cuda").manual_seed(D + page)
    freq = gpu(ref.inv_freq(rot, 1e4))
    w = (torch.rand((D,), generator=g, device="cuda") + 0.5).to(dt) if weights else None
    raw, ready = (make_cache(spec, B, Hkv, D, page, (first + T) // page + 1, np.random.RandomState(5)) for _ in range(2))
    v0 = torch.randn((B, first, Hkv, D), generator=g, device="cuda").to(dt)
    k, v = ((torch.randn((B, T, Hkv, D), generator=g, device="cuda") * 3).to(dt) for _ in range(2))
    num = gpu(np.array([T, T - 5, T - 30], dtype=np.int32)) - 1
    for c in (raw, ready):
        spec.spec_kv_append(v0, v0, gpu(np.array([first - 1, first // 2, 6], dtype=np.int32)), c)
    pos = raw.lengths[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)
    turned = spec.spec_qk_norm_rope(k, k, pos, freq, q_weight=w, k_weight=w, eps=1e-6, interleaved=inter)[1]
    spec.spec_kv_append(k, v, num, raw, inv_freq=freq, k_weight=w, eps=1e-6, interleaved=inter)
    spec.spec_kv_append(turned, v, num, ready)
    assert torch.equal(raw.lengths, ready.lengths)
    for name in ("k_pages", "v_pages", "k_scale", "v_scale", "k_open", "v_open"):
        assert torch.equal(getattr(raw, name).view(torch.uint8), getattr(ready, name).view(torch.uint8)), name


# ----------------------------------------------------------------------------- plan

def test_plan_of_a_row_without_a_sequence(spec):
    """A padded row's parents are not looked at: it gets its -1 and zeros, and nothing is reported."""
    parents = np.tile(np.arange(-1, 7, dtype=np.int32), (3, 1))
    parents[1] = 1 << 20
    ws = workspace(spec)
    pos, anc = spec.spec_tree_plan(gpu(parents), gpu(np.array([4, -1, 9], dtype=np.int32)), 8, workspace=ws)
    assert (pos[1] == -1).all() and (anc[1] == 0).all() and not flagged(spec, ws)
    assert pos[0].tolist() == list(range(4, 12)) and pos[2].tolist() == list(range(9, 17))


# ----------------------------------------------------------------------------- waits that give up

TIMEOUT, IN_FLIGHT = 1 << 5, 1 << 7


@pytest.mark.parametrize("N,Hq,Hkv,D,page,lengths", [
    (1, 8, 2, 128, 16, [40, 100, 7, 900]), (3, 8, 2, 64, 32, [3000, 65]), (20, 8, 2, 128, 16, [40, 100, 7, 900]),
    (20, 8, 2, 64, 128, [500, 20000]), (70, 4, 1, 128, 64, [300, 2000]), (24, 8, 2, 128, 32, [(i * 97) % 700 for i in range(90)])])
def test_attention_says_when_a_wait_gave_up(spec, N, Hq, Hkv, D, page, lengths):
    """With no patience for a copy (the copies land as ever) the call ends, its rows are NaN, and the status word says so;
    no copy is left in flight, and the next call on the same workspace is clean."""
    c, r, q, k, v, mask = attention_inputs(spec, len(lengths), N, Hq, Hkv, D, page, lengths, 11 * N + D)
    ws = workspace(spec, len(lengths), N, Hq, D)
    args = (q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda())
    clean, clean_lse = spec.spec_tree_attention(*args, return_lse=True, workspace=ws)
    assert spec.spec_read_device_status(ws) == 0
    spec.spec_debug_wait_budget(0)
    try:
        out, lse = spec.spec_tree_attention(*args, return_lse=True, workspace=ws)
    finally:
        spec.spec_debug_wait_budget(-1)
    status = spec.spec_read_device_status(ws)
    assert status & TIMEOUT and not status & IN_FLIGHT, status
    for b, n in enumerate(lengths):
        if n >= page:                                     # the row needed a copy
            assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
        else:
            assert torch.isnan(out[b]).all() or torch.equal(out[b], clean[b])
    again, again_lse = spec.spec_tree_attention(*args, return_lse=True, workspace=ws)
    assert spec.spec_read_device_status(ws) == 0
    assert torch.equal(again, clean) and torch.equal(again_lse, clean_lse)


# ----------------------------------------------------------------------------- workspaces and streams

def test_status_of_calls_without_a_workspace(spec):
    """What a call without a workspace reports can be read, per stream, also after that workspace has grown."""
    side = torch.cuda.Stream()
    parents = gpu(np.array([[-1, 5]], dtype=np.int32))
    lengths = gpu(np.array([3], dtype=np.int32))
    spec.spec_cache_status(), spec.spec_cache_status(stream=side)        # what other tests left
    spec.spec_tree_plan(parents, lengths, 4)
    assert spec.spec_cache_status() == 1 << 4 and spec.spec_cache_status() == 0
    spec.spec_tree_plan(parents, lengths, 4, stream=side)
    assert spec.spec_cache_status() == 0
    c, r, q, k, v, mask = attention_inputs(spec, 1, 200, 8, 1, 128, 16, [40], 1)
    torch.cuda.synchronize()
    spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda(), stream=side)     # needs a larger one
    assert spec.spec_cache_status("cuda", side) == 1 << 4 and spec.spec_cache_status("cuda", side) == 0
    with torch.cuda.stream(side):
        spec.spec_tree_plan(parents, lengths, 4)
        assert spec.spec_cache_status() == 1 << 4


def test_only_a_workspaces_state_has_to_be_zero(spec):
    """Behind the status word and the counters a workspace may hold anything."""
    B, N, Hq, lengths = 3, 40, 8, [3000, 30, 700]
    c, r, q, k, v, mask = attention_inputs(spec, B, N, Hq, 2, 128, 16, lengths, 3)
    args = (q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda())
    for n in (N, 1):
        args = tuple(x[:, :n] if i < 3 else x for i, x in enumerate(args[:4])) + (None,)
        want = spec.spec_tree_attention(*args, return_lse=True)
        ws = torch.full((spec.spec_cache_workspace_bytes(B, n, Hq, 128),), 255, dtype=torch.uint8, device="cuda")
        spec.spec_workspace_init(ws[:65792])
        got = spec.spec_tree_attention(*args, return_lse=True, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert spec.spec_read_device_status(ws) == 0


@pytest.mark.parametrize("N", [1, 40])
def test_tensors_may_be_dropped_after_a_call_on_another_stream(spec, N):
    """The memory of the inputs is not used again before the other stream has read it, nor that of the outputs before the
    current one has."""
    c, r, q, k, v, mask = attention_inputs(spec, 2, N, 8, 2, 128, 16, [100, 300], 2)
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    anc = ref.pack(mask).cuda()
    want = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, anc)
    others = (-q).cuda(), k.cuda(), v.cuda()
    assert not torch.equal(want, spec.spec_tree_attention(*others, c, anc))
    for _ in range(2):
        args = [x.cuda() for x in (q, k, v)] + [anc.clone()]
        shapes = [(x.shape, x.dtype) for x in args]
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                     # some 10 ms
        out = spec.spec_tree_attention(*args[:3], c.batch(c.page_table.clone(), c.lengths.clone()), args[3], stream=side)
        del args
        junk = [torch.full(s, -1, dtype=d, device="cuda") for s, d in shapes for _ in range(4)]
        junk += [torch.full_like(c.page_table, -1) for _ in range(4)] + [torch.full_like(c.lengths, -1) for _ in range(4)]
        main.wait_stream(side)
        torch.cuda._sleep(20_000_000)
        got = out.clone()
        del out
        keep = [spec.spec_tree_attention(*others, c, anc, stream=side) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and len(junk) + len(keep) > 0


def test_a_captured_branch_on_another_stream(spec):
    """Two branches of one graph, each with calls on a stream of its own and temporaries that are dropped at once."""
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    inputs = [attention_inputs(spec, 2, N, 8, 2, 128, 16, [900, 40], N) for N in (3, 40)]
    args = [(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda()) for c, r, q, k, v, mask in inputs]
    want = [spec.spec_tree_attention(*a) for a in args]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main, outs = torch.cuda.current_stream(), []
        for side, a in zip(sides, args):
            outs.append([])
            for _ in range(3):
                temps = [x * 1 for x in a[:3]]
                side.wait_stream(main)
                outs[-1].append(spec.spec_tree_attention(*temps, *a[3:], stream=side))
        for side in sides:
            main.wait_stream(side)
        got = [[o * 1 for o in branch] for branch in outs]
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, e) for branch, e in zip(got, want) for o in branch)


# ----------------------------------------------------------------------------- several layers

def test_rounds_of_several_layers_as_documented(spec):
    """The README's program on a model of three layers that share page table and lengths: after a prompt and a round every layer
    holds its own rows of the same tokens, as caches with lengths of their own do."""
    B, Hq, Hkv, D, page, dim, V = 3, 4, 2, 64, 16, 96, 64
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    program = re.search(r"### A round over the cache.*?```python\n(.*?)```", text, re.S).group(1)
    g = torch.Generator("cuda").manual_seed(0)
    r = lambda *s: (torch.randn(s, generator=g, device="cuda") / math.sqrt(s[0])).to(BF)  # noqa: E731

    class Layer:
        def __init__(self):
            self.w, self.o = r(dim, (Hq + 2 * Hkv) * D), r(Hq * D, dim)
            self.q_weight, self.k_weight = r(1, D)[0].abs() + 0.5, r(1, D)[0].abs() + 0.5
            self.seen = []

        def project(self, x):
            q, k, v = (x @ self.w).split((Hq * D, Hkv * D, Hkv * D), -1)
            self.seen.append((k.unflatten(-1, (Hkv, D)), v.unflatten(-1, (Hkv, D))))
            return q.unflatten(-1, (Hq, D)), *self.seen[-1]

        def finish(self, x, attn):
            return x + attn.flatten(2) @ self.o

    rs = np.random.RandomState(1)
    table, emb, unembed = gpu(rs.permutation(B * 4).astype(np.int32).reshape(B, 4)), r(V, dim), r(dim, V)
    parents = ref.random_parents(B, 6, rs)
    given = dict(layers=[Layer() for _ in range(3)], num_pages=B * 4, kv_heads=Hkv, page_size=page, head_dim=D, page_table=table,
                 lengths=torch.zeros(B, dtype=torch.int32, device="cuda"), inv_freq=gpu(ref.inv_freq(D)), max_depth=6,
                 embed=lambda t: emb[t.long()], head=lambda x: x @ unembed, parents=gpu(parents),
                 prompt=torch.randint(0, V, (B, 37), generator=g, device="cuda"), count=gpu(np.array([37, 15, 31], dtype=np.int32)),
                 draft_tokens=torch.randint(0, V, (B, 6), generator=g, device="cuda", dtype=torch.int32))
    exec(compile(program, "README.md", "exec"), given)
    space = types.SimpleNamespace(**{n: x for n, x in given.items() if n.isidentifier()})
    taken = (space.num + 1).clamp(min=0)
    assert torch.equal(space.lengths, space.count + taken)
    for layer, cache in zip(space.layers, space.caches):
        own = spec.KvCache.allocate(B * 4, Hkv, page, D, table, torch.zeros(B, dtype=torch.int32, device="cuda"))
        for (k, v), num, index in zip(layer.seen, (space.count - 1, space.num), (None, space.index)):
            if index is None:
                pos, _ = spec.spec_tree_plan(None, own.lengths, N=k.shape[1])
            else:
                pos, _ = spec.spec_tree_plan(space.parents, own.lengths, 6)
            k = spec.spec_qk_norm_rope(k, k, pos, space.inv_freq, q_weight=layer.q_weight, k_weight=layer.k_weight)[1]
            spec.spec_kv_append(k, v, num, own, accept_index=index)
        assert torch.equal(own.lengths, space.lengths)
        for name in ("k_pages", "v_pages", "k_scale", "v_scale", "k_open", "v_open"):
            assert torch.equal(getattr(own, name).view(torch.uint8), getattr(cache, name).view(torch.uint8)), name


# ----------------------------------------------------------------------------- large pools, items in many parts

@pytest.mark.parametrize("N,Hq,Hkv,D,length", [(1, 4, 1, 128, 40000), (2, 8, 1, 64, 30000), (24, 4, 1, 128, 25000),
                                               (80, 4, 1, 64, 25000)])
def test_attention_of_items_in_many_parts(spec, N, Hq, Hkv, D, length):
    """One kv head over a long cache: every CTA holds a part of the same item, and the join goes over more than 32 of them."""
    c, r, q, k, v, mask = attention_inputs(spec, 1, N, Hq, Hkv, D, 32, [length], N)
    out, lse = spec.spec_tree_attention(q.cuda(), k.cuda(), v.cuda(), c, ref.pack(mask).cuda(), return_lse=True)
    check_attention(r, [length], q, k, v, mask, out, lse, 1 / math.sqrt(D))


def test_a_pool_of_more_than_4_gb(spec):
    """Page ids whose bytes lie behind 2^32 give what low ones give, in the append and in both attention kernels."""
    Hkv, D, page, P, L = 8, 128, 128, 33000, 600
    g = torch.Generator("cuda").manual_seed(0)
    assert P * Hkv * page * D > 1 << 32
    lengths = torch.zeros(2, dtype=torch.int32, device="cuda")
    big = spec.KvCache.allocate(P, Hkv, page, D, gpu(np.array([[P - 1, 5, P - 7, 20000, P - 2]] * 2, dtype=np.int32)), lengths)
    big.page_table[1] = gpu(np.array([P - 11, 17000, 3, P - 4, 16999], dtype=np.int32))
    low = spec.KvCache.allocate(10, Hkv, page, D, gpu(np.arange(10, dtype=np.int32).reshape(2, 5)), lengths.clone())
    k, v = (torch.randn((2, L, Hkv, D), generator=g, device="cuda").to(BF) for _ in range(2))
    for c in (big, low):
        spec.spec_kv_append(k, v, None, c)
    assert big.lengths.tolist() == low.lengths.tolist() == [L, L]
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        x, y = (getattr(c, name).view(torch.uint8)[c.page_table[:, :L // page].long()] for c in (big, low))
        assert torch.equal(x, y), name
    for N in (1, 12):
        q = torch.randn((2, N, 2 * Hkv, D), generator=g, device="cuda").to(BF)
        outs = [spec.spec_tree_attention(q, k[:, :N], v[:, :N], c, return_lse=True) for c in (big, low)]
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
