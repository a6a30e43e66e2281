"""Measured cases of the cache operators around a verify round.

One case is one pass through one operator: the plan of a draft tree
(positions and ancestor masks), the norm and rotation of queries and keys, the
attention of the draft nodes over a paged 8-bit cache, and the append of the
accepted rows to that cache.  ``own`` selects the library's calls; otherwise
``run`` computes the same in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")
E4M3_MAX = 448.0


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # the plan of a round's trees, once per round: 64-node trees, and the widest trees over a large batch
        {"name": "plan_b32_n64", "op": "plan", "B": 32, "N": 64, "max_depth": 16},
        {"name": "plan_b256_n256", "op": "plan", "B": 256, "N": 256, "max_depth": 64},
        # norm + rotation: one decoded token (latency), a round of 64-node trees read out of a packed projection,
        # and an f32 model with interleaved pairs, a partial rotation and an odd node count
        {"name": "norm_rope_b1_n1", "op": "norm_rope", "B": 1, "N": 1, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "weights": True, "far": 4096},
        {"name": "norm_rope_b32_n64", "op": "norm_rope", "B": 32, "N": 64, "Hq": 64, "Hkv": 8, "D": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "weights": True, "far": 131072},
        {"name": "norm_rope_f32_b7_n33", "op": "norm_rope", "B": 7, "N": 33, "Hq": 24, "Hkv": 6, "D": 96, "rot": 48,
         "dtype": "f32", "interleaved": True, "weights": False, "far": 1000000},
        # append: the accepted path of a round of 64-node trees (already rotated rows, picked by index), and a
        # ragged prompt chunk whose raw keys are normed and rotated on the way
        {"name": "append_accepted_b32_n64", "op": "append", "B": 32, "T": 64, "W": 17, "Hkv": 8, "D": 128, "page": 16,
         "dtype": "bf16", "rot": 0, "weights": False, "index": True, "L": 4096},
        {"name": "append_prompt_b8_t2048", "op": "append", "B": 8, "T": 2048, "W": 2048, "Hkv": 8, "D": 128,
         "page": 64, "dtype": "bf16", "rot": 128, "weights": True, "index": False, "L": 0},
        # attention: one token of one sequence (latency); one token of a ragged batch (plain decode); a chain round
        # of gamma = 5; a round of 64-node trees (compute-bound); a 32-node tree on one very long context
        {"name": "attn_b1_n1_l1000", "op": "attention", "B": 1, "N": 1, "Hq": 32, "Hkv": 8, "D": 128, "page": 16,
         "L": 1000, "ragged": False, "tree": False},
        {"name": "attn_b64_n1_l8192", "op": "attention", "B": 64, "N": 1, "Hq": 32, "Hkv": 8, "D": 128, "page": 16,
         "L": 8192, "ragged": True, "tree": False},
        {"name": "attn_b64_n6_l4096", "op": "attention", "B": 64, "N": 6, "Hq": 64, "Hkv": 8, "D": 128, "page": 64,
         "L": 4096, "ragged": True, "tree": False},
        {"name": "attn_b32_n64_l8192", "op": "attention", "B": 32, "N": 64, "Hq": 64, "Hkv": 8, "D": 128, "page": 32,
         "L": 8192, "ragged": True, "tree": True},
        {"name": "attn_b1_n32_l131072", "op": "attention", "B": 1, "N": 32, "Hq": 32, "Hkv": 8, "D": 64, "page": 128,
         "L": 131072, "ragged": False, "tree": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    """One more case of the listed ranges.  Costs are bounded by the largest listed case of the operator."""
    op = rng.choice(["plan", "norm_rope", "norm_rope", "append", "append", "attention", "attention", "attention",
                     "attention"])
    if op == "plan":
        return {"op": op, "B": _log(rng, 1, 256), "N": _log(rng, 1, 256), "max_depth": rng.randint(8, 64)}
    if op == "norm_rope":
        while True:
            D = rng.choice([64, 96, 128])
            Hkv = rng.randint(1, 8)
            c = {"op": op, "B": _log(rng, 1, 64), "N": _log(rng, 1, 256), "Hq": Hkv * rng.randint(1, 8), "Hkv": Hkv,
                 "D": D, "rot": rng.choice([D, D, D // 2]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
                 "interleaved": rng.random() < 0.3, "weights": rng.random() < 0.7, "far": _log(rng, 1, 1000000)}
            if c["B"] * c["N"] * (c["Hq"] + Hkv) * D * (2 if c["dtype"] == "f32" else 1) <= 32 * 64 * 72 * 128:
                return c
    if op == "append":
        D, Hkv = rng.choice([64, 128]), rng.randint(1, 8)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if rng.random() < 0.5:
            page = rng.choice([16, 32, 64, 128])
            T = _log(rng, 1, 256)
            return {"op": op, "B": _log(rng, 1, 128), "T": T, "W": min(T, rng.randint(1, 17)), "Hkv": Hkv, "D": D,
                    "page": page, "dtype": dtype, "rot": 0, "weights": False, "index": True, "L": _log(rng, 1, 8192)}
        while True:
            T = _log(rng, 1, 4096)
            B = _log(rng, 1, 32)
            if B * T * (2 if dtype == "f32" else 1) * Hkv * D <= 8 * 2048 * 8 * 128:
                return {"op": op, "B": B, "T": T, "W": T, "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64, 128]),
                        "dtype": dtype, "rot": rng.choice([D, D // 2]), "weights": rng.random() < 0.5, "index": False,
                        "L": 0}
    while True:
        D, Hkv, G = rng.choice([64, 128, 128]), rng.randint(1, 8), rng.randint(1, 8)
        N = rng.choice([1, rng.randint(2, 17), _log(rng, 2, 256)])
        c = {"op": op, "B": _log(rng, 1, 128), "N": N, "Hq": Hkv * G, "Hkv": Hkv, "D": D,
             "page": rng.choice([16, 32, 64, 128]), "L": _log(rng, 1, 131072), "ragged": rng.random() < 0.6,
             "tree": N > 2 and rng.random() < 0.6}
        keys = c["B"] * (c["L"] + N)
        if keys * Hkv * D <= 32 * 8192 * 8 * 128 and keys * N * c["Hq"] <= 32 * 8192 * 64 * 64:
            return c


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * int(seed) + 17)


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _trees(B, N, max_depth, seed, tree=True):
    """Parent arrays [B, N]: chains, or random trees whose depth stays within max_depth."""
    if not tree:
        return np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1))
    rs = np.random.RandomState((int(seed) * 7919 + 11) % (1 << 31))
    parents = np.full((B, N), -1, dtype=np.int32)
    depth = np.zeros((B, N), dtype=np.int32)
    rows = np.arange(B)
    for n in range(1, N):
        lo = max(0, n - 8)                     # a drafted level's nodes hang off the few before them
        p = rs.randint(lo, n, size=B).astype(np.int32)
        p = np.where(depth[rows, p] < max_depth, p, 0)
        parents[:, n] = p
        depth[:, n] = depth[rows, p] + 1
    return parents


def _inv_freq(rot):
    """Frequencies of the rotation, base 1e6."""
    return torch.exp(torch.arange(0, rot, 2, dtype=torch.float64) * (-math.log(1e6) / rot)).to(torch.float32).cuda()


def _ancestors(parents):
    """[B, N, N] bool on the host: m is n or an ancestor of n."""
    B, N = parents.shape
    a = np.zeros((B, N, N), dtype=bool)
    rows = np.arange(B)
    for n in range(N):
        if n:
            a[:, n] = a[rows, parents[:, n]]
        a[:, n, n] = True
    return a


def _pack(a):
    """Bit words [B, N, ceil(N/32)] int32 of a host bool mask [B, N, N]."""
    B, N, _ = a.shape
    W = (N + 31) // 32
    p = np.zeros((B, N, W * 32), dtype=bool)
    p[:, :, :N] = a
    return np.packbits(p.reshape(B, N, W, 32), axis=-1, bitorder="little").view(np.int32).reshape(B, N, W)


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _kv_pool(pages, Hkv, page, D, g):
    """An 8-bit pool as a server holds it: channels of unequal size, each block scaled to its largest value."""
    channel = torch.exp(0.5 * torch.randn((1, Hkv, 1, D), generator=g, device="cuda"))
    data = torch.empty((pages, Hkv, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((pages, Hkv), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * D))
    for i in range(0, pages, step):
        x = torch.randn((min(step, pages - i), Hkv, page, D), generator=g, device="cuda") * channel
        s = x.abs().amax(dim=(2, 3)) / E4M3_MAX
        scale[i:i + step] = s
        data[i:i + step] = (x / s[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return data, scale


def prepare(case, seed):
    s = dict(case)
    s.pop("name", None)
    g = _gen(seed)
    rs = np.random.RandomState((int(seed) * 104729 + 7) % (1 << 31))
    op, B = case["op"], case["B"]
    if op == "plan":
        s["parents"] = _cuda(_trees(B, case["N"], case["max_depth"], seed))
        s["lengths"] = _cuda(rs.randint(0, 8192, size=B).astype(np.int32))
        return s
    D, Hkv = case["D"], case["Hkv"]
    dtype = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    if op == "norm_rope":
        N, Hq = case["N"], case["Hq"]
        qkv = _randn((B, N, (Hq + 2 * Hkv) * D), g, dtype)              # the packed projection of a layer
        s["q"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = qkv[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        s["positions"] = _cuda(rs.randint(0, case["far"], size=(B, N)).astype(np.int32))
        s["inv_freq"] = _inv_freq(case["rot"])
        s["q_weight"] = _randn((D,), g, dtype).abs() + 0.5 if case["weights"] else None
        s["k_weight"] = _randn((D,), g, dtype).abs() + 0.5 if case["weights"] else None
        return s
    page = case["page"]
    if op == "append":
        T, W = case["T"], case["W"]
        channel = torch.exp(0.5 * torch.randn((Hkv, D), generator=g, device="cuda"))
        s["k"] = (_randn((B, T, Hkv, D), g) * channel).to(dtype)
        s["v"] = (_randn((B, T, Hkv, D), g) * channel).to(dtype)
        if case["index"]:                      # the accepted path: the root, then increasing nodes, then -1
            count = rs.randint(1, W + 1, size=B)
            index = np.full((B, W), -1, dtype=np.int32)
            for b in range(B):
                index[b, 1:count[b]] = np.sort(rs.choice(np.arange(1, T), size=count[b] - 1, replace=False))
            index[:, 0] = 0
            s["index"] = _cuda(index)
            lengths = rs.randint(0, case["L"] + 1, size=B)
        else:                                  # a ragged prompt
            count = rs.randint(max(1, T // 2), T + 1, size=B)
            s["index"] = None
            lengths = np.zeros(B, dtype=np.int64)
        s["num_accepted"] = _cuda((count - 1).astype(np.int32))
        first = lengths // page
        fresh = -(-(W + page) // page)          # blocks of a sequence that this call may fill
        pages = B * fresh
        table = np.zeros((B, int(first.max()) + fresh), dtype=np.int32)
        ids = rs.permutation(pages).reshape(B, fresh).astype(np.int32)
        for b in range(B):
            table[b, first[b]:first[b] + fresh] = ids[b]
        # one page more than the pool has is where the plain form puts what it must not keep
        s["k_store"], s["k_scales"] = _kv_pool(pages + 1, Hkv, page, D, g)
        s["v_store"], s["v_scales"] = _kv_pool(pages + 1, Hkv, page, D, g)
        s["k_pages"], s["v_pages"] = s["k_store"][:pages], s["v_store"][:pages]
        s["k_scale"], s["v_scale"] = s["k_scales"][:pages], s["v_scales"][:pages]
        s["k_open"] = _randn((B, Hkv, 2 * page, D), g, torch.bfloat16)
        s["v_open"] = _randn((B, Hkv, 2 * page, D), g, torch.bfloat16)
        s["page_table"], s["lengths"] = _cuda(table), _cuda(lengths.astype(np.int32))
        s["inv_freq"] = _inv_freq(case["rot"]) if case["rot"] else None
        s["k_weight"] = _randn((D,), g, dtype).abs() + 0.5 if case["weights"] else None
        s["new_lengths"] = torch.empty_like(s["lengths"])
    else:
        N, Hq, L = case["N"], case["Hq"], case["L"]
        lengths = rs.randint(L // 4, L + 1, size=B) if case["ragged"] else np.full(B, L)
        lengths[0] = L
        blocks = L // page
        pages = max(1, B * blocks)
        table = rs.permutation(pages).astype(np.int32)[:B * blocks].reshape(B, blocks)
        s["k_pages"], s["k_scale"] = _kv_pool(pages, Hkv, page, D, g)
        s["v_pages"], s["v_scale"] = _kv_pool(pages, Hkv, page, D, g)
        s["k_open"] = _randn((B, Hkv, 2 * page, D), g, torch.bfloat16)
        s["v_open"] = _randn((B, Hkv, 2 * page, D), g, torch.bfloat16)
        s["page_table"], s["lengths"] = _cuda(table.reshape(B, blocks)), _cuda(lengths.astype(np.int32))
        s["q"] = _randn((B, N, Hq, D), g, torch.bfloat16)
        s["k"] = _randn((B, N, Hkv, D), g, torch.bfloat16)
        s["v"] = _randn((B, N, Hkv, D), g, torch.bfloat16)
        s["ancestors"] = _cuda(_pack(_ancestors(_trees(B, N, 16, seed, case["tree"]))))
    if own:
        import speculative_decoding_verify_temperature_b200 as spec
        s["cache"] = spec.KvCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["k_open"], s["v_open"],
                                  s["page_table"], s["lengths"])
    return s


# ----------------------------------------------------------------------------- the library's calls

def _run_own(s):
    import speculative_decoding_verify_temperature_b200 as spec
    op = s["op"]
    if op == "plan":
        return spec.spec_tree_plan(s["parents"], s["lengths"], s["max_depth"])
    if op == "norm_rope":
        return spec.spec_qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"],
                                      k_weight=s["k_weight"], eps=1e-6, interleaved=s["interleaved"])
    if op == "append":
        lengths = spec.spec_kv_append(s["k"], s["v"], s["num_accepted"], s["cache"], accept_index=s["index"],
                                      inv_freq=s["inv_freq"], k_weight=s["k_weight"], eps=1e-6,
                                      out_lengths=s["new_lengths"])
        return lengths, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["k_open"], s["v_open"]
    return spec.spec_tree_attention(s["q"], s["k"], s["v"], s["cache"], s["ancestors"], return_lse=True)


# ----------------------------------------------------------------------------- plain forms

def _plain_plan(s):
    parents, lengths = s["parents"].long(), s["lengths"]
    B, N = parents.shape
    # reach[n, m]: m is n or an ancestor of n; squaring doubles the steps that are covered
    reach = torch.eye(N, device="cuda").expand(B, N, N) + torch.nn.functional.one_hot(parents.clamp(min=0), N) * (
        parents >= 0)[..., None]
    for _ in range(7):                                                       # 2^7 steps cover every depth up to 64
        reach = (torch.bmm(reach, reach) > 0).float()
    positions = (lengths[:, None] + reach.sum(-1).to(torch.int32) - 1).to(torch.int32)
    W = (N + 31) // 32
    bits = torch.nn.functional.pad(reach.long(), (0, W * 32 - N)).view(B, N, W, 32)
    words = (bits << torch.arange(32, device="cuda")).sum(-1)
    return positions, torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def _norm_rotate(x, weight, positions, inv_freq, interleaved):
    """x [B, N, H, D] f32; the norm where there is a weight, then the rotation at positions [B, N]."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    if inv_freq is None:
        return x
    angle = positions.double()[..., None] * inv_freq.double()               # far positions need the 64 bits
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    r = 2 * inv_freq.numel()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _plain_norm_rope(s):
    return tuple(_norm_rotate(s[x].float(), s[x + "_weight"], s["positions"], s["inv_freq"], s["interleaved"]).to(
        s[x].dtype) for x in ("q", "k"))


def _block_scale(amax):
    """The least power of two that brings amax within 448; 1 for an empty block."""
    m, e = torch.frexp(amax)                                                 # amax = m * 2^e, 0.5 <= m < 1
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).int()),
                       torch.ones_like(amax))


def _plain_append(s):
    page, B, W = s["page"], s["B"], s["W"]
    lengths, count = s["lengths"].long(), s["num_accepted"].long() + 1
    i = torch.arange(W, device="cuda")
    rows = (s["index"].long() if s["index"] is not None else i.expand(B, W)).clamp(min=0)
    batch = torch.arange(B, device="cuda")[:, None]
    positions = lengths[:, None] + i
    new = lengths + count
    k = _norm_rotate(s["k"][batch, rows].float(), s["k_weight"], positions, s["inv_freq"], False).to(torch.bfloat16)
    v = s["v"][batch, rows].to(torch.bfloat16)
    # every block from the open one on, put together from the ring and the new rows
    first = lengths // page
    blocks = (page - 1 + W) // page
    at = first[:, None] * page + torch.arange(blocks * page, device="cuda")
    from_new = at >= lengths[:, None]
    full = (first[:, None] + torch.arange(blocks, device="cuda") + 1) * page <= new[:, None]
    spare = s["k_store"].shape[0] - 1
    entry = (first[:, None] + torch.arange(blocks, device="cuda")).clamp(max=s["page_table"].shape[1] - 1)
    target = torch.where(full, s["page_table"].long().gather(1, entry), spare)
    # the ring keeps what is left of the new rows: slot r holds position `turn` of the block that stays open
    last = (new // page * page)[:, None]
    turn = last + (torch.arange(2 * page, device="cuda") - last) % (2 * page)
    stay = ((turn >= lengths[:, None]) & (turn < new[:, None]))[:, None, :, None]
    turn = (turn - lengths[:, None]).clamp(0, W - 1)
    for x, store, scales, ring in ((k, s["k_store"], s["k_scales"], s["k_open"]),
                                   (v, s["v_store"], s["v_scales"], s["v_open"])):
        old = ring.transpose(1, 2)[batch, at % (2 * page)]
        fresh = x[batch, (at - lengths[:, None]).clamp(0, W - 1)]
        block = torch.where(from_new[..., None, None], fresh, old).float().unflatten(1, (blocks, page))
        block = block.transpose(2, 3)                                        # [B, blocks, Hkv, page, D]
        scale = _block_scale(block.abs().amax(dim=(3, 4)))
        store.view(torch.uint8)[target] = (block / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[target] = scale
        ring.copy_(torch.where(stay, x[batch, turn].transpose(1, 2), ring))
    s["new_lengths"].copy_(new)
    return (s["new_lengths"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["k_open"], s["v_open"])


def _plain_attention(s):
    q, page, D, Hkv = s["q"], s["page"], s["D"], s["Hkv"]
    B, N, Hq, _ = q.shape
    G = Hq // Hkv
    lengths, table = s["lengths"].long(), s["page_table"].long()
    full = lengths // page
    blocks = table.shape[1]

    def keys(pages, scale, ring, nodes):
        """[B, Hkv, blocks * page + page + N, D]: the full blocks, the open block, the nodes."""
        cached = pages.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        cached = (cached * scale[table][..., None, None]).transpose(1, 2).reshape(B, Hkv, -1, D)
        place = (full[:, None] * page + torch.arange(page, device="cuda")) % (2 * page)
        opened = ring.gather(2, place[:, None, :, None].expand(B, Hkv, page, D)).float()
        return torch.cat((cached, opened, nodes.float().transpose(1, 2)), 2)

    seen = torch.cat((torch.arange(blocks * page, device="cuda") < (full * page)[:, None],
                      torch.arange(page, device="cuda") < (lengths - full * page)[:, None]), 1)
    bits = s["ancestors"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32) & 1
    mask = torch.cat((seen[:, None].expand(B, N, -1), bits.flatten(2)[..., :N].bool()), 2)   # [B, N, keys]
    rows = q.float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    score = torch.matmul(rows, keys(s["k_pages"], s["k_scale"], s["k_open"], s["k"]).transpose(2, 3))
    score = score.mul_(1 / math.sqrt(D)).view(B, Hkv, N, G, -1)
    score.masked_fill_(~mask[:, None, :, None], NEG)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == NEG, torch.zeros_like(top), top)
    p = torch.exp_(score.sub_(top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hkv, N * G, -1), keys(s["v_pages"], s["v_scale"], s["v_open"], s["v"]))
    out = out.view(B, Hkv, N, G, D) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top).squeeze(-1)
    return out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(q.dtype), lse.permute(0, 2, 1, 3).reshape(B, N, Hq)


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plain_plan, "norm_rope": _plain_norm_rope, "append": _plain_append,
            "attention": _plain_attention}[state["op"]](state)


# ----------------------------------------------------------------------------- work

def work(case):
    op, B = case["op"], case["B"]
    if op == "plan":
        N = case["N"]
        return {"bytes": B * N * 4 + B * 4 + B * N * 4 + B * N * ((N + 31) // 32) * 4, "flops": 0}
    D, Hkv = case["D"], case["Hkv"]
    size = 4 if case.get("dtype") == "f32" else 2
    if op == "norm_rope":
        rows = B * case["N"] * (case["Hq"] + Hkv)
        return {"bytes": 2 * rows * D * size + B * case["N"] * 4, "flops": rows * D * (7 if case["weights"] else 3)}
    if op == "append":
        T, page = case["T"], case["page"]
        rows = B * ((case["W"] + 1) / 2 if case["index"] else 3 * T / 4)     # the mean count
        tail = min(page / 2, rows / B)                                       # what stays open, as bf16
        return {"bytes": rows * 2 * Hkv * D * (size + 1) + B * tail * 2 * Hkv * D, "flops": rows * 2 * Hkv * D * 4}
    N, Hq = case["N"], case["Hq"]
    keys = B * (case["L"] * (0.625 if case["ragged"] else 1.0))              # the mean length
    return {"bytes": keys * 2 * Hkv * D + B * N * (2 * Hq + 2 * Hkv) * D * 2 + B * N * Hq * 4,
            "flops": 4 * D * N * Hq * (keys + B * N / 2)}


# ----------------------------------------------------------------------------- 64 bits

def _exact_rotate(x, weight, positions, inv_freq, interleaved):
    """x [rows, H, D] f64, positions [rows]."""
    if weight is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * weight.double()
    if inv_freq is None:
        return x
    y = x.clone()
    half = inv_freq.numel()
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        angle = positions.double() * inv_freq[j].double()
        c, d = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * d
        y[..., b] = x[..., b] * c + x[..., a] * d
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "norm_rope":
        pos = s["positions"].flatten()
        return tuple(_exact_rotate(s[x].double().flatten(0, 1), s[x + "_weight"], pos, s["inv_freq"],
                                   s["interleaved"]).view(s[x].shape) for x in ("q", "k"))
    D, Hkv, page, B = case["D"], case["Hkv"], case["page"], case["B"]
    length = s["lengths"].tolist()
    if op == "append":
        count = (s["num_accepted"] + 1).tolist()
        table = s["page_table"].tolist()
        out = [None]
        stores = [s["k_pages"].double(), s["v_pages"].double(), s["k_scale"].double(), s["v_scale"].double(),
                  s["k_open"].double(), s["v_open"].double()]
        for b in range(B):
            rows = s["index"][b, :count[b]].long() if s["index"] is not None else torch.arange(count[b], device="cuda")
            pos = torch.arange(length[b], length[b] + count[b], device="cuda")
            k = _exact_rotate(s["k"][b, rows].double(), s["k_weight"], pos, s["inv_freq"], False)
            for which, x in enumerate((k, s["v"][b, rows].double())):
                x = x.to(torch.bfloat16).double()                            # what the cache is defined to hold
                begin = length[b] // page * page
                ring = stores[4 + which][b]
                held = [ring[:, t % (2 * page)].clone() for t in range(begin, length[b])]
                held = torch.cat((torch.stack(held), x)) if held else x      # tokens from `begin` on [n, Hkv, D]
                done = held.shape[0] // page
                for j in range(done):
                    block = held[j * page:(j + 1) * page].transpose(0, 1)    # [Hkv, page, D]
                    amax = block.abs().amax(dim=(1, 2))
                    m, e = torch.frexp(amax / E4M3_MAX)                      # the next power of two, itself included
                    scale = torch.ldexp(torch.ones_like(amax), torch.where(m > 0.5, e, e - 1))
                    scale = torch.where(amax > 0, scale, torch.ones_like(amax))
                    to = table[b][length[b] // page + j]
                    stores[which][to] = (block / scale[:, None, None]).float().to(torch.float8_e4m3fn).double()
                    stores[2 + which][to] = scale
                t = torch.arange(max(begin + done * page, length[b]), length[b] + count[b], device="cuda")
                ring[:, t % (2 * page)] = held[t - begin].transpose(0, 1)
        return tuple(out + stores)
    q, N, G = s["q"].double(), case["N"], case["Hq"] // Hkv
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float64, device="cuda")
    for b in range(B):
        n = length[b] // page
        ids = s["page_table"][b, :n].long()
        slots = torch.arange(n * page, length[b], device="cuda") % (2 * page)
        mask = torch.ones((N, length[b] + N), dtype=torch.bool, device="cuda")
        words = s["ancestors"][b].long()
        node = torch.arange(N, device="cuda")
        mask[:, length[b]:] = (words[:, node // 32] >> (node % 32)) & 1 == 1
        for h in range(Hkv):
            k, v = (torch.cat(((pages.view(torch.uint8)[ids, h].view(pages.dtype).double() *
                                scale[ids, h].double()[:, None, None]).reshape(-1, D),
                               ring[b, h, slots].double(), nodes[b, :, h].double()))
                    for pages, scale, ring, nodes in ((s["k_pages"], s["k_scale"], s["k_open"], s["k"]),
                                                      (s["v_pages"], s["v_scale"], s["v_open"], s["v"])))
            x = torch.einsum("ngd,td->ngt", q[b, :, h * G:(h + 1) * G], k) / math.sqrt(D)
            x = x.masked_fill(~mask[:, None], NEG)
            lse[b, :, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            out[b, :, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return out, lse
