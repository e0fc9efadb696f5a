"""What is measured of the operators for speculative serving: attention of drafted
token trees over the hybrid cache (tree), block tables resized on the GPU from
request lengths (tables) and slot maps of packed tokens (slots).

A case is a dict with "op".  `run` computes its operator in plain torch
operations, or, where `own` is true, through the package.
"""
import math

import torch

own = False

D = 128            # head dimension
TILE = 64 * D      # bytes of an INT8 K or V tile of 64 tokens
DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a single user's chat: one sequence, 8 heads, four drafted tokens in a chain
        dict(name="tree_one_seq_mha8_L1024", op="tree", batch=1, hq=8, hkv=8, lo=1024, hi=1024, nodes=4, shape="chain",
             bits=8, int4=0.0, hot=32, block=64),
        # a small batch of equal lengths under a 16-node tree
        dict(name="tree_llama3_8b_b8_L2048", op="tree", batch=8, hq=32, hkv=8, lo=2048, hi=2048, nodes=16, shape="tree",
             bits=8, int4=0.0, hot=32, block=64),
        # a serving batch of mixed lengths, eight drafted tokens each
        dict(name="tree_var64_gqa4_L256_8192", op="tree", batch=64, hq=32, hkv=8, lo=256, hi=8192, nodes=8, shape="tree",
             bits=8, int4=0.0, hot=32, block=64),
        # long contexts: 32K to 128K tokens, 32 nodes (128 query rows for each kv head)
        dict(name="tree_long_b4_L32k_128k", op="tree", batch=4, hq=32, hkv=8, lo=32768, hi=131072, nodes=32, shape="tree",
             bits=8, int4=0.0, hot=32, block=64),
        # a mixed load with groups of 7 heads, the oldest quarter of the blocks in INT4, ragged trees
        dict(name="tree_qwen2_7b_b128_mixed_int4", op="tree", batch=128, hq=28, hkv=4, lo=64, hi=8192, nodes=6,
             shape="ragged", bits=8, int4=0.25, hot=32, block=64),
        # the widest trees: 64 nodes, groups of 8 heads (512 query rows for each kv head): bound by the products
        dict(name="tree_wide64_b8_L16k", op="tree", batch=8, hq=64, hkv=8, lo=16384, hi=16384, nodes=64, shape="tree",
             bits=8, int4=0.0, hot=32, block=64),
        # cold zone kept in FP16, 128-token blocks and hot zone, odd node count, short and empty sequences among them
        dict(name="tree_fp16_cold_b16_hot128", op="tree", batch=16, hq=32, hkv=8, lo=0, hi=4001, nodes=21,
             shape="ragged", bits=0, int4=0.0, hot=128, block=128),
        # tables of a small batch that grows by its drafted tokens
        dict(name="tables_b8_L2048", op="tables", batch=8, lo=1, hi=2048, hot=32, block=64, grow=16, turnover=0.1),
        # a serving batch: sequences end, others take their place
        dict(name="tables_b128_L8192", op="tables", batch=128, lo=64, hi=8192, hot=32, block=64, grow=64, turnover=0.2),
        # many long sequences in small blocks
        dict(name="tables_b2048_L32k_block32", op="tables", batch=2048, lo=1, hi=32768, hot=16, block=32, grow=64,
             turnover=0.1),
        # slots of the tokens that a verification step may write, for each sequence
        dict(name="slots_b64_step", op="slots", batch=64, lo=256, hi=8192, hot=32, block=64, span=16),
        # slots of every token of a large batch (moving or reading out whole sequences)
        dict(name="slots_b1024_whole", op="slots", batch=1024, lo=1, hi=8192, hot=32, block=64, span=0),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "tables", "slots"])
    if op == "tree":
        top = 3e-4
        while True:
            hq, hkv = rng.choice([(8, 8), (8, 4), (32, 8), (28, 4), (16, 2), (64, 8)])
            hi = _spread(rng, 1, 131072)
            c = dict(op="tree", batch=_spread(rng, 1, 128), hq=hq, hkv=hkv, lo=rng.randint(0, hi), hi=hi,
                     nodes=_spread(rng, 1, 64), shape=rng.choice(["chain", "tree", "ragged"]),
                     bits=rng.choice([8, 8, 8, 4, 0]), int4=rng.choice([0.0, 0.0, 0.25, 0.6]),
                     hot=rng.choice([16, 32, 32, 64, 128]), block=rng.choice([32, 64, 64, 128]))
            # the padded length bounds what the plain form holds
            padded = c["batch"] * c["hkv"] * c["hi"]
            if _tree_cost(c) <= top and padded <= 5_000_000 and padded * (hq // hkv) * c["nodes"] <= 600_000_000:
                return c
    if op == "tables":
        hi = _spread(rng, 1, 32768)
        return dict(op="tables", batch=_spread(rng, 1, 2048), lo=rng.randint(1, hi), hi=hi,
                    hot=rng.choice([16, 32, 64, 128]), block=rng.choice([32, 64, 128]), grow=_spread(rng, 1, 64),
                    turnover=rng.choice([0.0, 0.1, 0.3]))
    while True:
        hi = _spread(rng, 1, 32768)
        c = dict(op="slots", batch=_spread(rng, 1, 1024), lo=rng.randint(1, hi), hi=hi, hot=rng.choice([16, 32, 64, 128]),
                 block=rng.choice([32, 64, 128]), span=rng.choice([0, 1, 16, 64]))
        if c["batch"] * c["hi"] <= 1024 * 8192:
            return c


def _lens(case, gen):
    """Lengths of a case, spread over [lo, hi] (both ends among them when the
    batch has two sequences): the same set for every seed, in another order."""
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    lens = torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(n + hi))
    if n > 1:
        lens[0], lens[1] = hi, lo
    return lens[torch.randperm(n, generator=gen)]


def _mean_len(case):
    return float(_lens(case, torch.Generator()).double().mean())


# ---------------------------------------------------------------- work

def _tree_parts(case):
    """(bytes, flops), from the mean length."""
    b, hq, hkv, t = case["batch"], case["hq"], case["hkv"], case["nodes"]
    mean = _mean_len(case)
    hot = min(mean, case["hot"])
    cold = mean - hot
    blocks = cold / case["block"]
    per8, per4, per16 = 2 * D, D, 4 * D
    if case["bits"] == 0:
        code = per16
    elif case["bits"] == 4:
        code = per4
    else:
        code = per8 - case["int4"] * (per8 - per4)
    if case["shape"] == "ragged":
        t = 0.5 * (t + 1)
    nbytes = b * (hkv * (cold * code + hot * per16 + t * per16 + (0 if case["bits"] == 0 else blocks * 8)) + blocks * 4
                  + t * hq * (2 * D * 2 + 4) + t * 8)
    flops = 4.0 * D * b * hq * t * (mean + 0.5 * t)
    return nbytes, flops


def _tree_cost(case):
    """Seconds, roughly, that the bytes or the products of a case need."""
    nbytes, flops = _tree_parts(case)
    return max(nbytes / 6.5e12, flops / 1.6e15)


def work(case):
    if case["op"] == "tree":
        nbytes, flops = _tree_parts(case)
        return {"bytes": int(nbytes), "flops": int(flops)}
    b = case["batch"]
    if case["op"] == "tables":
        width = _table_width(case)
        held = _mean_len(case) / case["block"]
        # lengths, counts, the held entries read; the whole table and the counts written; entries moved to and from the ring
        return {"bytes": int(b * (12 + 4 * held + 4 * width + 8 * held * case["turnover"])), "flops": int(b * 8)}
    tokens = b * (min(case["span"], _mean_len(case)) if case["span"] else _mean_len(case))
    return {"bytes": int(8 * tokens + 4 * tokens / case["block"] + 16 * b), "flops": int(4 * tokens)}


# ---------------------------------------------------------------- inputs

def _blocks_for(lens, hot, block):
    return (lens - hot).clamp(min=0).add(block - 1).div(block, rounding_mode="floor")


def _table_width(case):
    return max(1, -(-(case["hi"] + case.get("grow", 0)) // case["block"]))


def _v8_places():
    """Byte of (channel, slot) in an INT8 V tile: 16-slot chunks swizzled by channel."""
    c = torch.arange(D, device=DEV)[:, None]
    t = torch.arange(64, device=DEV)[None, :]
    return (c * 64 + 16 * ((t // 16) ^ ((c // 2) % 4)) + t % 16).reshape(-1)


def _k4_places():
    """(byte, is high nibble) of (slot, channel) in an INT4 K tile."""
    t = torch.arange(64, device=DEV)[:, None]
    c = torch.arange(D, device=DEV)[None, :]
    e = c % 8
    return (t * 64 + (c // 8) * 4 + e % 4).reshape(-1), (e >= 4).expand(64, D).reshape(-1)


def _v4_places():
    """(byte, is high nibble) of (channel, slot) in an INT4 V tile."""
    c = torch.arange(D, device=DEV)[:, None]
    t = torch.arange(64, device=DEV)[None, :]
    e = t % 8
    at = c * 32 + 8 * ((t // 16) ^ ((c // 4) % 4)) + 4 * ((t % 16) // 8) + e % 4
    return at.reshape(-1), (e >= 4).expand(D, 64).reshape(-1)


def _fill_quantized(cold, scales, is4, gen):
    """Codes and scales of standard normal values, in place.  cold uint8
    [phys][hkv][parts][8192]; is4 bool [phys]: blocks held in INT4.  Slots past
    a sequence's length hold codes too: nothing reads them."""
    phys, hkv, parts, _ = cold.shape
    v8 = _v8_places()
    (k4at, k4hi), (v4at, v4hi) = _k4_places(), _v4_places()
    step = max(1, (1 << 26) // (hkv * parts * TILE))
    for p0 in range(0, phys, step):
        n = min(step, phys - p0)
        x = torch.randn((n, hkv, parts // 2, 2, TILE), generator=gen, device=DEV)
        top = x.abs().amax(dim=(2, 4))                        # [n][hkv][2]: the sub-blocks share their scales
        levels = torch.where(is4[p0:p0 + n], 7.0, 127.0)[:, None, None]
        s = top / levels
        scales[p0:p0 + n] = s
        code = torch.round(x / s[:, :, None, :, None]).to(torch.int8)
        out = cold[p0:p0 + n].view(n, hkv, parts // 2, 2, TILE)
        out[:, :, :, 0] = code[:, :, :, 0].view(torch.uint8)  # K: token-major
        v = torch.empty_like(out[:, :, :, 1])
        v[..., v8] = code[:, :, :, 1].view(torch.uint8)       # V: channel-major
        out[:, :, :, 1] = v
        four = is4[p0:p0 + n].nonzero()[:, 0]
        if four.numel():
            nib = (code[four].to(torch.int16) & 15).to(torch.uint8)
            for kv, at, hi in ((0, k4at, k4hi), (1, v4at, v4hi)):
                half = torch.zeros((four.numel(), hkv, parts // 2, TILE), dtype=torch.uint8, device=DEV)
                half[..., at[~hi]] = nib[:, :, :, kv][..., ~hi]
                half[..., at[hi]] |= nib[:, :, :, kv][..., hi] << 4
                out[four, :, :, kv] = half


def _masks(case, n_tree, gen):
    """Ancestor masks int64 [batch][nodes] (bit j: node j is attended; own bit set)."""
    b, t = case["batch"], case["nodes"]
    if case["shape"] == "chain":
        parent = torch.arange(-1, t - 1).expand(b, t)
    else:
        # a random tree for each sequence: the parent is one of the last four nodes, or the root
        back = torch.randint(1, 5, (b, t), generator=gen)
        parent = (torch.arange(t)[None, :] - back).clamp(min=-1)
    mask = torch.zeros((b, t), dtype=torch.int64)
    for j in range(t):
        up = parent[:, j]
        above = torch.gather(mask, 1, up.clamp(min=0)[:, None])[:, 0]
        bit = torch.tensor(1, dtype=torch.int64) << j
        mask[:, j] = torch.where(up >= 0, above, torch.zeros_like(above)) | bit
    return mask


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    if case["op"] == "tables":
        return _prepare_tables(case, cpu)
    if case["op"] == "slots":
        return _prepare_slots(case, cpu)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    b, hq, hkv, t = case["batch"], case["hq"], case["hkv"], case["nodes"]
    hot, block, bits = case["hot"], case["block"], case["bits"]
    lens = _lens(case, cpu)
    nblk = _blocks_for(lens, hot, block)
    phys, width = max(1, int(nblk.sum())), max(1, int(nblk.max()))
    order = torch.randperm(phys, generator=cpu).to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32)
    here = torch.arange(width)[None, :] < nblk[:, None]
    table[here] = order[: int(nblk.sum())]
    n_int4 = (nblk * case["int4"]).floor().to(torch.int32) if bits == 8 and case["int4"] else None
    is4 = torch.zeros(phys, dtype=torch.bool)
    if bits == 4:
        is4[:] = True
    elif n_int4 is not None:
        is4[table[here & (torch.arange(width)[None, :] < n_int4[:, None])].long()] = True
    n_tree = torch.full((b,), t, dtype=torch.int32)
    if case["shape"] == "ragged":
        n_tree = torch.randint(1, t + 1, (b,), generator=cpu).to(torch.int32)
    mask = _masks(case, n_tree, cpu)
    cache = None
    if own:
        from int8_paged_kv_hybrid_b200 import HybridKVCache
        cache = HybridKVCache(b, hkv, hq, phys, width, quant_bits=bits, block_table=table,
                              n_int4=n_int4, hot_tokens=hot, block_size=block, device=DEV)
        ring, cold, scales, table, dev_lens = cache.hot, cache.cold, cache.scales, cache.block_table, cache.seq_lens
        n_int4 = cache.n_int4
    else:
        parts = block // 16 if bits == 0 else 2 * max(1, block // 64)
        ring = torch.zeros((b, hkv, hot, 2, D), dtype=torch.float16, device=DEV)
        cold = torch.zeros((phys, hkv, parts, TILE), dtype=torch.uint8, device=DEV)
        scales = torch.zeros((phys, hkv, 2), dtype=torch.float32, device=DEV)
        table, dev_lens = table.to(DEV), torch.zeros(b, dtype=torch.int32, device=DEV)
        n_int4 = None if n_int4 is None else n_int4.to(DEV)
    dev_lens.copy_(lens)
    ring.copy_(torch.randn(ring.shape, generator=gen, device=DEV))
    if bits == 0:
        flat = cold.view(torch.float16).view(phys, -1)
        step = max(1, (1 << 26) // flat.shape[1])
        for p0 in range(0, phys, step):
            part = flat[p0:p0 + step]
            part.copy_(torch.randn(part.shape, generator=gen, device=DEV))
    else:
        _fill_quantized(cold, scales, is4.to(DEV), gen)
    f16 = lambda *shape: torch.randn(shape, generator=gen, device=DEV).to(torch.float16)  # noqa: E731
    s = dict(case=case, ring=ring, cold=cold, scales=scales, table=table, lens=dev_lens, n_int4=n_int4,
             q=f16(b, t, hq, D), k=f16(b, t, hkv, D), v=f16(b, t, hkv, D), mask=mask.to(DEV), n_tree=n_tree.to(DEV),
             scale=1.0 / math.sqrt(D), top=int(lens.max()),
             out=torch.zeros((b, t, hq, D), dtype=torch.float16, device=DEV),
             lse=torch.zeros((b, t, hq), dtype=torch.float32, device=DEV))
    if own:
        s["cache"], s["workspace"] = cache, cache.tree_workspace(t)
    return s


def _prepare_tables(case, cpu):
    b, hot, block = case["batch"], case["hot"], case["block"]
    lens = _lens(case, cpu)
    held = _blocks_for(lens, hot, block)
    width = _table_width(case)
    # what comes next: most sequences grow by their drafted tokens, some end, some are replaced by others
    new = lens + torch.randint(1, case["grow"] + 1, (b,), generator=cpu)
    dice = torch.rand(b, generator=cpu)
    new = torch.where(dice < 0.5 * case["turnover"], torch.zeros_like(new), new)
    other = torch.randint(case["lo"], case["hi"] + 1, (b,), generator=cpu)
    new = torch.where(dice > 1 - 0.5 * case["turnover"], other, new)
    used = int(held.sum())
    phys = used + used // 4 + b + 64             # a pool without much to spare: some requests may have to wait
    order = torch.randperm(phys, generator=cpu).to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32)
    table[torch.arange(width)[None, :] < held[:, None]] = order[:used]
    head = int(torch.randint(0, phys, (1,), generator=cpu))
    ring = torch.full((phys,), -1, dtype=torch.int32)
    ring[(head + torch.arange(phys - used)) % phys] = order[used:]
    to = lambda x: x.to(torch.int32).to(DEV)     # noqa: E731
    s = dict(case=case, lens=to(new), table=to(table), held=to(held), ring=to(ring),
             state=to(torch.tensor([head, phys - used])), phys=phys)
    if own:
        from int8_paged_kv_hybrid_b200 import BlockPool
        here = BlockPool(b, phys, width, hot_tokens=hot, block_size=block, device=DEV, ring=s["ring"], state=s["state"],
                         n_blocks=s["held"], block_table=s["table"])
        s["pool"], s["next"], s["workspace"] = here, here.successor(), here.workspace()
    return s


def _prepare_slots(case, cpu):
    b, hot, block = case["batch"], case["hot"], case["block"]
    lens = _lens(case, cpu)
    nblk = _blocks_for(lens, hot, block)
    width, phys = max(1, int(nblk.max())), max(1, int(nblk.sum()))
    table = torch.full((b, width), -1, dtype=torch.int32)
    table[torch.arange(width)[None, :] < nblk[:, None]] = torch.randperm(phys, generator=cpu).to(torch.int32)[: int(nblk.sum())]
    n_tok = lens if case["span"] == 0 else torch.clamp(lens, max=case["span"])
    first = lens - n_tok
    total = int(n_tok.sum())
    to = lambda x: x.to(torch.int32).to(DEV)     # noqa: E731
    s = dict(case=case, lens=to(lens), first=to(first), n_tok=to(n_tok), table=to(table), total=total, phys=phys,
             cu=torch.zeros(b + 1, dtype=torch.int32, device=DEV),
             slots=torch.zeros(total, dtype=torch.int64, device=DEV))
    if own:
        from int8_paged_kv_hybrid_b200 import BlockPool
        s["pool"] = BlockPool(b, phys, width, hot_tokens=hot, block_size=block, device=DEV, block_table=s["table"],
                              n_blocks=to(nblk))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        if op == "tree":
            s["cache"].tree_decode(s["q"], s["k"], s["v"], s["mask"], s["scale"], n_tree=s["n_tree"], out=s["out"],
                                   lse=s["lse"], workspace=s["workspace"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "tables":
            nxt = s["next"]
            s["pool"].resize(s["lens"], to=nxt, workspace=s["workspace"])
            return {"table": nxt.block_table, "n_blocks": nxt.n_blocks, "state": nxt.state, "ring": nxt.ring}
        s["pool"].slot_map(s["lens"], s["n_tok"], s["total"], first=s["first"], cu=s["cu"], slots=s["slots"])
        return {"cu": s["cu"], "slots": s["slots"]}
    return {"tree": _plain_tree, "tables": _plain_tables, "slots": _plain_slots}[op](s)


def _plain_codes(cold, is4):
    """K [.., slots, 128] and V [.., 128, slots] codes of every 64-token sub-block, FP32."""
    k = cold[..., 0, :].view(torch.int8).float()
    v = cold[..., 1, :].index_select(-1, _v8_places()).view(torch.int8).float()
    if is4 is not None:
        nib = lambda x: ((x.to(torch.int16) ^ 8) - 8).float()  # noqa: E731
        (ka, kh), (va, vh) = _k4_places(), _v4_places()
        k4 = (cold[..., 0, :].index_select(-1, ka) >> (kh.to(torch.uint8) * 4)) & 15
        v4 = (cold[..., 1, :].index_select(-1, va) >> (vh.to(torch.uint8) * 4)) & 15
        k, v = torch.where(is4, nib(k4), k), torch.where(is4, nib(v4), v)
    return k.unflatten(-1, (64, D)), v.unflatten(-1, (D, 64)).transpose(-1, -2)


def _plain_tree(s):
    c = s["case"]
    b, hq, hkv, t, hot, block, bits = c["batch"], c["hq"], c["hkv"], c["nodes"], c["hot"], c["block"], c["bits"]
    lens = s["lens"].long()
    cold_len = (lens - hot).clamp(min=0)
    nb = s["table"].shape[1]
    at = s["table"].clamp(min=0).long()
    blocks = s["cold"][at]                                              # [b][nb][hkv][parts][8192]
    if bits == 0:
        rows = blocks.view(torch.float16).view(b, nb, hkv, block, 2, D)
        k, v = rows[..., 0, :].float(), rows[..., 1, :].float()
    else:
        n4 = s["n_int4"]
        if bits == 4:
            is4 = torch.ones((b, nb, 1, 1, 1), dtype=torch.bool, device=DEV)
        elif n4 is not None:
            is4 = (torch.arange(nb, device=DEV)[None, :] < n4[:, None])[:, :, None, None, None]
        else:
            is4 = None
        k, v = _plain_codes(blocks.unflatten(3, (-1, 2)), is4)          # [b][nb][hkv][sub][64][128]
        k, v = (x.reshape(b, nb, hkv, -1, D)[:, :, :, :block] for x in (k, v))
        sc = s["scales"][at]                                            # [b][nb][hkv][2]
        k, v = k * sc[..., 0, None, None], v * sc[..., 1, None, None]
    k, v = (x.transpose(1, 2).reshape(b, hkv, nb * block, D) for x in (k, v))
    # the ring's rows are attended in ring order; slot r holds a token when the sequence has reached it
    ring = s["ring"].float()
    k = torch.cat([k, ring[..., 0, :], s["k"].float().transpose(1, 2)], 2)
    v = torch.cat([v, ring[..., 1, :], s["v"].float().transpose(1, 2)], 2)
    pos = torch.arange(nb * block, device=DEV)
    seen = torch.cat([pos[None, :] < cold_len[:, None],
                      torch.arange(hot, device=DEV)[None, :] < lens[:, None]], 1)   # [b][cached]
    node = torch.arange(t, device=DEV)
    alive = node[None, :] < s["n_tree"][:, None]                                    # [b][t]
    anc = ((s["mask"][:, :, None] >> node) & 1).bool() & alive[:, None, :]          # [b][t][t]
    ok = torch.cat([seen[:, None, :].expand(b, t, -1), anc], 2)[:, None, None]      # [b][1][1][t][keys]
    q = s["q"].float().view(b, t, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4)         # [b][hkv][g][t][128]
    z = torch.matmul(q.reshape(b, hkv, -1, D), k.transpose(-1, -2)).view(b, hkv, hq // hkv, t, -1)
    z = torch.where(ok, z * s["scale"], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hkv, -1, p.shape[-1]), v).view(b, hkv, hq // hkv, t, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (torch.log(total) + top)[..., 0]
    live = alive[:, None, None, :]
    o, lse = torch.where(live[..., None], o, 0.0), torch.where(live, lse, 0.0)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(b, t, hq, D).to(torch.float16),
            "lse": lse.permute(0, 3, 1, 2).reshape(b, t, hq)}


def _plain_tables(s):
    c, phys = s["case"], s["phys"]
    held, table, ring = s["held"].long(), s["table"], s["ring"]
    width = table.shape[1]
    want = _blocks_for(s["lens"].long(), c["hot"], c["block"])
    want = torch.where(want <= width, want, held)                  # beyond the table: left unchanged
    need, back = (want - held).clamp(min=0), (held - want).clamp(min=0)
    head, count = s["state"][0].long(), s["state"][1].long()
    upto = need.cumsum(0)
    fits = (upto <= count) | (need == 0)
    new = torch.where(fits, want, held)
    taken = torch.where(fits, need, 0).sum()
    col = torch.arange(width, device=DEV)[None, :]
    at = (head + (upto - need)[:, None] + (col - held[:, None])) % phys
    fresh = ring.index_select(0, at.reshape(-1)).view_as(at).to(torch.int32)
    out = torch.where(col < torch.minimum(held, new)[:, None], table, torch.where(col < new[:, None], fresh, -1))
    gone = (col >= new[:, None]) & (col < held[:, None])
    place = (head + count + (back.cumsum(0) - back)[:, None] + (col - new[:, None])) % phys
    ring = ring.clone()
    ring[place[gone]] = table[gone]
    state = torch.stack([(head + taken) % phys, count - taken + back.sum()]).to(torch.int32)
    return {"table": out.to(torch.int32), "n_blocks": new.to(torch.int32), "state": state, "ring": ring}


def _plain_slots(s):
    c = s["case"]
    hot, block = c["hot"], c["block"]
    n_tok = s["n_tok"].long()
    cu = torch.cat([n_tok.new_zeros(1), n_tok.cumsum(0)])
    seq = torch.repeat_interleave(torch.arange(c["batch"], device=DEV), n_tok, output_size=s["total"])
    pos = torch.arange(s["total"], device=DEV) - cu[seq] + s["first"].long()[seq]
    length = s["lens"].long()[seq]
    entry = s["table"][seq, (pos // block).clamp(max=s["table"].shape[1] - 1)].long()
    slots = torch.where(pos < length - hot, entry * block + pos % block, -2 - (seq * hot + pos % hot))
    return {"cu": cu.to(torch.int32), "slots": torch.where((pos >= 0) & (pos < length), slots, -1)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The tree's attention from its definition, sequence by sequence, in 64
    bits; None for the operators whose outputs are whole numbers."""
    if case["op"] != "tree":
        return None
    s = prepare(case, seed)
    b, hq, hkv, t, hot, block, bits = (case[x] for x in ("batch", "hq", "hkv", "nodes", "hot", "block", "bits"))
    g = hq // hkv
    out = torch.zeros((b, t, hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((b, t, hq), dtype=torch.float64, device=DEV)
    lens, trees = s["lens"].tolist(), s["n_tree"].tolist()
    fours = [0] * b if s["n_int4"] is None else s["n_int4"].tolist()
    byte = s["cold"].view(-1)
    half = byte.view(torch.float16)
    ch = torch.arange(D, device=DEV)
    per = s["cold"].shape[2] * TILE
    for i in range(b):
        n, cold = lens[i], max(0, lens[i] - hot)
        if trees[i] == 0:
            continue
        p = torch.arange(cold, device=DEV)
        phys = s["table"][i].long()[p // block]
        four = (p // block < fours[i])[:, None] if bits == 8 else torch.full((cold, 1), bits == 4, device=DEV)
        slot = p % block
        ringpos = torch.arange(cold, n, device=DEV) % hot
        bits_of = (s["mask"][i, :trees[i], None] >> torch.arange(trees[i], device=DEV)) & 1
        ok = torch.cat([torch.ones((trees[i], n), dtype=torch.int64, device=DEV), bits_of], 1) == 1
        for h in range(hkv):
            base = (phys * hkv + h) * per
            rows = []
            for kv in (0, 1):
                if bits == 0:
                    at = base // 2 + slot * 2 * D + kv * D
                    x = half[at[:, None] + ch].double()
                else:
                    tile = base + (slot // 64) * 2 * TILE + kv * TILE
                    u = slot[:, None] % 64
                    if kv == 0:
                        at8, at4, e = u * 128 + ch, u * 64 + ch // 8 * 4 + ch % 4, ch % 8 + 0 * u
                    else:
                        at8 = ch * 64 + ((u // 16) ^ (ch // 2 % 4)) * 16 + u % 16
                        at4 = ch * 32 + ((u // 16) ^ (ch // 4 % 4)) * 8 + (u % 16 // 8) * 4 + u % 4
                        e = u % 8 + 0 * ch
                    raw8 = byte[tile[:, None] + at8].long()
                    raw4 = byte[tile[:, None] + at4].long() // torch.where(e % 8 >= 4, 16, 1) % 16
                    code = torch.where(four, raw4 - 16 * (raw4 >= 8), raw8 - 256 * (raw8 >= 128))
                    x = code.double() * s["scales"][phys, h, kv].double()[:, None]
                new = (s["k"] if kv == 0 else s["v"])[i, :trees[i], h].double()
                rows.append(torch.cat([x, s["ring"][i, h, ringpos, kv].double(), new]))
            for j in range(g):
                z = s["q"][i, :trees[i], h * g + j].double() @ rows[0].T * s["scale"]
                z = z.masked_fill(~ok, -math.inf)
                e = torch.logsumexp(z, 1)
                w = torch.exp(z - e.nan_to_num(neginf=0.0)[:, None])
                out[i, :trees[i], h * g + j] = w @ rows[1]
                lse[i, :trees[i], h * g + j] = e
    return {"out": out, "lse": lse}
