"""hyb_pool_resize and hyb_slot_map on the GPU against sequential models, and
the calls of one verification step together."""
import numpy as np
import pytest

from harness import make_pair
from int8_paged_kv_hybrid_b200 import BlockPool, HybridKVCache, _lib, synth, tree_masks
from tree_ref import PoolModel, cached_kv, slot_map, tree_attention

pytestmark = pytest.mark.gpu


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def assert_pool(pool, model, what=""):
    table, n = pool.block_table.cpu().numpy(), pool.n_blocks.cpu().numpy()
    head, count = pool.state.tolist()
    ring = pool.ring.cpu().numpy()
    assert n.tolist() == [len(h) for h in model.held], what
    for b, h in enumerate(model.held):
        assert table[b, :len(h)].tolist() == h and (table[b, len(h):] == -1).all(), (what, b)
    assert head == model.head and count == len(model.free), what
    assert ring[(head + np.arange(count)) % model.phys].tolist() == model.free, what


@pytest.mark.parametrize("batch,width,phys,hot,block", [
    (1, 1, 1, 16, 32), (1, 700, 900, 32, 64), (3, 4, 8, 32, 64), (8, 33, 200, 32, 64), (150, 20, 1500, 128, 128),
    (2500, 6, 7000, 32, 32), (300, 513, 40000, 16, 64),
])
@pytest.mark.parametrize("place", ["in place", "successor", "mixed"])
def test_random_walk(batch, width, phys, hot, block, place):
    """Sequences grow, shrink and end over many calls; pools run dry."""
    rng = np.random.default_rng([batch, width])
    pool = BlockPool(batch, phys, width, hot_tokens=hot, block_size=block)
    model = PoolModel(batch, phys, width, hot, block)
    ws = pool.workspace()
    lens = np.zeros(batch, np.int64)
    for call in range(12):
        grow = rng.integers(0, 2 * block + 2, size=batch)
        lens = np.minimum(lens + grow, hot + width * block)
        anew = rng.random(batch) < 0.2
        lens[anew] = rng.integers(0, hot + width * block + 1, size=batch)[anew] * (rng.random(batch) < 0.7)[anew]
        refused = model.resize(lens.tolist())
        if place == "in place":
            pool.resize(dev(lens), workspace=ws)
        elif place == "successor":
            pool = pool.resize(dev(lens), to=pool.successor(), workspace=ws)
        else:                                      # the table in place, the counts and state in other memory
            nxt = pool.successor()
            nxt.block_table, nxt.desc.block_table = pool.block_table, pool.desc.block_table
            pool = pool.resize(dev(lens), to=nxt, workspace=ws)
        assert_pool(pool, model, "call %d" % call)
        assert pool.status(clear=True) == (_lib.HYB_STATUS_POOL if refused else 0), call
        lens = np.array([max(min(n, hot), hot + block * (len(h) - 1) + 1 if h else 0) if b in set(refused) else n
                         for b, (n, h) in enumerate(zip(lens, model.held))])


def test_refused_sequences_and_bad_counts():
    pool = BlockPool(5, 40, 4)
    pool.resize(dev([100, 200, 40, 0, 288]))                       # 2, 3, 1, 0, 4 blocks
    assert pool.status() == 0
    table = pool.block_table.cpu().numpy().copy()
    nxt = pool.resize(dev([100, -1, 40, 64, 289]), to=pool.successor())
    assert nxt.n_blocks.tolist() == [2, 3, 1, 1, 4] and pool.status(clear=True) in (
        _lib.HYB_STATUS_SEQ_LEN, _lib.HYB_STATUS_CAPACITY)
    table[3, 0] = 10
    assert np.array_equal(nxt.block_table.cpu().numpy(), table)
    # a count outside the table: that sequence stays, whatever its row holds
    for bad in (-1, 5):
        nxt.n_blocks[1] = bad
        got = nxt.resize(dev([100, 0, 0, 64, 288]), to=nxt.successor())
        assert got.n_blocks.tolist() == [2, bad, 0, 1, 4]
        assert got.block_table[1].tolist() == table[1].tolist()
        assert nxt.status(clear=True) == _lib.HYB_STATUS_CAPACITY
    # a pool whose counts contradict each other: nothing changes
    nxt.n_blocks[1] = 3
    for head, count in ((-1, 5), (40, 5), (0, -1), (0, 41), (3, 39)):
        nxt.state.copy_(dev([head, count]))
        ring = nxt.ring.clone()
        got = nxt.resize(dev([0, 0, 0, 0, 0]), to=nxt.successor())
        assert got.n_blocks.tolist() == [2, 3, 1, 1, 4] and got.state.tolist() == [head, count]
        assert np.array_equal(got.block_table.cpu().numpy(), table) and bool((ring == nxt.ring).all())
        assert nxt.status(clear=True) == _lib.HYB_STATUS_POOL
    # an entry of the ring that is no block
    pool = BlockPool(1, 8, 4)
    pool.ring[1] = 8
    pool.resize(dev([200]))
    assert pool.status(clear=True) == _lib.HYB_STATUS_BAD_BLOCK


def test_captured_in_place():
    import torch
    pool, model = BlockPool(70, 600, 9), PoolModel(70, 600, 9, 32, 64)
    ws, lens = pool.workspace(), torch.zeros(70, dtype=torch.int32, device="cuda")
    pool.resize(lens, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.resize(lens, workspace=ws)
    rng = np.random.default_rng(3)
    for _ in range(6):
        n = rng.integers(0, 500, size=70)
        lens.copy_(dev(n))
        g.replay()
        model.resize(n.tolist())
        assert_pool(pool, model)


@pytest.mark.parametrize("batch,hi,hot,block", [(1, 1, 16, 32), (5, 300, 32, 64), (64, 2000, 64, 128), (3000, 90, 16, 32),
                                                (2, 70000, 128, 64)])
@pytest.mark.parametrize("whole", [True, False])
def test_slot_map(batch, hi, hot, block, whole):
    rng = np.random.default_rng([batch, hi])
    lens = rng.integers(0, hi + 1, size=batch)
    lens[0] = hi
    width = max(1, -(-max(0, hi - hot) // block))
    phys = batch * width + 3
    table = rng.permutation(phys)[:batch * width].reshape(batch, width)
    pool = BlockPool(batch, phys, width, hot_tokens=hot, block_size=block, block_table=dev(table))
    if whole:
        first, n = np.zeros(batch, int), lens
    else:                                          # windows that start before and end behind the sequence
        first = rng.integers(-5, hi + 5, size=batch)
        n = rng.integers(0, 40, size=batch)
    cu, want = slot_map(table, lens, first, n, hot, block)
    import torch
    slots = torch.full((len(want) + 5,), -99, dtype=torch.int64, device="cuda")
    got_cu, _ = pool.slot_map(dev(lens), dev(n), len(want) + 5, first=None if whole else dev(first), slots=slots)
    assert np.array_equal(got_cu.cpu().numpy(), cu)
    assert np.array_equal(slots[:len(want)].cpu().numpy(), want) and (slots[len(want):] == -99).all()
    assert pool.status() == 0
    # too little room: the rest is dropped
    room = len(want) // 2
    slots.fill_(-99)
    got_cu, _ = pool.slot_map(dev(lens), dev(n), room, first=None if whole else dev(first), slots=slots[:room])
    assert np.array_equal(slots[:room].cpu().numpy(), want[:room]) and (slots[room:] == -99).all()
    assert np.array_equal(got_cu.cpu().numpy(), np.minimum(cu, room))
    assert pool.status(clear=True) == (_lib.HYB_STATUS_CAPACITY if room < len(want) else 0)


def test_slot_map_errors():
    pool = BlockPool(3, 10, 2, block_table=dev([[0, 10], [3, -1], [5, 6]]))
    cu, s = pool.slot_map(dev([200, 96, 400]), dev([200, -4, 300]), 500)
    assert pool.status(clear=True) in (_lib.HYB_STATUS_BAD_N_NEW, _lib.HYB_STATUS_BAD_BLOCK)
    assert cu.tolist() == [0, 200, 200, 500]
    s = s.cpu().numpy()
    assert s[:64].tolist() == list(range(64)) and (s[64:128] == -1).all()      # block 10 does not exist
    assert s[168:200].tolist() == [-2 - p % 32 for p in range(168, 200)]
    assert s[200:264].tolist() == list(range(320, 384)) and (s[328:] == -1).all()  # beyond the table's columns


def test_verification_steps_together():
    """Tables from lengths, the drafted tree over the cache, the accepted path
    appended: four steps, the cache bit for bit and the attention within its
    bound, with slots that find every cached token's codes."""
    import torch
    batch, hq, hkv, nodes, width = 5, 8, 2, 6, 12
    rng = np.random.default_rng(12)
    start = np.array([0, 20, 100, 300, 33])
    pool = BlockPool(batch, 40, width)
    cache = HybridKVCache(batch, hkv, hq, 40, width, block_table=pool.block_table)
    assert cache.block_table.data_ptr() == pool.block_table.data_ptr()
    w = synth.custom_workload("steps", [32 + 64 * width] * batch, hq, hkv, seed=1)
    _, ora = make_pair(w, gpu=False)
    ws, pool_ws = cache.tree_workspace(nodes), pool.workspace()
    parents = np.array([-1, 0, 0, 1, 1, 2])
    mask = np.repeat(tree_masks(parents)[None], batch, 0)
    paths = [[0], [0, 1, 4], [0, 2, 5], [], [0, 2]]
    half = lambda *s: rng.standard_normal(s).astype(np.float16)  # noqa: E731
    cuda = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731

    def append(k, v, n):
        ora.append(n.astype(np.int32), k, v)
        cache.append(dev(n), cuda(k), cuda(v))

    pool.resize(dev(start), workspace=pool_ws)
    append(half(batch, 300, hkv, 128), half(batch, 300, hkv, 128), start)
    scale = 0.088
    for _ in range(4):
        lens = ora.lens()
        pool.resize(dev(lens + nodes), workspace=pool_ws)
        q, k, v = half(batch, nodes, hq, 128), half(batch, nodes, hkv, 128), half(batch, nodes, hkv, 128)
        out = cache.tree_decode(cuda(q), cuda(k), cuda(v), cuda(mask), scale, workspace=ws).float().cpu().numpy()
        for b in range(batch):
            kk, vv = cached_kv(ora, b, int(lens[b]))
            o, _, tol, _ = tree_attention(kk, vv, q[b], k[b], v[b], mask[b], nodes, scale)
            assert (np.abs(out[b] - o) <= tol).all(), b
        n = np.array([len(p) for p in paths])
        ka, va = np.zeros((batch, 3, hkv, 128), np.float16), np.zeros((batch, 3, hkv, 128), np.float16)
        for b, p in enumerate(paths):
            ka[b, :len(p)], va[b, :len(p)] = k[b, p], v[b, p]
        append(ka, va, n)
    assert cache.status() == 0 and pool.status() == 0
    # the codes of every cold token through the slot map, against the oracle's
    lens = ora.lens()
    cu, slots = pool.slot_map(cache.seq_lens, cache.seq_lens, int(lens.sum()))
    cu, slots = cu.cpu().numpy(), slots.cpu().numpy()
    cold, scales = cache.cold.view(torch.int8).cpu().numpy(), cache.scales.cpu().numpy()
    for b in range(batch):
        kk, _ = cached_kv(ora, b, int(lens[b]))
        s = slots[cu[b]:cu[b + 1]]
        c = max(0, lens[b] - 32)
        got = cold[s[:c] // 64, :, 0].reshape(c, hkv, 64, 128)[np.arange(c), :, s[:c] % 64].astype(np.float64)
        got *= scales[s[:c] // 64, :, 0].astype(np.float64)[:, :, None]
        assert np.array_equal(got.transpose(1, 0, 2), kk[:, :c])
        ring = cache.hot[b].cpu().numpy().astype(np.float64)
        assert np.array_equal(ring[:, (-2 - s[c:]) % 32, 0], kk[:, c:]) and ((-2 - s[c:]) // 32 == b).all()


def busy(stream, scratch):
    """Copies that keep a stream at work for some milliseconds."""
    import torch
    with torch.cuda.stream(stream):
        for _ in range(20):
            scratch[1].copy_(scratch[0])


@pytest.mark.parametrize("raw", [False, True])
def test_calls_on_another_stream_make_their_own_buffers(raw):
    """tree_decode, resize in place and slot_map on a side stream, without
    buffers, first while the current stream is at work, then while the side stream
    is and the current one takes and fills memory of the same sizes."""
    import torch
    batch, hq, hkv, nodes, width = 6, 8, 2, 5, 6
    rng = np.random.default_rng(3)
    half = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float16)).cuda()  # noqa: E731
    pool, model = BlockPool(batch, 40, width), PoolModel(batch, 40, width, 32, 64)
    cache = HybridKVCache(batch, hkv, hq, 40, width, block_table=pool.block_table)
    lens = np.array([0, 20, 100, 300, 33, 400])
    model.resize(lens.tolist())
    pool.resize(dev(lens))
    cache.append(dev(lens), half(batch, 400, hkv, 128), half(batch, 400, hkv, 128))
    q, k, v = half(batch, nodes, hq, 128), half(batch, nodes, hkv, 128), half(batch, nodes, hkv, 128)
    n_tree = dev([5, 0, 3, 5, 1, 2])
    want = cache.tree_decode(q, k, v, None, 0.09, n_tree=n_tree)
    room = int(lens.sum()) + 9
    want_cu, want_slots = pool.slot_map(dev(lens), dev(lens), room)
    scratch = torch.empty((2, 1 << 28), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    s = side.cuda_stream if raw else side
    torch.cuda.synchronize()
    for turn in range(4):
        lens = rng.integers(0, 32 + 64 * width, size=batch)
        now, of = dev(lens), dev([0, 20, 100, 300, 33, 400])
        torch.cuda.synchronize()
        busy(torch.cuda.current_stream() if turn % 2 == 0 else side, scratch)
        got = cache.tree_decode(q, k, v, None, 0.09, n_tree=n_tree, stream=s)
        cu, slots = pool.slot_map(of, of, room, stream=s) if turn == 0 else (want_cu, want_slots)
        pool.resize(now, stream=s)
        if turn % 2:
            for n in (cache.tree_workspace(nodes).numel(), pool.workspace().numel(), 2 * q.numel()):
                for _ in range(3):
                    torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        refused = model.resize(lens.tolist())
        assert_pool(pool, model, turn)
        assert pool.status(clear=True) == (_lib.HYB_STATUS_POOL if refused else 0)
        assert torch.equal(cu, want_cu) and torch.equal(slots, want_slots)
        if turn == 0:
            assert torch.equal(got, want)
        else:                                      # the table is another one now
            assert bool((got[1] == 0).all()) and bool((got[2, 3:] == 0).all())
    assert torch.cuda.current_stream().cuda_stream != side.cuda_stream


def test_the_stream_of_another_device_is_refused(monkeypatch):
    import torch
    pool = BlockPool(1, 4, 2)
    other = torch.cuda.Stream()
    pool.device = torch.device("cuda", torch.cuda.current_device() + 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: other)
    monkeypatch.setattr(pool, "_check", lambda *a: None)
    with pytest.raises(_lib.HybError):
        pool.resize(dev([1]), stream=other)


def test_steps_with_successors():
    """Each step's tables are built into the other of two pools, which the cache
    then takes: appends and attention as with one table resized in place."""
    import torch
    batch, hq, hkv, nodes, width = 4, 8, 2, 4, 8
    rng = np.random.default_rng(5)
    half = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float16)).cuda()  # noqa: E731
    pools = [BlockPool(batch, 30, width)]
    pools.append(pools[0].successor())
    inplace = BlockPool(batch, 30, width)
    cache, other = (HybridKVCache(batch, hkv, hq, 30, width, block_table=p.block_table) for p in (pools[0], inplace))
    lens = np.zeros(batch, int)
    for step in range(5):
        n = rng.integers(0, 90, size=batch)
        lens = lens + n
        now = pools[step % 2].resize(dev(lens + nodes), to=pools[1 - step % 2])
        cache.use_table(now.block_table)
        inplace.resize(dev(lens + nodes))
        assert torch.equal(now.block_table, inplace.block_table)
        k, v = half(batch, 90, hkv, 128), half(batch, 90, hkv, 128)
        q, kt, vt = half(batch, nodes, hq, 128), half(batch, nodes, hkv, 128), half(batch, nodes, hkv, 128)
        outs = []
        for c in (cache, other):
            c.append(dev(n), k, v)
            outs.append(c.tree_decode(q, kt, vt, None, 0.09))
            assert c.status() == 0
        assert torch.equal(outs[0], outs[1]) and torch.equal(cache.cold, other.cold)
        pools[step % 2].block_table.fill_(-7)       # the table of the last step is not read any more
    assert pools[0].status() == 0 and inplace.status() == 0
