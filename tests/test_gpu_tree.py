"""hyb_tree_attn on the GPU against FP64 attention over the oracle's cache.
Every element is held to a bound that is derived in tree_ref.tree_attention
from the roundings the kernel may make."""
import numpy as np
import pytest

from harness import make_pair, replay
from int8_paged_kv_hybrid_b200 import _lib, synth, tree_masks
from tree_ref import cached_kv, random_masks, tree_attention

pytestmark = pytest.mark.gpu

LENS = [0, 1, 5, 31, 32, 33, 64, 95, 96, 97, 130, 161, 255, 700, 1201]
MARK = 777.0   # rows that the call must leave as they were


def inputs(w, nodes, seed, q_gain=1.0):
    rng = np.random.default_rng([seed, 9])
    q = (rng.standard_normal((w.batch, nodes, w.num_q_heads, 128)) * q_gain).astype(np.float16)
    k, v = (rng.standard_normal((w.batch, nodes, w.num_kv_heads, 128)).astype(np.float16) for _ in range(2))
    return q, k, v


def run(cache, q, k, v, mask, n_tree, scale, workspace=None):
    import torch
    dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    out = torch.full(q.shape, MARK, dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:3], MARK, dtype=torch.float32, device="cuda")
    cache.tree_decode(dev(q), dev(k), dev(v), dev(mask), scale, n_tree=dev(n_tree), out=out, lse=lse,
                      workspace=workspace)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def check(w, ora, got, lse, q, k, v, mask, n_tree, scale, lens=None, seqs=None):
    nodes = q.shape[1]
    lens = ora.lens() if lens is None else lens
    chain = tree_masks(np.arange(-1, nodes - 1))
    for b in range(w.batch) if seqs is None else seqs:
        n = nodes if n_tree is None else int(n_tree[b])
        kk, vv = cached_kv(ora, b, int(lens[b]))
        o, l, tol_o, tol_l = tree_attention(kk, vv, q[b], k[b], v[b], chain if mask is None else mask[b], n, scale)
        over = np.abs(got[b, :n] - o) - tol_o
        assert (over <= 0).all(), "sequence %d (L=%d): %g over, at %s" % (
            b, lens[b], over.max(), np.unravel_index(over.argmax(), over.shape))
        none = np.isneginf(l)
        assert np.isneginf(lse[b, :n][none]).all() and (got[b, :n][none] == 0).all(), b
        assert (np.abs(lse[b, :n][~none] - l[~none]) <= tol_l[~none]).all(), b
        assert (got[b, n:] == MARK).all() and (lse[b, n:] == MARK).all(), "rows behind sequence %d's tree" % b


def ragged(rng, batch, nodes):
    n = rng.integers(0, nodes + 1, size=batch).astype(np.int32)
    n[0], n[-1] = nodes, nodes
    return n


def case(hq, hkv, nodes, kind, bits=8, int4=False, hot=32, block=64, lens=LENS, gain=1.0, seed=1):
    nb = [synth.cold_blocks_for(n, hot, block) for n in lens]
    w = synth.custom_workload("tree", lens, hq, hkv, seed=seed + 7 * nodes + hq, max_step=64, hot=hot, block=block,
                              n_int4=[n // 3 for n in nb] if int4 else None)
    cache, ora = make_pair(w, quant_bits=bits)
    replay(w, cache, ora)
    rng = np.random.default_rng(seed)
    q, k, v = inputs(w, nodes, seed, gain)
    mask = None if kind == "chain" else random_masks(rng, w.batch, nodes, "tree" if kind == "ragged" else kind)
    n_tree = ragged(rng, w.batch, nodes) if kind == "ragged" else None
    before = [x.clone() for x in (cache.hot, cache.cold, cache.scales, cache.seq_lens)]
    got, lse = run(cache, q, k, v, mask, n_tree, w.softmax_scale)
    check(w, ora, got, lse, q, k, v, mask, n_tree, w.softmax_scale)
    assert cache.status() == 0
    for x, y in zip(before, (cache.hot, cache.cold, cache.scales, cache.seq_lens)):
        assert bool((x == y).all()), "the cache is only read"


@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 4), (32, 8), (28, 4), (16, 2)])
@pytest.mark.parametrize("nodes,kind", [(1, "chain"), (4, "tree"), (17, "ragged"), (64, "any")])
def test_heads_and_nodes(hq, hkv, nodes, kind):
    lens = LENS if nodes < 64 else LENS[::3] + [1201]
    case(hq, hkv, nodes, kind, lens=lens)


@pytest.mark.parametrize("bits,int4", [(4, False), (8, True), (0, False)])
@pytest.mark.parametrize("hot,block", [(32, 64), (16, 32), (64, 128), (128, 64), (128, 128), (32, 32)])
def test_tiers_and_geometry(bits, int4, hot, block):
    case(8, 2, 9, "ragged", bits=bits, int4=int4, hot=hot, block=block,
         lens=[0, 3, hot, hot + 1, hot + 31, hot + 33, hot + 64, hot + 129, hot + 160, 515, 901], seed=hot + block)


@pytest.mark.parametrize("nodes", [2, 3, 5, 16, 31, 32, 33, 63])
def test_odd_node_counts(nodes):
    case(28, 4, nodes, "tree", lens=[0, 77, 300], seed=nodes)


def test_peaked_logits():
    """q x 8: the softmax is nearly one-hot, running maxima jump between tiles."""
    case(8, 2, 6, "tree", lens=[40, 600, 1500], gain=8.0)
    case(8, 2, 6, "tree", lens=[40, 600], bits=0, gain=8.0)


def test_growing_maxima():
    """Keys whose logits grow along the sequence: every tile raises the
    maximum, by much more than the sums may lag."""
    import torch
    w = synth.custom_workload("grow", [1100, 530], 4, 2, seed=5, schedule="one")
    cache, ora = make_pair(w)
    k, v = synth.step_tokens(w, 0, w.schedule[0])
    k = (k.astype(np.float32) * np.linspace(0.05, 4.0, k.shape[1])[None, :, None, None]).astype(np.float16)
    k = np.abs(k)
    ora.append(w.schedule[0], k, v)
    cache.append(torch.from_numpy(w.schedule[0]).cuda(), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
    q, kt, vt = inputs(w, 5, 3)
    q = np.abs(q)
    got, lse = run(cache, q, kt, vt, None, None, w.softmax_scale)
    check(w, ora, got, lse, q, kt, vt, None, None, w.softmax_scale)
    got, lse = run(cache, -q, kt, vt, None, None, w.softmax_scale)      # and fall
    check(w, ora, got, lse, -q, kt, vt, None, None, w.softmax_scale)


def test_scales_far_apart():
    """Blocks whose V differ by 10^5 in size, and an all-zero block."""
    import torch
    w = synth.custom_workload("apart", [32 + 64 * 9 + 11], 4, 2, seed=6, schedule="chunk", chunk=64)
    cache, ora = make_pair(w)
    for si, n in enumerate(w.schedule):
        k, v = synth.step_tokens(w, si, n)
        v = (v.astype(np.float32) * [1.0, 1e-4, 300.0, 0.0, 1e-5][si % 5]).astype(np.float16)
        ora.append(n, k, v)
        cache.append(torch.from_numpy(n).cuda(), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
    q, kt, vt = inputs(w, 7, 3)
    mask = random_masks(np.random.default_rng(1), 1, 7, "tree")
    got, lse = run(cache, q, kt, vt, mask, None, w.softmax_scale)
    check(w, ora, got, lse, q, kt, vt, mask, None, w.softmax_scale)


@pytest.mark.parametrize("scale", [0.0, -0.09])
def test_zero_and_negative_scale(scale):
    w = synth.custom_workload("neg", [0, 40, 333], 8, 4, seed=8)
    cache, ora = make_pair(w)
    replay(w, cache, ora)
    q, k, v = inputs(w, 5, 2)
    got, lse = run(cache, q, k, v, None, None, scale)
    check(w, ora, got, lse, q, k, v, None, None, scale)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_values_that_are_not_attended_do_not_matter(bad):
    """Node 2 (K and V), the rows behind the tree, and unused ring rows hold
    NaN or infinities: only rows that attend node 2 may show them."""
    import torch
    w = synth.custom_workload("nan", [0, 7, 300], 8, 2, seed=8)
    cache, ora = make_pair(w)
    replay(w, cache, ora)
    q, k, v = inputs(w, 9, 2)
    n_tree = np.array([6, 6, 6], np.int32)
    parents = [-1, 0, 0, 1, 3, 0, -1, -1, -1]                     # nobody descends from node 2
    mask = np.repeat(tree_masks(parents)[None], 3, 0)
    want, want_lse = run(cache, q, k, v, mask, n_tree, w.softmax_scale)
    check(w, ora, want, want_lse, q, k, v, mask, n_tree, w.softmax_scale)
    k[:, 2], v[:, 2], k[:, 6:], v[:, 6:], q[:, 6:] = bad, bad, bad, bad, bad
    cache.hot[0] = bad                                            # an empty sequence's ring
    cache.hot[1, :, 7:] = bad                                     # seven tokens: slots 7.. are unused
    got, lse = run(cache, q, k, v, mask, n_tree, w.softmax_scale)
    keep = [0, 1, 3, 4, 5]
    assert np.array_equal(got[:, keep], want[:, keep]) and np.array_equal(lse[:, keep], want_lse[:, keep])
    assert (got[:, 6:] == MARK).all()


def test_an_infinite_value_reaches_the_rows_that_attend_it():
    """V of node 1 has +inf in channel 3: rows that attend it get +inf there and
    exact values elsewhere; the others nothing."""
    w = synth.custom_workload("inf", [300], 8, 2, seed=8)
    cache, ora = make_pair(w)
    replay(w, cache, ora)
    q, k, v = inputs(w, 5, 2)
    mask = tree_masks([[-1, 0, 0, 1, 2]])
    want, _ = run(cache, q, k, v, mask, None, w.softmax_scale)
    v[:, 1, :, 3] = np.inf
    got, _ = run(cache, q, k, v, mask, None, w.softmax_scale)
    with_it = [1, 3]
    assert np.isposinf(got[0, with_it, :, 3]).all()
    rest = np.arange(128) != 3
    assert np.array_equal(got[0][:, :, rest], want[0][:, :, rest])
    assert np.array_equal(got[0, [0, 2, 4]], want[0, [0, 2, 4]])


def test_a_single_node_is_a_decode_step():
    """FP16 cold blocks: appending a token and attending it (hyb_decode_step's
    dense attention) is the tree of one node."""
    import torch
    w = synth.custom_workload("one", [1, 31, 32, 90, 500], 8, 2, seed=4)
    cache, ora = make_pair(w, quant_bits=0)
    replay(w, cache, ora)
    lens = ora.lens() - 1                                         # the last token is the node
    q, _, _ = inputs(w, 1, 1)
    kv = [cached_kv(ora, b, int(n) + 1) for b, n in enumerate(lens)]
    k = np.stack([x[0][:, -1] for x in kv])[:, None].astype(np.float16)
    v = np.stack([x[1][:, -1] for x in kv])[:, None].astype(np.float16)
    step = cache.decode(torch.from_numpy(q[:, 0]).cuda(), w.softmax_scale, int(lens.max()) + 1).float().cpu().numpy()
    # shortening the sequences hides the last token; where the ring was full, the
    # last token took the slot of the position that would be hot again: skip those
    cache.seq_lens.copy_(torch.from_numpy(lens.astype(np.int32)))
    got, _ = run(cache, q, k, v, None, None, w.softmax_scale)
    short = [b for b in range(w.batch) if lens[b] < 32]
    assert len(short) == 3
    assert np.abs(got[short, 0] - step[short]).max() <= 4e-3


def test_device_errors():
    import torch
    w = synth.custom_workload("err", [100, 300, 200, 260], 8, 4, seed=2)
    cache, ora = make_pair(w)
    replay(w, cache, ora)
    q, k, v = inputs(w, 4, 2)
    for bad in (-1, 5):
        got, lse = run(cache, q, k, v, None, np.array([4, bad, 4, 0], np.int32), w.softmax_scale)
        assert cache.status(clear=True) == _lib.HYB_STATUS_BAD_TREE
        check(w, ora, got, lse, q, k, v, None, np.array([4, 0, 4, 0]), w.softmax_scale)   # row 1 left as it was
    for bad in (-3, 32 + 64 * w.max_blocks + 1):
        lens = ora.lens().copy()
        lens[2] = bad
        cache.seq_lens.copy_(torch.from_numpy(lens))
        got, lse = run(cache, q, k, v, None, None, w.softmax_scale)
        assert cache.status(clear=True) == _lib.HYB_STATUS_SEQ_LEN
        assert (got[2] == 0).all() and np.isneginf(lse[2]).all()
        check(w, ora, got, lse, q, k, v, None, None, w.softmax_scale, lens=ora.lens(), seqs=[0, 1, 3])
    cache.seq_lens.copy_(torch.from_numpy(ora.lens()))
    for bad in (-1, w.num_phys_blocks):
        keep = int(cache.block_table[1, 2])
        cache.block_table[1, 2] = bad
        got, lse = run(cache, q, k, v, None, None, w.softmax_scale)
        cache.block_table[1, 2] = keep
        assert cache.status(clear=True) == _lib.HYB_STATUS_BAD_BLOCK
        check(w, ora, got, lse, q, k, v, None, None, w.softmax_scale, seqs=[0, 2, 3])
        kk, vv = cached_kv(ora, 1, 300)
        without = np.r_[0:128, 192:300]
        o, _, tol, _ = tree_attention(kk[:, without], vv[:, without], q[1], k[1], v[1],
                                      tree_masks(np.arange(-1, 3)), 4, w.softmax_scale)
        assert (np.abs(got[1] - o) <= tol).all()


def test_long_sequence():
    """A sequence cut among every SM, beside short ones."""
    w = synth.custom_workload("long", [20000, 0, 129, 5003], 8, 2, seed=2, schedule="one")
    cache, ora = make_pair(w)
    replay(w, cache, ora)
    q, k, v = inputs(w, 6, 2)
    mask = random_masks(np.random.default_rng(1), 4, 6, "tree")
    got, lse = run(cache, q, k, v, mask, None, w.softmax_scale)
    check(w, ora, got, lse, q, k, v, mask, None, w.softmax_scale)


def test_pool_beyond_32_bit_offsets():
    """Blocks at byte offsets above 2^32 of the cold pool."""
    import torch
    from int8_paged_kv_hybrid_b200 import HybridKVCache
    hkv, phys = 8, 40000                                           # 128 KB per block: 5.2 GB
    w = synth.custom_workload("far", [700, 90], 32, hkv, seed=3)
    _, ora = make_pair(w, gpu=False)
    bt = np.where(w.block_table >= 0, phys - 1 - w.block_table, -1).astype(np.int32)
    cache = HybridKVCache(w.batch, hkv, 32, phys, w.max_blocks, block_table=bt)
    replay(w, cache, ora)
    q, k, v = inputs(w, 5, 2)
    got, lse = run(cache, q, k, v, None, None, w.softmax_scale)
    check(w, ora, got, lse, q, k, v, None, None, w.softmax_scale)
    del cache
    torch.cuda.empty_cache()


def test_workspace_contents_do_not_matter_and_results_repeat():
    w = synth.custom_workload("ws", [900, 40, 2100], 32, 8, seed=3)
    cache, ora = make_pair(w)
    replay(w, cache, ora)
    q, k, v = inputs(w, 12, 2)
    ws = cache.tree_workspace(12)
    ws.fill_(255)
    a = run(cache, q, k, v, None, None, w.softmax_scale, workspace=ws)
    b = run(cache, q, k, v, None, None, w.softmax_scale, workspace=ws)
    check(w, ora, *a, q, k, v, None, None, w.softmax_scale)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_graph_replayed_after_growth_and_two_streams():
    """A captured call, replayed after the cache grew; then two calls at once on
    two streams, each with its workspace."""
    import torch
    w = synth.custom_workload("graph", [200, 1000, 33], 8, 2, seed=3, schedule="chunk", pool_extra=0)
    cache, ora = make_pair(w)
    replay(w, cache, ora, steps=3)
    q, k, v = inputs(w, 6, 2)
    qt, kt, vt = (torch.from_numpy(x).cuda() for x in (q, k, v))
    out = torch.zeros_like(qt)
    lse = torch.zeros(q.shape[:3], device="cuda")
    ws = [cache.tree_workspace(6) for _ in range(2)]
    cache.tree_decode(qt, kt, vt, None, w.softmax_scale, out=out, lse=lse, workspace=ws[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.tree_decode(qt, kt, vt, None, w.softmax_scale, out=out, lse=lse, workspace=ws[0])
    for si in range(3, len(w.schedule)):
        kk, vv = synth.step_tokens(w, si, w.schedule[si])
        ora.append(w.schedule[si], kk, vv)
        cache.append(*(torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (w.schedule[si], kk, vv)))
    g.replay()
    torch.cuda.synchronize()
    both = lambda o, l: (o.float().cpu().numpy().astype(np.float64), l.cpu().numpy().astype(np.float64))  # noqa: E731
    check(w, ora, *both(out, lse), q, k, v, None, None, w.softmax_scale)
    outs = [torch.zeros_like(qt) for _ in range(2)]
    lses = [torch.zeros_like(lse) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i, s in enumerate(streams):
            cache.tree_decode(qt, kt, vt, None, w.softmax_scale, out=outs[i], lse=lses[i], workspace=ws[i], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], out) and torch.equal(lses[i], lse)


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    """The kernel's bounded waits cut to a few cycles: the call ends, the status
    says so, the cache is untouched, and a call with the default limit is right."""
    w = synth.custom_workload("limit", [3000, 1200, 0, 700], 32, 8, seed=17, schedule="chunk")
    cache, ora = make_pair(w)
    replay(w, cache, ora)
    for nodes in (8, 64):                      # one and two tiles of 128 rows per CTA
        q, k, v = inputs(w, nodes, 2)
        ws = cache.tree_workspace(nodes)
        try:
            _lib.hyb_set_wait_limit(4)
            run(cache, q, k, v, None, None, w.softmax_scale, workspace=ws)
        finally:
            _lib.hyb_set_wait_limit(0)
        assert cache.status(clear=True) == _lib.HYB_STATUS_TIMEOUT
        got, lse = run(cache, q, k, v, None, None, w.softmax_scale, workspace=ws)
        check(w, ora, got, lse, q, k, v, None, None, w.softmax_scale)
        assert cache.status() == 0


@pytest.mark.parametrize("batch,nodes", [(700, 3), (1500, 1)])
def test_more_sequences_than_threads(batch, nodes):
    """Short sequences, many of them without a node: units of one tile, several
    sequences per thread in the search for a CTA's first tile."""
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 70, size=batch)
    lens[::97] = 300
    w = synth.custom_workload("many", [int(n) for n in lens], 4, 2, seed=5, schedule="one")
    cache, ora = make_pair(w)
    replay(w, cache, ora)
    q, k, v = inputs(w, nodes, 3)
    n_tree = rng.integers(0, nodes + 1, size=batch).astype(np.int32)
    n_tree[100:400] = 0
    n_tree[-1] = 0
    got, lse = run(cache, q, k, v, None, n_tree, w.softmax_scale)
    check(w, ora, got, lse, q, k, v, None, n_tree, w.softmax_scale)
    assert cache.status() == 0


def test_no_node_anywhere():
    """n_tree 0 for every sequence: nothing is written."""
    w = synth.custom_workload("none", [40, 200], 8, 2, seed=5)
    cache, ora = make_pair(w)
    replay(w, cache, ora)
    q, k, v = inputs(w, 4, 3)
    got, lse = run(cache, q, k, v, None, np.zeros(2, np.int32), w.softmax_scale)
    assert (got == MARK).all() and (lse == MARK).all() and cache.status() == 0


@pytest.mark.parametrize("bits,hot,block", [(8, 32, 64), (4, 16, 32), (0, 128, 128)])
def test_two_row_tiles_with_short_trees(bits, hot, block):
    """Room for 64 nodes of eight heads each (four tiles of 128 rows), trees of
    one to some nodes: rows and whole row tiles without a query."""
    w = synth.custom_workload("short", [0, 31, 500, 1030, 129, 77], 16, 2, seed=11, hot=hot, block=block, max_step=64)
    cache, ora = make_pair(w, quant_bits=bits)
    replay(w, cache, ora)
    q, k, v = inputs(w, 64, 3)
    mask = random_masks(np.random.default_rng(4), w.batch, 64, "any")
    n_tree = np.array([1, 16, 17, 33, 64, 0], np.int32)
    got, lse = run(cache, q, k, v, mask, n_tree, w.softmax_scale)
    check(w, ora, got, lse, q, k, v, mask, n_tree, w.softmax_scale)
    assert cache.status() == 0


@pytest.mark.parametrize("bits,sizes", [
    (8, [0.0, 0.0, 1e-4, 1e-4, 1e-4, 1e-4]), (4, [0.0, 0.0, 3e-5, 3e-5, 3e-5, 3e-5]),
    (8, [1e-4, 1e-4, 0.0, 0.0, 300.0, 300.0]), (8, [0.0, 0.0, 0.0, 0.0, 0.0, 0.0])])
@pytest.mark.parametrize("nodes", [7, 64])        # one and two tiles of 128 rows per CTA
def test_values_of_zero_or_far_apart_within_a_run(bits, sizes, nodes):
    """Enough units that a CTA's run holds several whole ones: their tiles (of two
    blocks each, the ring and the nodes last) have V of size `sizes`, zero first."""
    import torch
    rng = np.random.default_rng([nodes, bits])
    lens = rng.integers(32 + 64 * 5, 32 + 64 * 6, size=90)
    w = synth.custom_workload("zeros", [int(n) for n in lens], 16, 4, seed=6, schedule="chunk", chunk=64)
    cache, ora = make_pair(w, quant_bits=bits)
    for si, n in enumerate(w.schedule):
        k, v = synth.step_tokens(w, si, n)
        v = (v.astype(np.float32) * sizes[min(si, 5)]).astype(np.float16)
        ora.append(n, k, v)
        cache.append(torch.from_numpy(n).cuda(), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
    q, kt, vt = inputs(w, nodes, 3)
    vt = (vt.astype(np.float32) * sizes[5]).astype(np.float16)
    n_tree = np.full(w.batch, nodes, np.int32)
    if nodes > 7:                                  # (trees of 3, but for one: the reference's time)
        n_tree[1:] = 3
    got, lse = run(cache, q, kt, vt, None, n_tree, w.softmax_scale)
    check(w, ora, got, lse, q, kt, vt, None, n_tree, w.softmax_scale, seqs=[0, 1, 2, 3, 30, 47, 60, 88, 89])
    assert cache.status() == 0


def growing(bits, lens):
    """A cache whose keys grow along the sequence, so that a query of positive
    values raises its maximum with every tile."""
    import torch
    w = synth.custom_workload("rows", lens, 16, 4, seed=5, schedule="one")
    cache, _ = make_pair(w, quant_bits=bits)
    k, v = synth.step_tokens(w, 0, w.schedule[0])
    k = (np.abs(k.astype(np.float32)) * np.linspace(0.05, 4.0, k.shape[1])[None, :, None, None]).astype(np.float16)
    cache.append(*(torch.from_numpy(x).cuda() for x in (w.schedule[0], k, v)))
    return w, cache


@pytest.mark.parametrize("bits", [8, 0])
@pytest.mark.parametrize("nodes", [8, 64])        # one and two tiles of 128 rows per CTA
def test_a_row_does_not_depend_on_its_neighbours(bits, nodes):
    """Nodes 1.. with other queries leave node 0's bits alone: their maxima grow
    tile by tile, or not at all."""
    w, cache = growing(bits, [700 + 3 * i for i in range(40)])
    q, kt, vt = inputs(w, nodes, 3)
    mask = np.zeros((w.batch, nodes), np.int64)
    out = []
    for others in (0.0, 3.0):
        q[:, 1:] = np.abs(q[:, 1:]) * 0 + others
        out.append(run(cache, q, kt, vt, mask, None, w.softmax_scale))
    assert np.array_equal(out[0][0][:, 0], out[1][0][:, 0]) and np.array_equal(out[0][1][:, 0], out[1][1][:, 0])
    assert cache.status() == 0


@pytest.mark.parametrize("bits", [8, 0])
@pytest.mark.parametrize("nodes", [8, 64])
def test_results_repeat_whatever_ran_before(bits, nodes):
    """A call whose trees leave rows of the tiles empty, after calls that left
    other queries in shared memory."""
    w, cache = growing(bits, [700 + 3 * i for i in range(40)])
    q, kt, vt = inputs(w, nodes, 3)
    few = np.full(w.batch, 1, np.int32)
    out = []
    for before in (0.0, 3.0, -3.0):
        run(cache, np.full_like(q, before), kt, vt, None, None, w.softmax_scale)
        out.append(run(cache, q, kt, vt, None, few, w.softmax_scale))
    for o in out[1:]:
        assert np.array_equal(o[0], out[0][0]) and np.array_equal(o[1], out[0][1])
    assert cache.status() == 0


def test_a_single_node_over_fp16_cold_blocks_is_a_decode_step():
    """FP16 cold blocks hold the tokens as they came: a cache of L tokens that is
    decoded, and one of L - 1 tokens under a tree of the last one, attend the same
    values.  The decode call has its accuracy bar, the tree its bound."""
    import torch
    from harness import MAX_ABS
    w = synth.custom_workload("last", [33, 65, 90, 129, 500, 1201], 8, 2, seed=4, schedule="one")
    k, v = synth.step_tokens(w, 0, w.schedule[0])
    n = w.schedule[0]
    whole, _ = make_pair(w, quant_bits=0)
    whole.append(*(torch.from_numpy(x).cuda() for x in (n, k, v)))
    cache, ora = make_pair(w, quant_bits=0)
    cache.append(*(torch.from_numpy(x).cuda() for x in (n - 1, k, v)))
    ora.append(n - 1, k, v)
    q, _, _ = inputs(w, 1, 1)
    last = np.arange(w.batch), n - 1
    kt, vt = np.ascontiguousarray(k[last][:, None]), np.ascontiguousarray(v[last][:, None])
    got, lse = run(cache, q, kt, vt, None, None, w.softmax_scale)
    check(w, ora, got, lse, q, kt, vt, None, None, w.softmax_scale)
    step = whole.decode(torch.from_numpy(q[:, 0]).cuda(), w.softmax_scale, int(n.max())).float().cpu().numpy()
    for b in range(w.batch):
        kk, vv = cached_kv(ora, b, int(n[b]) - 1)
        _, _, tol, _ = tree_attention(kk, vv, q[b], kt[b], vt[b], np.ones(1, np.int64), 1, w.softmax_scale)
        assert (np.abs(got[b, 0] - step[b]) <= tol[0] + MAX_ABS).all(), b


@pytest.mark.parametrize("nodes", [5, 64])
def test_the_output_may_be_the_queries(nodes):
    """In place: whole units, shared ones and values that are not finite."""
    import torch
    w = synth.custom_workload("place", [0, 40, 700, 3000], 16, 4, seed=4)
    cache, ora = make_pair(w)
    replay(w, cache, ora)
    q, k, v = inputs(w, nodes, 2)
    v[1, 1, 0, 7] = np.inf
    q, k, v = (torch.from_numpy(x).cuda() for x in (q, k, v))
    want = cache.tree_decode(q, k, v, None, w.softmax_scale)
    assert cache.tree_decode(q, k, v, None, w.softmax_scale, out=q) is q
    assert torch.equal(q, want) and bool(torch.isinf(want).any())
