"""Host side of the speculative-decoding calls (no GPU): argument checks of
hyb_tree_attn, hyb_pool_resize and hyb_slot_map, the binding's checks of shapes
and devices, tree masks, and the references the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import int8_paged_kv_hybrid_b200 as hk
from int8_paged_kv_hybrid_b200 import _lib
from test_abi import _desc
from tree_ref import PoolModel, random_masks, slot_map

BAD, UNS, WS = _lib.HYB_ERR_INVALID_VALUE, _lib.HYB_ERR_UNSUPPORTED, _lib.HYB_ERR_WORKSPACE
BASE = 0x7e0000000000


def _tree(d, nodes=8, ws_bytes=None, **change):
    lib = hk.load()
    a = dict(q=BASE, k=BASE + 0x1000000, v=BASE + 0x2000000, mask=BASE + 0x3000000, n=BASE + 0x3100000, scale=0.1,
             ws=BASE + 0x4000000, out=BASE + 0x5000000, lse=BASE + 0x6000000)
    a.update(change)
    need = lib.hyb_tree_workspace_bytes(ctypes.byref(d), nodes)
    return lib.hyb_tree_attn(ctypes.byref(d), a["q"], a["k"], a["v"], a["mask"], a["n"], nodes, a["scale"], a["ws"],
                             need if ws_bytes is None else ws_bytes, a["out"], a["lse"], None)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(out=None), BAD),
    (dict(q=BASE + 8), BAD), (dict(k=BASE + 8), BAD), (dict(v=BASE + 8), BAD), (dict(out=BASE + 8), BAD),
    (dict(lse=BASE + 2), BAD), (dict(mask=BASE + 4), BAD), (dict(n=BASE + 2), BAD),
    (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD),
    (dict(nodes=0), BAD), (dict(nodes=-1), BAD), (dict(nodes=65), UNS),
    (dict(ws=None), WS), (dict(ws=BASE + 8), WS), (dict(ws_bytes=0), WS),
])
def test_tree_refusals(change, want):
    assert _tree(_desc(), **change) == want


def test_tree_refuses_bad_descriptors():
    assert _tree(_desc(hot=33)) == BAD
    assert _tree(_desc(hq=72)) == UNS
    assert hk.load().hyb_tree_workspace_bytes(ctypes.byref(_desc(hot=33)), 4) == 0
    assert hk.hyb_tree_workspace_bytes(_desc(), 65) == 0 and hk.hyb_tree_workspace_bytes(_desc(), 0) == 0
    assert hk.hyb_tree_workspace_bytes(_desc(), 64) > 0


def _pool(batch=4, width=8, phys=32, hot=32, block=64, base=BASE):
    p = _lib.PoolDesc()
    p.batch, p.max_blocks_per_seq, p.num_phys_blocks, p.hot_tokens, p.block_size, p.reserved = \
        batch, width, phys, hot, block, 0
    p.ring, p.state, p.n_blocks = base, base + 0x10000, base + 0x20000
    p.block_table, p.status = base + 0x30000, base + 0x40000
    return p


@pytest.mark.parametrize("field,val,want", [
    ("batch", 0, BAD), ("max_blocks_per_seq", 0, BAD), ("num_phys_blocks", 0, BAD), ("hot_tokens", 33, BAD),
    ("block_size", 12, BAD), ("block_size", 96, UNS), ("reserved", 1, BAD), ("ring", None, BAD),
    ("state", None, BAD), ("n_blocks", None, BAD), ("block_table", None, BAD), ("status", None, BAD),
    ("block_table", BASE + 2, BAD), ("state", BASE + 0x10002, BAD),
])
def test_pool_refusals(field, val, want):
    p = _pool()
    assert hk.hyb_check_pool(p) == 0 and hk.hyb_pool_workspace_bytes(p) > 0
    setattr(p, field, val)
    assert hk.hyb_check_pool(p) == want and hk.hyb_pool_workspace_bytes(p) == 0
    lib, lens = hk.load(), ctypes.c_void_p(BASE + 0x50000)
    ws = ctypes.c_void_p(BASE + 0x60000)
    assert lib.hyb_pool_resize(ctypes.byref(p), None, lens, ws, 4096, None) == want


def test_pool_resize_refuses_overlaps_and_other_geometry():
    lib, lens, ws = hk.load(), ctypes.c_void_p(BASE + 0x50000), ctypes.c_void_p(BASE + 0x60000)

    def call(to, lens=lens, ws=ws, n=4096):
        return lib.hyb_pool_resize(ctypes.byref(_pool()), None if to is None else ctypes.byref(to), lens, ws, n, None)

    for field, val in (("batch", 3), ("max_blocks_per_seq", 4), ("num_phys_blocks", 31), ("hot_tokens", 16),
                       ("block_size", 32), ("ring", BASE + 0x900000)):
        to = _pool()
        setattr(to, field, val)
        assert call(to) == BAD, field
    for field, val in (("n_blocks", BASE + 0x20004), ("block_table", BASE + 0x30010), ("state", BASE + 0x10004),
                       ("n_blocks", BASE + 0x30000), ("state", BASE + 0x20000), ("n_blocks", BASE),
                       ("block_table", BASE + 0x50000)):
        to = _pool()
        setattr(to, field, val)
        assert call(to) == BAD, (field, hex(val))
    to = _pool(base=BASE + 0x800000)
    to.ring = _pool().ring
    to.n_blocks = to.block_table
    assert call(to) == BAD                        # two outputs in the same memory
    assert call(None, lens=None) == BAD
    assert call(None, lens=ctypes.c_void_p(BASE + 0x50002)) == BAD
    assert call(None, lens=ctypes.c_void_p(BASE + 0x20000)) == BAD    # lens are the counts themselves
    assert call(None, ws=None) == WS and call(None, n=8) == WS


def test_slot_map_refusals():
    lib = hk.load()
    a = [ctypes.c_void_p(BASE + 0x100000 * i) for i in range(1, 6)]

    def call(p=None, lens=a[0], first=a[1], n_tok=a[2], total=8, cu=a[3], slots=a[4]):
        return lib.hyb_slot_map(ctypes.byref(p or _pool()), lens, first, n_tok, total, cu, slots, None)

    odd = ctypes.c_void_p(BASE + 0x100002)
    assert call(lens=None) == BAD and call(n_tok=None) == BAD and call(slots=None) == BAD
    assert call(total=-1) == BAD and call(lens=odd) == BAD and call(first=odd) == BAD and call(cu=odd) == BAD
    assert call(slots=ctypes.c_void_p(BASE + 0x100004)) == BAD
    assert call(p=_pool(block=96)) == UNS and call(p=_pool(hot=8)) == BAD


def test_status_texts():
    for c in (_lib.HYB_STATUS_POOL, _lib.HYB_STATUS_BAD_TREE):
        assert hk.strerror(100 + c) != "unknown code"


def test_tree_masks():
    # 0 -> 1 -> 3, 0 -> 2, 4 a second root
    assert hk.tree_masks([-1, 0, 0, 1, -1]).tolist() == [1, 3, 5, 11, 16]
    chain = hk.tree_masks(np.arange(-1, 63))
    assert chain.dtype == np.int64 and chain[63] == -1 and chain[2] == 7
    both = hk.tree_masks([[-1, 0], [-1, -1]])
    assert both.tolist() == [[1, 3], [1, 2]]
    for bad in ([0], [-1, 1], [-2], [-1, 2, 0], list(range(-1, 64))):
        with pytest.raises(hk.HybError):
            hk.tree_masks(bad)


def test_binding_checks():
    import torch
    p = hk.BlockPool(2, 8, 4, device="cpu")
    assert p.state.tolist() == [0, 8] and p.block_table.tolist() == [[-1] * 4] * 2
    with pytest.raises(hk.HybError):
        p.resize(torch.zeros(2, dtype=torch.int32))                   # no GPU buffers
    with pytest.raises(hk.HybError):
        p.resize(torch.zeros(3, dtype=torch.int32))
    with pytest.raises(hk.HybError):
        p.slot_map(torch.zeros(2), torch.zeros(2, dtype=torch.int32), 4)
    with pytest.raises(hk.HybError):
        hk.BlockPool(2, 8, 4, device="cpu", ring=torch.zeros(8))
    with pytest.raises(hk.HybError):
        hk.BlockPool(2, 8, 4, device="cpu", hot_tokens=20)
    c = object.__new__(hk.HybridKVCache)          # a CPU cache's buffers need not have the alignment
    c.batch, c.hkv, c.hq, c.device, c.desc = 2, 2, 4, torch.device("cpu"), _desc(hkv=2, hq=4)
    h = dict(dtype=torch.float16)
    q, k = torch.zeros((2, 3, 4, 128), **h), torch.zeros((2, 3, 2, 128), **h)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :2]), dict(q=q[0]), dict(k_tree=k[:1]), dict(v_tree=k.transpose(1, 2)),
                dict(tree_mask=torch.zeros((2, 3), dtype=torch.int32)), dict(n_tree=torch.zeros(2)),
                dict(out=torch.zeros((2, 3, 4, 64), **h)), dict(lse=torch.zeros((2, 4)))):
        a = dict(q=q, k_tree=k, v_tree=k, tree_mask=None, softmax_scale=0.1)
        a.update(bad)
        with pytest.raises(hk.HybError):
            c.tree_decode(**a)
    with pytest.raises(hk.HybError):
        c.tree_workspace(65)


def test_references():
    """The sequential models on cases worked by hand."""
    m = PoolModel(3, 6, 4, 32, 64)
    assert m.resize([100, 32, 160]) == [] and m.held == [[0, 1], [], [2, 3]] and m.free == [4, 5]
    # 300 tokens need a fifth column: left unchanged; the blocks given back are free for the next call
    assert m.resize([0, 300, 161]) == [] and m.held == [[], [], [2, 3, 4]] and m.free == [5, 0, 1]
    assert m.resize([288, 33, 161]) == [0, 1] and m.held == [[], [], [2, 3, 4]]   # 4 > 3 free; 4 + 1 > 3
    cu, s = slot_map([[7, 9]], [100], [30], [4], 32, 64)
    assert cu.tolist() == [0, 4] and s.tolist() == [7 * 64 + 30, 7 * 64 + 31, 7 * 64 + 32, 7 * 64 + 33]
    _, s = slot_map([[7, 9]], [100], [66], [4], 32, 64)
    assert s.tolist() == [9 * 64 + 2, 9 * 64 + 3, -2 - 68 % 32, -2 - 69 % 32]
    r = random_masks(np.random.default_rng(0), 2, 5, "any")
    assert (r[:, 0] == 0).all()


def test_buffers_that_a_call_makes_are_made_on_its_stream(monkeypatch):
    """tree_decode, resize and slot_map make and fill their own buffers inside
    on_device, which makes the call's stream the current one."""
    import torch
    pool = hk.BlockPool(2, 8, 4, device="cpu")
    c = object.__new__(hk.HybridKVCache)
    c.batch, c.hkv, c.hq, c.device, c.desc = 2, 2, 4, torch.device("cpu"), _desc(hkv=2, hq=4)
    q, k = torch.zeros((2, 3, 4, 128), dtype=torch.float16), torch.zeros((2, 3, 2, 128), dtype=torch.float16)
    lens = torch.zeros(2, dtype=torch.int32)
    inside, handed = [], []

    def on_device(device, stream, call, made=None):
        assert made is not None, "the call makes buffers"
        inside.append(stream)
        r = call(stream)
        inside.pop()
        handed.append(len(made))
        return r

    def watched(make):
        def f(*a, **kw):
            assert inside, "a buffer made outside the call's stream"
            return make(*a, **kw)
        return f

    monkeypatch.setattr(_lib, "on_device", on_device)
    for name in ("hyb_tree_attn", "hyb_pool_resize", "hyb_slot_map"):
        monkeypatch.setattr(_lib, name, lambda *a: None)
    for name in ("zeros", "empty", "full", "zeros_like", "empty_like", "full_like"):
        monkeypatch.setattr(torch, name, watched(getattr(torch, name)))
    out = c.tree_decode(q, k, k, None, 0.1, stream=5)
    assert out.shape == q.shape and not out.any()
    assert c.tree_decode(q, k, k, None, 0.1, out=q, stream=5) is q
    assert pool.resize(lens, stream=5) is pool
    cu, slots = pool.slot_map(lens, lens, 7, stream=5)
    assert cu.shape == (3,) and slots.tolist() == [-1] * 7
    assert handed == [1, 0, 0, 2]                 # what the caller gets


def test_buffers_of_the_decode_calls_are_made_on_their_stream(monkeypatch):
    """The same of decode, decode_sparse, step and migrate."""
    import torch
    c = object.__new__(hk.HybridKVCache)
    c.batch, c.hkv, c.hq, c.device, c.desc, c.max_blocks = 2, 2, 4, torch.device("cpu"), _desc(hkv=2, hq=4), 16
    c.n_int4, c._make_desc = None, lambda: _desc(hkv=2, hq=4)
    q, k = torch.zeros((2, 4, 128), dtype=torch.float16), torch.zeros((2, 1, 2, 128), dtype=torch.float16)
    n_new, target = torch.ones(2, dtype=torch.int32), torch.ones(2, dtype=torch.int64)
    inside, handed = [], []

    def on_device(device, stream, call, made=None):
        assert made is not None and stream == 5
        inside.append(stream)
        r = call(stream)
        inside.pop()
        handed.append(len(made))
        return r

    def watched(make):
        def f(*a, **kw):
            assert inside, "a buffer made outside the call's stream"
            return make(*a, **kw)
        return f

    monkeypatch.setattr(_lib, "on_device", on_device)
    for name in ("hyb_decode_attn", "hyb_decode_attn_sparse", "hyb_decode_step", "hyb_kv_migrate"):
        monkeypatch.setattr(_lib, name, lambda *a: None)
    for name in ("zeros", "empty", "full", "as_tensor"):
        monkeypatch.setattr(torch, name, watched(getattr(torch, name)))
    assert c.decode(q, 0.1, 64, stream=5).shape == q.shape
    assert c.decode(q, 0.1, 64, out=q, stream=5) is q
    assert c.decode_sparse(q, 0.1, 64, 4, stream=5).shape == q.shape
    assert c.step(n_new, k, k, q, 0.1, 64, stream=5).shape == q.shape
    c.migrate(target, stream=5)
    assert c.n_int4 is not None
    c.migrate(target, stream=5)
    assert handed == [1, 0, 1, 1, 1, 0]


def test_sizes_and_plans_are_asked_on_the_caches_device(monkeypatch):
    """The current device is another one than the cache's."""
    import contextlib

    import torch
    c = object.__new__(hk.HybridKVCache)
    c.batch, c.hkv, c.hq, c.device, c.desc = 2, 2, 4, torch.device("cuda", 1), _desc(hkv=2, hq=4)
    current, asked = [0], []

    @contextlib.contextmanager
    def device(d):
        current.append(d.index)
        yield
        current.pop()

    def size(*a):
        asked.append(current[-1])
        return 64

    monkeypatch.setattr(torch.cuda, "device", device)
    names = ["hyb_tree_workspace_bytes", "hyb_decode_workspace_bytes", "hyb_decode_step_workspace_bytes",
             "hyb_decode_sparse_workspace_bytes", "hyb_decode_plan", "hyb_decode_launch_info"]
    for name in names:
        monkeypatch.setattr(_lib, name, size)
    monkeypatch.setattr(_lib, "hyb_decode_sparse_selection", lambda *a: (0, size()))
    for make in ("empty", "zeros"):
        monkeypatch.setattr(torch, make, lambda n, **kw: kw["device"].index)
    assert c.tree_workspace(4) == 1 and c.workspace(99) == 1 and c.step_workspace(99) == 1 and c.sparse_workspace(99) == 1
    c.plan(99)
    c.launch_info(99)
    c.sparse_selection(torch.arange(4096, dtype=torch.uint8), 99)
    assert asked == [1] * 7 and current == [0]


def test_append_and_status_go_to_the_caches_device(monkeypatch):
    """As the other calls: the stream is one of the cache's device, not of the current one."""
    import torch
    c = object.__new__(hk.HybridKVCache)
    c.device, c.desc = torch.device("cuda", 1), _desc()
    went = []
    monkeypatch.setattr(_lib, "on_device", lambda device, stream, call, made=None: (went.append(device), call(stream))[1])
    monkeypatch.setattr(_lib, "hyb_kv_append", lambda *a: went.append(a[-1]))
    monkeypatch.setattr(_lib, "hyb_read_status", lambda *a: 9)
    x = torch.zeros((1, 2, 3))
    c.append(x, x, x, stream=5)
    assert c.status(stream=6) == 9 and went == [c.device, 5, c.device]


def test_use_table():
    import torch
    c = object.__new__(hk.HybridKVCache)
    c.device, c.desc, c.block_table = torch.device("cpu"), _desc(), torch.zeros((2, 4), dtype=torch.int32)
    t = torch.ones((2, 4), dtype=torch.int32)
    for bad in (t[:1], t.long(), torch.ones((4, 2), dtype=torch.int32).t(), torch.ones((2, 5), dtype=torch.int32)[:, :4]):
        with pytest.raises(hk.HybError):
            c.use_table(bad)
    desc = c.desc
    c.use_table(t)
    assert c.block_table is t and c.desc is desc and desc.block_table == t.data_ptr()


@pytest.mark.parametrize("bad", [[], [[], []], 0, -1, [-1.0, 0.4], [True], ["a"], [None], [-1, 2 ** 70]])
def test_tree_masks_refuses_what_is_no_tree(bad):
    """No nodes, no axis of nodes, and parents that are no whole numbers."""
    with pytest.raises(hk.HybError):
        hk.tree_masks(bad)


def test_tree_masks_of_whole_numbers_of_any_type():
    for t in (np.int8, np.int32, np.int64):
        assert hk.tree_masks(np.array([-1, 0, 0], t)).tolist() == [1, 3, 5]
    assert hk.tree_masks(np.zeros((0, 3), np.int32)).shape == (0, 3)
