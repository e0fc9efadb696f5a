"""BlockPool: free blocks and block tables of a batch, and tree masks.

As in cache.py, PyTorch only allocates the buffers and supplies the stream;
tables and slot maps are built by libhybkv.so (include/hyb_spec.h).
"""
from __future__ import annotations

import numpy as np

from . import _lib
from .cache import BLOCK, HOT, indexed_device


def tree_masks(parents):
    """Ancestor masks of a drafted tree: parents[t] < t is the parent node of
    node t, or -1 for a child of the last cached token.  Returns int64 masks of
    the same shape (bit j of mask t: node t is j or descends from it); the last
    axis is the nodes, 1 to 64.  Host only."""
    p = np.asarray(parents)
    _lib.need(p.dtype.kind in "iu" and p.ndim > 0 and 1 <= p.shape[-1] <= _lib.HYB_MAX_TREE, "tree_masks")
    p, nodes = p.astype(np.int64), p.shape[-1]
    _lib.need(((p >= -1) & (p < np.arange(nodes))).all(), "tree_masks")
    flat = p.reshape(-1, nodes)
    mask = np.zeros(flat.shape, np.uint64)
    rows = np.arange(flat.shape[0])
    for t in range(nodes):
        up = flat[:, t]
        mask[:, t] = np.where(up >= 0, mask[rows, np.maximum(up, 0)], np.uint64(0)) | (np.uint64(1) << np.uint64(t))
    return mask.view(np.int64).reshape(p.shape)


class BlockPool:
    """The physical blocks of a cache: the free ones as a ring, the others held
    by the sequences of a batch (hyb_pool_desc).  A new pool has every block
    free.  Existing buffers may be given: ring int32 [num_phys_blocks], state
    int32 [2] (head, count), n_blocks int32 [batch], block_table int32
    [batch][max_blocks_per_seq].  `block_table` is what HybridKVCache takes
    (a successor's: HybridKVCache.use_table).
    A call works on `stream` (default: the current one of the pool's device),
    where the buffers that it is not given are made too."""

    def __init__(self, batch, num_phys_blocks, max_blocks_per_seq, hot_tokens=HOT, block_size=BLOCK, device="cuda",
                 ring=None, state=None, n_blocks=None, block_table=None, status_word=None):
        import torch
        self.batch, self.num_phys, self.max_blocks = int(batch), int(num_phys_blocks), int(max_blocks_per_seq)
        self.hot_tokens, self.block_size = int(hot_tokens), int(block_size)
        self.device = dev = indexed_device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.ring = torch.arange(self.num_phys, **i32) if ring is None else ring
        self.state = torch.tensor([0, self.num_phys], **i32) if state is None else state
        self.n_blocks = torch.zeros(self.batch, **i32) if n_blocks is None else n_blocks
        self.block_table = torch.full((self.batch, self.max_blocks), -1, **i32) if block_table is None else block_table
        self.status_word = torch.zeros(1, **i32) if status_word is None else status_word
        for name, x, shape in (("ring", self.ring, (self.num_phys,)), ("state", self.state, (2,)),
                               ("n_blocks", self.n_blocks, (self.batch,)), ("status_word", self.status_word, (1,)),
                               ("block_table", self.block_table, (self.batch, self.max_blocks))):
            self._check(x, shape, "BlockPool: " + name)
        d = self.desc = _lib.PoolDesc()
        d.batch, d.max_blocks_per_seq, d.num_phys_blocks = self.batch, self.max_blocks, self.num_phys
        d.hot_tokens, d.block_size, d.reserved = self.hot_tokens, self.block_size, 0
        d.ring, d.state, d.n_blocks = self.ring.data_ptr(), self.state.data_ptr(), self.n_blocks.data_ptr()
        d.block_table, d.status = self.block_table.data_ptr(), self.status_word.data_ptr()
        rc = _lib.hyb_check_pool(d)
        if rc != _lib.HYB_OK:
            raise _lib.HybError(rc, "hyb_check_pool")

    def _check(self, x, shape, what, dtype=None):
        import torch
        _lib.need(x.shape == shape and x.dtype == (dtype or torch.int32) and x.device == self.device and
                  x.is_contiguous(), what)

    def successor(self):
        """A pool of the same blocks with state, counts and table of its own
        (not yet filled in), for resize(..., to=)."""
        import torch
        return BlockPool(self.batch, self.num_phys, self.max_blocks, self.hot_tokens, self.block_size, self.device,
                         self.ring, torch.empty_like(self.state), torch.empty_like(self.n_blocks),
                         torch.empty_like(self.block_table), self.status_word)

    def workspace(self):
        import torch
        return torch.zeros(_lib.hyb_pool_workspace_bytes(self.desc), dtype=torch.uint8, device=self.device)

    def resize(self, lens, to=None, workspace=None, stream=None):
        """Give each sequence the blocks that lens[b] tokens need (hyb_pool_resize):
        lens int32 CUDA [batch]; in place, or into the successor `to`."""
        self._check(lens, (self.batch,), "BlockPool.resize: lens")
        _lib.need(to is None or to.device == self.device, "BlockPool.resize: to")
        _lib.need(workspace is None or (workspace.device == self.device and workspace.is_contiguous()),
                  "BlockPool.resize: workspace")
        _lib.on_device(self.device, stream, lambda s: _lib.hyb_pool_resize(
            self.desc, None if to is None else to.desc, lens, self.workspace() if workspace is None else workspace, s),
            [] if workspace is None else None)
        return self if to is None else to

    def slot_map(self, lens, n_tok, max_total, first=None, cu=None, slots=None, stream=None):
        """Slots of the packed tokens first[b] .. first[b] + n_tok[b] - 1 of each
        sequence of lens[b] tokens (hyb_slot_map): int64 [max_total], and the
        offsets cu int32 [batch + 1].  Returns (cu, slots); entries of `slots`
        behind cu[batch] are left as they were (HYB_SLOT_NONE in one that this
        call makes)."""
        import torch
        total = int(max_total)
        for name, x in (("lens", lens), ("n_tok", n_tok), ("first", first)):
            if x is not None or name != "first":
                self._check(x, (self.batch,), "BlockPool.slot_map: " + name)
        if cu is not None:
            self._check(cu, (self.batch + 1,), "BlockPool.slot_map: cu")
        if slots is not None:
            self._check(slots, (total,), "BlockPool.slot_map: slots", torch.int64)
        made = []

        def call(s):
            c, o = cu, slots
            if c is None:
                c = torch.empty(self.batch + 1, dtype=torch.int32, device=self.device)
                made.append(c)
            if o is None:
                o = torch.full((total,), _lib.HYB_SLOT_NONE, dtype=torch.int64, device=self.device)
                made.append(o)
            _lib.hyb_slot_map(self.desc, lens, first, n_tok, total, c, o, s)
            return c, o
        return _lib.on_device(self.device, stream, call, made if cu is None or slots is None else None)

    def status(self, clear=False, stream=None):
        """The sticky device status word (0 = ok); waits for the stream."""
        d = _lib.CacheDesc()
        d.status = self.status_word.data_ptr()
        return _lib.on_device(self.device, stream, lambda s: _lib.hyb_read_status(d, clear, s))
