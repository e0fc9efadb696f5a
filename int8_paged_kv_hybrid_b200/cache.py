"""HybridKVCache: device buffers of one hybrid_v2 cache plus its descriptor.

PyTorch only allocates the buffers and supplies the stream; appends and
attention go through the C ABI (libhybkv.so).  Layouts are those of
include/hyb_kv.h.
"""
from __future__ import annotations

import contextlib
import math

from . import _lib

HOT, BLOCK, HEAD_DIM = 32, 64, 128
TILE_BYTES = BLOCK * HEAD_DIM


def indexed_device(device):
    """torch.device with its index (the current device's where none is given)."""
    import torch
    dev = torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    return dev


class HybridKVCache:
    def __init__(self, batch, num_kv_heads, num_q_heads, num_phys_blocks, max_blocks_per_seq,
                 quant_bits=8, block_table=None, n_int4=None, device="cuda", hot_tokens=HOT,
                 block_size=BLOCK):
        import torch
        self.batch, self.hkv, self.hq = int(batch), int(num_kv_heads), int(num_q_heads)
        self.num_phys, self.max_blocks = int(num_phys_blocks), int(max_blocks_per_seq)
        self.quant_bits = int(quant_bits)
        self.hot_tokens = int(hot_tokens)
        self.block_size = int(block_size)
        dev = indexed_device(device)
        self.device = dev
        self.hot = torch.zeros((self.batch, self.hkv, self.hot_tokens, 2, HEAD_DIM), dtype=torch.float16,
                               device=dev)
        # 8 KB parts per block and kv head: K and V tiles of each 64-token
        # sub-block (a 32-token block uses half of one); FP16 blocks
        # (quant_bits 0) hold 512-byte rows of K then V
        parts = self.block_size // 16 if self.quant_bits == 0 else 2 * max(1, self.block_size // BLOCK)
        self.cold = torch.zeros((self.num_phys, self.hkv, parts, TILE_BYTES), dtype=torch.uint8, device=dev)
        self.scales = torch.zeros((self.num_phys, self.hkv, 2), dtype=torch.float32, device=dev)
        if block_table is None:
            self.block_table = torch.full((self.batch, self.max_blocks), -1, dtype=torch.int32, device=dev)
        else:
            self.block_table = torch.as_tensor(block_table, dtype=torch.int32).to(dev).contiguous()
            assert tuple(self.block_table.shape) == (self.batch, self.max_blocks)
        self.seq_lens = torch.zeros(self.batch, dtype=torch.int32, device=dev)
        self.n_int4 = None
        if n_int4 is not None:
            self.n_int4 = torch.as_tensor(n_int4, dtype=torch.int32).to(dev).contiguous()
        self.status_word = torch.zeros(1, dtype=torch.int32, device=dev)
        self.desc = self._make_desc()
        rc = _lib.hyb_check_desc(self.desc)
        if rc != _lib.HYB_OK:
            raise _lib.HybError(rc, "hyb_check_desc")

    def _make_desc(self):
        d = _lib.CacheDesc()
        d.hot_tokens, d.block_size, d.head_dim = self.hot_tokens, self.block_size, HEAD_DIM
        d.quant_bits = self.quant_bits
        d.num_kv_heads, d.num_q_heads = self.hkv, self.hq
        d.num_phys_blocks, d.max_blocks_per_seq, d.batch = self.num_phys, self.max_blocks, self.batch
        d.reserved = 0
        d.hot = self.hot.data_ptr()
        d.cold = self.cold.data_ptr()
        d.scales = self.scales.data_ptr()
        d.block_table = self.block_table.data_ptr()
        d.seq_lens = self.seq_lens.data_ptr()
        d.n_int4_blocks = None if self.n_int4 is None else self.n_int4.data_ptr()
        d.status = self.status_word.data_ptr()
        return d

    def use_table(self, block_table):
        """Go on with another block table, from the next call on: int32
        [batch][max_blocks_per_seq], contiguous, on the cache's device; it is kept,
        not copied.  This is how the table of a pool's successor gets here.  A
        captured call stays with the table that it was captured with."""
        import torch
        _lib.need(block_table.shape == self.block_table.shape and block_table.dtype == torch.int32 and
                  block_table.device == self.device and block_table.is_contiguous(), "use_table")
        self.block_table = block_table
        self.desc.block_table = block_table.data_ptr()

    def _here(self):
        """The cache's device as the current one: sizes and plans go by its SM count."""
        import torch
        return torch.cuda.device(self.device) if self.device.type == "cuda" else contextlib.nullcontext()

    def _attend(self, call, out, make_out, workspace, make_workspace, stream):
        """call(workspace, out, stream) -> out; buffers not given are made on the stream."""
        made = []

        def run(s):
            ws = make_workspace() if workspace is None else workspace
            o = out
            if o is None:
                o = make_out()
                made.append(o)
            call(ws, o, s)
            return o
        return _lib.on_device(self.device, stream, run, made if out is None or workspace is None else None)

    def _empty_out(self):
        import torch
        return torch.empty((self.batch, self.hq, HEAD_DIM), dtype=torch.float16, device=self.device)

    # ---- the three calls ----
    def append(self, n_new, k_new, v_new, stream=None):
        """n_new: int32 CUDA [batch]; k_new, v_new: FP16 CUDA [batch][max_new][Hkv][128]."""
        assert k_new.is_contiguous() and v_new.is_contiguous() and n_new.is_contiguous()
        _lib.on_device(self.device, stream, lambda s: _lib.hyb_kv_append(self.desc, n_new, k_new.shape[1], k_new,
                                                                         v_new, s))

    def migrate(self, target_n_int4, max_delta=None, stream=None):
        """Move every sequence's INT4 block count to target_n_int4 (int32
        [batch], host or CUDA), re-quantizing the blocks in between in place
        (hyb_kv_migrate).  max_delta: bound on the move (default: the table width)."""
        import torch
        made = []

        def call(s):
            if self.n_int4 is None:
                self.n_int4 = torch.zeros(self.batch, dtype=torch.int32, device=self.device)
                made.append(self.n_int4)
                self.desc = self._make_desc()
            tgt = torch.as_tensor(target_n_int4, dtype=torch.int32).to(self.device).contiguous()
            _lib.hyb_kv_migrate(self.desc, tgt, self.max_blocks if max_delta is None else int(max_delta), s)
        _lib.on_device(self.device, stream, call, made)

    def plan(self, max_seq_len, split_tokens=0):
        with self._here():
            return _lib.hyb_decode_plan(self.desc, max_seq_len, split_tokens)

    def launch_info(self, max_seq_len, split_tokens=0):
        """(kernel, CTAs, CTAs per SM) of the decode launch for these arguments."""
        with self._here():
            return _lib.hyb_decode_launch_info(self.desc, max_seq_len, split_tokens)

    def workspace(self, max_seq_len, split_tokens=0):
        import torch
        with self._here():
            n = _lib.hyb_decode_workspace_bytes(self.desc, max_seq_len, split_tokens)
        return None if n == 0 else torch.zeros(n, dtype=torch.uint8, device=self.device)

    def decode(self, q, softmax_scale, max_seq_len, split_tokens=0, out=None, lse=None,
               workspace=None, stream=None):
        """q: FP16 CUDA [batch][Hq][128] -> out FP16 [batch][Hq][128] (and lse FP32 [batch][Hq])."""
        assert q.is_contiguous()
        return self._attend(lambda ws, o, s: _lib.hyb_decode_attn(self.desc, q, softmax_scale, max_seq_len,
                                                                  split_tokens, ws, o, lse, s),
                            out, self._empty_out, workspace, lambda: self.workspace(max_seq_len, split_tokens), stream)

    def sparse_workspace(self, max_seq_len, split_tokens=0):
        import torch
        with self._here():
            n = _lib.hyb_decode_sparse_workspace_bytes(self.desc, max_seq_len, split_tokens)
        return torch.zeros(max(n, 16), dtype=torch.uint8, device=self.device)

    def decode_sparse(self, q, softmax_scale, max_seq_len, top_k, split_tokens=0, out=None, lse=None,
                      workspace=None, stream=None):
        """As decode, but each query head attends only the top_k of the tokens
        in its sequence's INT4 (L2) blocks (hyb_decode_attn_sparse)."""
        assert q.is_contiguous()
        return self._attend(lambda ws, o, s: _lib.hyb_decode_attn_sparse(self.desc, q, softmax_scale, max_seq_len,
                                                                         split_tokens, top_k, ws, o, lse, s),
                            out, self._empty_out, workspace,
                            lambda: self.sparse_workspace(max_seq_len, split_tokens), stream)

    def sparse_selection(self, workspace, max_seq_len, split_tokens=0):
        """The selected L2 positions the last decode_sparse call with this
        workspace left: int32 CUDA view [batch][Hq][stride] (row (b, h): the
        first min(top_k, L2 tokens of b) entries, ascending)."""
        import torch
        with self._here():
            off, stride = _lib.hyb_decode_sparse_selection(self.desc, max_seq_len, split_tokens)
        n = self.batch * self.hq * stride * 4
        return workspace[off:off + n].view(torch.int32).view(self.batch, self.hq, stride)

    def step_workspace(self, max_seq_len, split_tokens=0):
        import torch
        with self._here():
            n = _lib.hyb_decode_step_workspace_bytes(self.desc, max_seq_len, split_tokens)
        return torch.zeros(max(n, 16), dtype=torch.uint8, device=self.device)

    def step(self, n_new, k_new, v_new, q, softmax_scale, max_seq_len, split_tokens=0, out=None,
             lse=None, workspace=None, stream=None):
        """Fused decode step: append n_new[b] in {0, 1} tokens (k_new, v_new FP16
        [batch][1][Hkv][128]) and attend q; max_seq_len bounds the new lengths."""
        assert q.is_contiguous() and k_new.is_contiguous() and v_new.is_contiguous()
        return self._attend(lambda ws, o, s: _lib.hyb_decode_step(self.desc, n_new, k_new, v_new, q, softmax_scale,
                                                                  max_seq_len, split_tokens, ws, o, lse, s),
                            out, self._empty_out, workspace, lambda: self.step_workspace(max_seq_len, split_tokens),
                            stream)

    def tree_workspace(self, max_tree):
        """Workspace of tree_decode for trees of up to max_tree nodes (any lengths)."""
        import torch
        with self._here():
            n = _lib.hyb_tree_workspace_bytes(self.desc, max_tree)
        _lib.need(n > 0, "tree_workspace: max_tree %r" % (max_tree,))
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def tree_decode(self, q, k_tree, v_tree, tree_mask, softmax_scale, n_tree=None, out=None, lse=None,
                    workspace=None, stream=None):
        """Attention of drafted nodes (hyb_tree_attn) on `stream` (default: the
        current one of the cache's device), where buffers not given are made too:
        q FP16 CUDA [batch][nodes][Hq][128], k_tree / v_tree FP16
        [batch][nodes][Hkv][128], tree_mask int64 [batch][nodes] (bit j: the node
        attends node j; see tree_masks) or None for a chain, n_tree int32 [batch] or
        None for all nodes -> out FP16 [batch][nodes][Hq][128], and into `lse` FP32
        [batch][nodes][Hq] where it is given.  Rows at and behind n_tree[b] are left
        as they were (zero in an `out` that this call makes)."""
        import torch
        need, dev, nodes = _lib.need, self.device, q.shape[1] if q.dim() == 4 else 0
        q_shape, kv_shape = (self.batch, nodes, self.hq, HEAD_DIM), (self.batch, nodes, self.hkv, HEAD_DIM)
        for name, x, shape in (("q", q, q_shape), ("k_tree", k_tree, kv_shape), ("v_tree", v_tree, kv_shape)):
            need(x.shape == shape and x.dtype == torch.float16 and x.device == dev and x.is_contiguous(),
                 "tree_decode: " + name)
        for name, x, shape, dtype in (("out", out, q_shape, torch.float16),
                                      ("tree_mask", tree_mask, (self.batch, nodes), torch.int64),
                                      ("n_tree", n_tree, (self.batch,), torch.int32),
                                      ("lse", lse, (self.batch, nodes, self.hq), torch.float32)):
            need(x is None or (x.shape == shape and x.dtype == dtype and x.device == dev and x.is_contiguous()),
                 "tree_decode: " + name)
        need(workspace is None or (workspace.device == dev and workspace.is_contiguous()), "tree_decode: workspace")
        return self._attend(lambda ws, o, s: _lib.hyb_tree_attn(self.desc, q, k_tree, v_tree, tree_mask, n_tree, nodes,
                                                                softmax_scale, ws, o, lse, s),
                            out, lambda: torch.zeros(q_shape, dtype=torch.float16, device=dev),
                            workspace, lambda: self.tree_workspace(nodes), stream)

    def status(self, clear=False, stream=None):
        return _lib.on_device(self.device, stream, lambda s: _lib.hyb_read_status(self.desc, clear, s))


def default_softmax_scale(head_dim=HEAD_DIM):
    return 1.0 / math.sqrt(head_dim)
