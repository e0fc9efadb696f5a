// spec_host.cu -- the C ABI declared in include/hyb_spec.h: argument checks,
// workspace sizes and launches.  No memory is allocated here.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "spec.cuh"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [p, p + n) and [q, q + m) share no byte
bool disjoint(const void *p, size_t n, const void *q, size_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
  return x + n <= y || y + m <= x;
}

int block_shift(int block_size) { return block_size == 32 ? 5 : block_size == 64 ? 6 : 7; }

// sizes and table of a pool descriptor (what hyb_slot_map needs)
int check_geometry(const hyb_pool_desc *p) {
  if (!p) return HYB_ERR_INVALID_VALUE;
  const int h = p->hot_tokens;
  if (!(h == 16 || h == 32 || h == 64 || h == 128)) return HYB_ERR_INVALID_VALUE;
  if (p->block_size <= 0 || p->block_size % 8 != 0 || p->reserved != 0) return HYB_ERR_INVALID_VALUE;
  if (p->batch <= 0 || p->max_blocks_per_seq <= 0 || p->num_phys_blocks <= 0) return HYB_ERR_INVALID_VALUE;
  if (!p->block_table || !p->status || !aligned(p->block_table, 4) || !aligned(p->status, 4))
    return HYB_ERR_INVALID_VALUE;
  if (p->block_size != 32 && p->block_size != 64 && p->block_size != 128) return HYB_ERR_UNSUPPORTED;
  return HYB_OK;
}

}  // namespace

extern "C" {

// Workspace of hyb_tree_attn: the partial outputs, their sums and maxima, and
// the units that CTAs share (TreeArgs).
struct TreeWs {
  size_t o, ml, units, total;
};

static TreeWs tree_ws(const hyb_cache_desc *d, int32_t max_tree, int sms) {
  const int group = d->num_q_heads / d->num_kv_heads;
  const size_t rows = static_cast<size_t>(2) * sms * 128 * hyb::tree_m_tiles(max_tree, group);
  TreeWs w;
  w.o = 0;
  w.ml = w.o + rows * hyb::kDim * sizeof(float);
  w.units = w.ml + rows * 2 * sizeof(float);
  w.total = w.units + static_cast<size_t>(sms) * sizeof(int4);
  return w;
}

size_t hyb_tree_workspace_bytes(const hyb_cache_desc *d, int32_t max_tree) {
  if (hyb_check_desc(d) != HYB_OK || max_tree < 1 || max_tree > HYB_MAX_TREE) return 0;
  return tree_ws(d, max_tree, hyb::host_sm_count()).total;
}

int hyb_tree_attn(const hyb_cache_desc *d, const void *q, const void *k_tree, const void *v_tree,
                  const uint64_t *tree_mask, const int32_t *n_tree, int32_t max_tree, float softmax_scale,
                  void *workspace, size_t workspace_bytes, void *out, float *lse_out, hyb_stream_t stream) {
  const int rc = hyb_check_desc(d);
  if (rc != HYB_OK) return rc;
  if (!q || !k_tree || !v_tree || !out || max_tree < 1 || !aligned(q, 16) || !aligned(k_tree, 16) ||
      !aligned(v_tree, 16) || !aligned(out, 16) || (lse_out && !aligned(lse_out, 4)) ||
      (tree_mask && !aligned(tree_mask, 8)) || (n_tree && !aligned(n_tree, 4)) || !std::isfinite(softmax_scale))
    return HYB_ERR_INVALID_VALUE;
  if (max_tree > HYB_MAX_TREE) return HYB_ERR_UNSUPPORTED;
  const int sms = hyb::host_sm_count();
  const TreeWs w = tree_ws(d, max_tree, sms);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < w.total) return HYB_ERR_WORKSPACE;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  hyb::TreeArgs a;
  const long long wait = hyb::host_wait_cycles();
  a.wait_cycles = wait < 0xf0000000ll ? static_cast<uint32_t>(wait) : 0xf0000000u;
  a.ctas = sms;
  a.group = d->num_q_heads / d->num_kv_heads;
  // two Q buffers where two of 64 rows do
  a.q_bufs = max_tree * a.group <= 64 ? 2 : 1;
  a.q_rows = a.q_bufs == 2 ? 64 : 128;
  a.group_recip = 65536 / a.group + 1;
  a.part_o = reinterpret_cast<float *>(ws + w.o);
  a.part_ml = reinterpret_cast<float *>(ws + w.ml);
  a.shared_units = reinterpret_cast<int4 *>(ws + w.units);
  a.hot = static_cast<const uint8_t *>(d->hot);
  a.cold = static_cast<const uint8_t *>(d->cold);
  a.scales = d->scales;
  a.block_table = d->block_table;
  a.seq_lens = d->seq_lens;
  a.n_int4 = d->quant_bits == 8 ? d->n_int4_blocks : nullptr;
  a.status = d->status;
  a.q = static_cast<const __half *>(q);
  a.k_tree = static_cast<const __half *>(k_tree);
  a.v_tree = static_cast<const __half *>(v_tree);
  a.mask = tree_mask;
  a.n_tree = n_tree;
  a.out = static_cast<__half *>(out);
  a.lse_out = lse_out;
  a.batch = d->batch;
  a.hkv = d->num_kv_heads;
  a.hq = d->num_q_heads;
  a.num_phys = d->num_phys_blocks;
  a.max_blocks = d->max_blocks_per_seq;
  a.quant_bits = d->quant_bits;
  a.hot_tokens = d->hot_tokens;
  a.max_tree = max_tree;
  a.lsub = d->block_size == 2 * hyb::kBlock ? 1 : 0;
  a.bshift = block_shift(d->block_size);
  a.qk_scale = softmax_scale * 1.4426950408889634f;
  const cudaError_t e = hyb::launch_tree_attn(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HYB_OK : hyb::host_cuda_fail(e);
}

int hyb_check_pool(const hyb_pool_desc *p) {
  const int rc = check_geometry(p);
  if (rc == HYB_ERR_INVALID_VALUE) return rc;
  if (!p->ring || !p->state || !p->n_blocks || !aligned(p->ring, 4) || !aligned(p->state, 4) ||
      !aligned(p->n_blocks, 4))
    return HYB_ERR_INVALID_VALUE;
  return rc;
}

size_t hyb_pool_workspace_bytes(const hyb_pool_desc *p) {
  if (hyb_check_pool(p) != HYB_OK) return 0;
  return (static_cast<size_t>(p->batch) + 4) * sizeof(int32_t);
}

int hyb_pool_resize(const hyb_pool_desc *from, const hyb_pool_desc *to, const int32_t *lens, void *workspace,
                    size_t workspace_bytes, hyb_stream_t stream) {
  int rc = hyb_check_pool(from);
  if (rc != HYB_OK) return rc;
  if (!to) to = from;
  rc = hyb_check_pool(to);
  if (rc != HYB_OK) return rc;
  if (to->batch != from->batch || to->max_blocks_per_seq != from->max_blocks_per_seq ||
      to->num_phys_blocks != from->num_phys_blocks || to->hot_tokens != from->hot_tokens ||
      to->block_size != from->block_size || to->ring != from->ring || !lens || !aligned(lens, 4))
    return HYB_ERR_INVALID_VALUE;
  const size_t nb = static_cast<size_t>(from->batch) * sizeof(int32_t);
  const size_t tb = nb * static_cast<size_t>(from->max_blocks_per_seq);
  const size_t rb = static_cast<size_t>(from->num_phys_blocks) * sizeof(int32_t);
  // what is written overlaps nothing that is read, but for the same pointer
  const struct {
    const void *p;
    size_t n;
  } in[] = {{from->state, 8}, {from->n_blocks, nb}, {from->block_table, tb}, {from->ring, rb}, {lens, nb}},
    outs[] = {{to->state, 8}, {to->n_blocks, nb}, {to->block_table, tb}};
  for (int i = 0; i < 3; i++) {
    for (int k = 0; k < 5; k++)
      if (!(i == k && outs[i].p == in[k].p) && !disjoint(outs[i].p, outs[i].n, in[k].p, in[k].n))
        return HYB_ERR_INVALID_VALUE;
    for (int k = 0; k < i; k++)
      if (!disjoint(outs[i].p, outs[i].n, outs[k].p, outs[k].n)) return HYB_ERR_INVALID_VALUE;
  }
  if (!disjoint(lens, nb, from->ring, rb)) return HYB_ERR_INVALID_VALUE;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < hyb_pool_workspace_bytes(from))
    return HYB_ERR_WORKSPACE;
  hyb::PoolArgs a;
  a.batch = from->batch;
  a.width = from->max_blocks_per_seq;
  a.cap = from->num_phys_blocks;
  a.hot = from->hot_tokens;
  a.bshift = block_shift(from->block_size);
  a.lens = lens;
  a.n_in = from->n_blocks;
  a.state_in = from->state;
  a.table_in = from->block_table;
  a.ring = from->ring;
  a.n_out = to->n_blocks;
  a.state_out = to->state;
  a.table_out = to->block_table;
  a.status = to->status;
  a.ws = to->state == from->state || to->n_blocks == from->n_blocks ? static_cast<int32_t *>(workspace) : nullptr;
  const cudaError_t e = hyb::launch_pool_resize(a, hyb::host_sm_count(), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HYB_OK : hyb::host_cuda_fail(e);
}

int hyb_slot_map(const hyb_pool_desc *p, const int32_t *lens, const int32_t *first, const int32_t *n_tok,
                 int32_t max_total, int32_t *cu, int64_t *slots, hyb_stream_t stream) {
  const int rc = check_geometry(p);
  if (rc != HYB_OK) return rc;
  if (!lens || !n_tok || !aligned(lens, 4) || !aligned(n_tok, 4) || (first && !aligned(first, 4)) ||
      (cu && !aligned(cu, 4)) || max_total < 0 || (max_total > 0 && !slots) || (slots && !aligned(slots, 8)))
    return HYB_ERR_INVALID_VALUE;
  hyb::SlotArgs a;
  a.batch = p->batch;
  a.width = p->max_blocks_per_seq;
  a.num_phys = p->num_phys_blocks;
  a.hot = p->hot_tokens;
  a.bshift = block_shift(p->block_size);
  a.max_total = max_total;
  a.lens = lens;
  a.first = first;
  a.n_tok = n_tok;
  a.table = p->block_table;
  a.cu = cu;
  a.slots = slots;
  a.status = p->status;
  const cudaError_t e = hyb::launch_slot_map(a, hyb::host_sm_count(), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HYB_OK : hyb::host_cuda_fail(e);
}

}  // extern "C"
