// spec.cuh -- argument blocks and launchers of the speculative-decoding
// kernels (tree attention, block tables, slot maps) and the host helpers they
// share with hyb_host.cu.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "hyb_spec.h"

namespace hyb {

struct TreeArgs {
  const uint8_t *hot;         // FP16 [batch][Hkv][hot][2][128]
  const uint8_t *cold;        // see hyb_kv.h
  const float *scales;        // [num_phys][Hkv][2]
  const int32_t *block_table; // [batch][max_blocks]
  const int32_t *seq_lens;    // [batch]
  const int32_t *n_int4;      // [batch] or null
  int32_t *status;
  const __half *q;            // FP16 [batch][max_tree][Hq][128]
  const __half *k_tree;       // FP16 [batch][max_tree][Hkv][128]
  const __half *v_tree;
  const uint64_t *mask;       // [batch][max_tree] or null (a chain)
  const int32_t *n_tree;      // [batch] or null (max_tree everywhere)
  __half *out;                // FP16 [batch][max_tree][Hq][128]
  float *lse_out;             // [batch][max_tree][Hq] or null
  int batch, hkv, hq, num_phys, max_blocks, quant_bits, hot_tokens, max_tree;
  int lsub;                   // log2 of the 64-token sub-blocks per block
  int bshift;                 // log2 of the tokens per block
  float qk_scale;             // softmax_scale * log2(e)
  int group;                  // Hq / Hkv
  int group_recip;            // 2^16 / group, rounded up
  int q_rows, q_bufs;         // rows of a Q buffer and buffers
  uint32_t wait_cycles;       // limit (SM cycles) of the bounded waits
  int ctas;                   // CTAs of the launch
  // units that several CTAs share (see tree.cu): sums and maxima [2 ctas][rows]
  // and outputs [2 ctas][32][rows][4] of the CTAs' parts, rows = 128 * MT, and for
  // each CTA the unit it has the first tile of {sequence, kv head, row group,
  // later CTAs} (0 later CTAs: none)
  float *part_ml;
  float *part_o;
  int4 *shared_units;
};

struct PoolArgs {
  int batch, width, cap, hot, bshift;
  const int32_t *lens;        // [batch]
  const int32_t *n_in;        // [batch]
  const int32_t *state_in;    // {head, count}
  const int32_t *table_in;    // [batch][width]
  int32_t *ring;              // [cap]
  int32_t *n_out, *state_out, *table_out;
  int32_t *status;
  // counts or state updated in place: {ticket, head, count}, then the new
  // counts [batch]; null when both go to other memory
  int32_t *ws;
};

struct SlotArgs {
  int batch, width, num_phys, hot, bshift, max_total;
  const int32_t *lens, *first, *n_tok, *table;
  int32_t *cu;
  int64_t *slots;
  int32_t *status;
};

cudaError_t launch_tree_attn(const TreeArgs &a, cudaStream_t stream);
// 128-row tiles a CTA takes at once for trees of max_tree nodes
inline int tree_m_tiles(int max_tree, int group) { return max_tree * group > 128 ? 2 : 1; }
cudaError_t launch_pool_resize(const PoolArgs &a, int sms, cudaStream_t stream);
cudaError_t launch_slot_map(const SlotArgs &a, int sms, cudaStream_t stream);

// hyb_host.cu: record a CUDA error for hyb_last_cuda_error and return
// HYB_ERR_CUDA; SMs of the current device; the limit of hyb_set_wait_limit
int host_cuda_fail(cudaError_t e);
int host_sm_count();
long long host_wait_cycles();

}  // namespace hyb
