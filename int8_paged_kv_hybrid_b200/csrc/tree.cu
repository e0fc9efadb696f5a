// tree.cu -- hyb_tree_attn: attention of drafted tree nodes over the cache.
//
// One CTA of 128 threads per (node, query head) row.  Keys are taken 128 at a
// time: thread = key for the logits, thread = channel for the weighted sum of
// V, with the running maximum and sum of an online softmax between them.
#include "spec.cuh"

namespace hyb {

constexpr int kTreeThreads = 128;

// Code of (slot, channel) of a K or V tile (slot within its 64-slot sub-block).
__device__ __forceinline__ int tile_code(const uint8_t *tile, int kv, bool int4, int slot, int ch) {
  if (!int4)
    return static_cast<int8_t>(kv == 0 ? tile[slot * 128 + ch]
                                       : tile[ch * 64 + 16 * ((slot >> 4) ^ ((ch >> 1) & 3)) + (slot & 15)]);
  const int e = kv == 0 ? ch & 7 : slot & 7;
  const int word = kv == 0 ? slot * 16 + (ch >> 3)
                           : ch * 8 + 2 * ((slot >> 4) ^ ((ch >> 2) & 3)) + ((slot >> 3) & 1);
  return nib_get(reinterpret_cast<const uint32_t *>(tile)[word], e);
}

struct TreeKey {
  int kind;  // 0 not attended, 1 cold, 2 ring, 3 node
  int slot, phys;
};

__device__ __forceinline__ float key_value(const TreeArgs &a, const TreeKey &k, int b, int h, int kv, int ch, int block) {
  if (k.kind == 2)
    return __half2float(reinterpret_cast<const __half *>(
        a.hot)[((((size_t)b * a.hkv + h) * a.hot_tokens + k.slot) * 2 + kv) * kDim + ch]);
  if (k.kind == 3)
    return __half2float((kv ? a.v_tree : a.k_tree)[(((size_t)b * a.max_tree + k.slot) * a.hkv + h) * kDim + ch]);
  if (a.quant_bits == 0)
    return __half2float(reinterpret_cast<const __half *>(
        a.cold + (((size_t)k.phys * a.hkv + h) << a.bshift) * kHotTokenBytes)[(k.slot * 2 + kv) * kDim + ch]);
  const bool int4 = a.quant_bits == 4 || (a.n_int4 != nullptr && block < a.n_int4[b]);
  const uint8_t *tile = a.cold + ((((size_t)k.phys * a.hkv + h) << a.lsub) + (k.slot >> 6)) * kTilePairBytes + kv * kTileBytes;
  return tile_code(tile, kv, int4, k.slot & 63, ch) * a.scales[((size_t)k.phys * a.hkv + h) * 2 + kv];
}

__global__ void __launch_bounds__(kTreeThreads) tree_kernel(const TreeArgs a) {
  const int hq = blockIdx.x, t = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int h = hq / (a.hq / a.hkv);
  const int nt = a.n_tree ? a.n_tree[b] : a.max_tree;
  if (nt < 0 || nt > a.max_tree) {
    if (tid == 0 && t == 0 && hq == 0) set_status(a.status, HYB_STATUS_BAD_TREE);
    return;
  }
  if (t >= nt) return;
  int L = a.seq_lens[b];
  const bool bad_len = L < 0 || static_cast<long long>(L) - a.hot_tokens > (static_cast<long long>(a.max_blocks) << a.bshift);
  if (bad_len && tid == 0 && t == 0 && hq == 0) set_status(a.status, HYB_STATUS_SEQ_LEN);
  uint64_t m = a.mask ? a.mask[(size_t)b * a.max_tree + t] : (~0ull >> (63 - t));
  if (nt < 64) m &= (1ull << nt) - 1;
  const int keys = bad_len ? 0 : L + nt;
  const int cold = bad_len ? 0 : max(0, L - a.hot_tokens);
  __shared__ float s_q[kDim], s_p[kTreeThreads], s_red[4];
  __shared__ TreeKey s_key[kTreeThreads];
  s_q[tid] = __half2float(a.q[(((size_t)b * a.max_tree + t) * a.hq + hq) * kDim + tid]);
  float top = -INFINITY, sum = 0.f, acc = 0.f;
  for (int k0 = 0; k0 < keys; k0 += kTreeThreads) {
    __syncthreads();
    const int p = k0 + tid;
    TreeKey k{0, 0, 0};
    if (p < cold) {
      k.slot = p & ((1 << a.bshift) - 1);
      k.phys = a.block_table[(size_t)b * a.max_blocks + (p >> a.bshift)];
      k.kind = k.phys >= 0 && k.phys < a.num_phys;
      if (!k.kind) set_status(a.status, HYB_STATUS_BAD_BLOCK);
    } else if (p < L) {
      k.kind = 2;
      k.slot = p & (a.hot_tokens - 1);
    } else if (p < keys && (m >> (p - L) & 1)) {
      k.kind = 3;
      k.slot = p - L;
    }
    float z = -INFINITY;
    if (k.kind) {
      z = 0.f;
      for (int c = 0; c < kDim; c++) z = fmaf(s_q[c], key_value(a, k, b, h, 0, c, p >> a.bshift), z);
      z *= a.qk_scale;
    }
    s_key[tid] = k;
    float mx = z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) s_red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])), top);
    const float base = mx == -INFINITY ? 0.f : mx;
    s_p[tid] = k.kind ? exp2f(z - base) : 0.f;
    __syncthreads();
    const float r = exp2f(top - base);
    acc *= r;
    sum *= r;
    top = mx;
    for (int j = 0; j < kTreeThreads; j++) {
      if (s_key[j].kind == 0) continue;
      sum += s_p[j];
      acc = fmaf(s_p[j], key_value(a, s_key[j], b, h, 1, tid, (k0 + j) >> a.bshift), acc);
    }
  }
  const size_t row = ((size_t)b * a.max_tree + t) * a.hq + hq;
  a.out[row * kDim + tid] = __float2half_rn(sum > 0.f ? acc / sum : 0.f);
  if (tid == 0 && a.lse_out) a.lse_out[row] = sum > 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

cudaError_t launch_tree_attn(const TreeArgs &a, cudaStream_t stream) {
  tree_kernel<<<dim3(a.hq, a.max_tree, a.batch), kTreeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace hyb
