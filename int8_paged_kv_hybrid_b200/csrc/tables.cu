// tables.cu -- hyb_pool_resize (block tables of a batch from request lengths)
// and hyb_slot_map (where packed tokens live).
//
// Both are prefix sums over the batch followed by a ragged fill.  With need_b
// = max(0, want_b - held_b) and back_b = max(0, held_b - want_b), sequence b
// takes the free entries [sum_{b'<b} need, + need_b) and gives its blocks back
// behind sum_{b'<b} back others; a token i of the packed list belongs to the
// sequence with cu[b] <= i < cu[b+1].  A decode batch's sums are a few KB, so
// every CTA computes them itself from the lengths (L2 hits) instead of waiting
// for a scan kernel: one launch, and no CTA depends on another.  What bounds
// them is the latency of launch, two dependent loads and the scan for batches
// up to some hundred sequences, and the table or slot writes above that.
#include "spec.cuh"

namespace hyb {

constexpr int kTabThreads = 256;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kTabPer = 8;                            // sequences per thread and scan
constexpr int kTabTile = kTabThreads * kTabPer;       // sequences per scan
constexpr int kTabSeg = 512;                          // table columns per unit of a warp
constexpr int kSlotChunk = 256;                       // tokens per unit of a warp

// Exclusive prefix of x over the CTA's threads; *total = the sum.
__device__ __forceinline__ long long cta_exclusive(long long x, long long *s_warp, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kTabWarps; w++) {
    const long long v = s_warp[w];
    if (w < warp) before += v;
    all += v;
  }
  __syncthreads();  // s_warp is reused
  *total = all;
  return before + inc - x;
}

// ---- hyb_pool_resize ----

struct PoolRow {
  int held;   // blocks held (a count out of range: the whole row stays)
  int want;   // blocks wanted (held where the request is refused)
  int status; // 0 or why the sequence stays as it is
};

__device__ __forceinline__ PoolRow pool_row(const PoolArgs &a, int b, bool frozen) {
  PoolRow r;
  const int n = a.n_in[b], len = a.lens[b];
  const bool bad_n = n < 0 || n > a.width;
  r.held = bad_n ? a.width : n;
  r.want = r.held;
  r.status = bad_n ? HYB_STATUS_CAPACITY : 0;
  if (bad_n || frozen) return r;
  if (len < 0) {
    r.status = HYB_STATUS_SEQ_LEN;
    return r;
  }
  const long long cold = max(0, len - a.hot);
  const long long want = (cold + (1ll << a.bshift) - 1) >> a.bshift;
  if (want > a.width) r.status = HYB_STATUS_CAPACITY;
  else r.want = static_cast<int>(want);
  return r;
}

__global__ void __launch_bounds__(kTabThreads) pool_resize_kernel(const PoolArgs a) {
  __shared__ long long s_warp[kTabWarps];
  __shared__ int s_take[kTabTile], s_give[kTabTile], s_new[kTabTile];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int segs = (a.width + kTabSeg - 1) / kTabSeg;
  const long long units = static_cast<long long>(a.batch) * segs;
  const long long u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  const long long head = a.state_in[0], count = a.state_in[1];

  // blocks given back by the whole batch: the ring must hold them beside its
  // free ones, and then no entry taken and no place given back to coincide
  long long back = 0, total_back, unused;
  for (int b = tid; b < a.batch; b += kTabThreads) {
    const PoolRow r = pool_row(a, b, false);
    back += max(0, r.held - r.want);
  }
  cta_exclusive(back, s_warp, &total_back);
  const bool frozen = head < 0 || head >= a.cap || count < 0 || count > a.cap || count + total_back > a.cap;
  if (frozen) total_back = 0;
  if (frozen && blockIdx.x == 0 && tid == 0) set_status(a.status, HYB_STATUS_POOL);

  long long need0 = 0, back0 = 0;  // sums over the sequences before the tile
  long long taken = 0;             // blocks handed out (CTA 0)
  for (int t0 = 0; t0 < a.batch; t0 += kTabTile) {
    // the others stop behind their last row; CTA 0 sums the blocks handed out
    if (blockIdx.x != 0 && static_cast<long long>(t0) * segs >= u1) break;
    const int b0 = t0 + tid * kTabPer;
    int need[kTabPer], give[kTabPer];
    PoolRow row[kTabPer];
    long long nsum = 0, gsum = 0;
#pragma unroll
    for (int k = 0; k < kTabPer; k++) {
      row[k] = PoolRow{0, 0, 0};
      if (b0 + k < a.batch) row[k] = pool_row(a, b0 + k, frozen);
      need[k] = max(0, row[k].want - row[k].held);
      give[k] = max(0, row[k].held - row[k].want);
      nsum += need[k];
      gsum += give[k];
    }
    long long tile_need, tile_back;
    long long n = need0 + cta_exclusive(nsum, s_warp, &tile_need);
    long long g = back0 + cta_exclusive(gsum, s_warp, &tile_back);
    long long got = 0;
#pragma unroll
    for (int k = 0; k < kTabPer; k++) {
      const int b = b0 + k, i = tid * kTabPer + k;
      const bool fits = need[k] == 0 || n + need[k] <= count;
      s_take[i] = fits ? static_cast<int>(n < count ? n : count) : 0;  // <= count where it is used
      s_give[i] = static_cast<int>(g);                                 // <= total_back
      s_new[i] = fits ? row[k].want : row[k].held;
      if (fits) got += need[k];
      if (b < a.batch) {
        const long long u = static_cast<long long>(b) * segs;
        if (u >= u0 && u < u1) {  // the CTA with the row's first unit
          const int nb = row[k].status == HYB_STATUS_CAPACITY ? a.n_in[b] : s_new[i];
          if (a.ws) a.ws[4 + b] = nb;
          else a.n_out[b] = nb;
          if (row[k].status) set_status(a.status, row[k].status);
          if (!fits) set_status(a.status, HYB_STATUS_POOL);
        }
      }
      n += need[k];
      g += give[k];
    }
    if (blockIdx.x == 0) {
      cta_exclusive(got, s_warp, &unused);
      taken += unused;
    }
    __syncthreads();
    // the rows of this tile that are this CTA's, kTabSeg columns per warp
    const long long ua = max(u0, static_cast<long long>(t0) * segs);
    const long long ub = min(u1, static_cast<long long>(min(t0 + kTabTile, a.batch)) * segs);
    for (long long u = ua + warp; u < ub; u += kTabWarps) {
      const int b = static_cast<int>(u / segs), i = b - t0;
      const int c0 = static_cast<int>(u % segs) * kTabSeg, c1 = min(c0 + kTabSeg, a.width);
      const PoolRow r = pool_row(a, b, frozen);
      const int now = s_new[i], keep = min(r.held, now);
      const long long from = head + s_take[i] - r.held, to = head + count + s_give[i] - now;
      const int32_t *in = a.table_in + static_cast<size_t>(b) * a.width;
      int32_t *out = a.table_out + static_cast<size_t>(b) * a.width;
      bool bad = false;
      for (int c = c0 + lane; c < c1; c += 32) {
        int v = -1;
        if (c < keep) {
          if (in == out) continue;
          v = in[c];
        } else if (c < now) {
          long long at = from + c;
          if (at >= a.cap) at -= a.cap;
          v = a.ring[at];
          bad |= v < 0 || v >= a.cap;
        } else if (c < r.held) {
          long long at = to + c;
          if (at >= a.cap) at -= a.cap;
          if (at >= a.cap) at -= a.cap;
          const int x = in[c];
          bad |= x < 0 || x >= a.cap;
          a.ring[at] = x;
        }
        out[c] = v;
      }
      if (bad) set_status(a.status, HYB_STATUS_BAD_BLOCK);
    }
    __syncthreads();  // the tile's sums are replaced
    need0 += tile_need;
    back0 += tile_back;
  }
  if (blockIdx.x == 0 && tid == 0) {
    const long long c = frozen ? count : count - taken + total_back;
    long long h = frozen ? head : head + taken;
    if (!frozen && h >= a.cap) h -= a.cap;
    int32_t *st = a.ws ? a.ws + 1 : a.state_out;
    st[0] = static_cast<int32_t>(h);
    st[1] = static_cast<int32_t>(c);
  }
  if (!a.ws) return;
  // counts or state in place: every CTA reads all of them, so the last one to
  // come here stores the new ones
  __syncthreads();
  if (tid == 0) s_last = atomic_add_acq_rel_gpu(a.ws, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (!s_last) return;
  for (int b = tid; b < a.batch; b += kTabThreads) a.n_out[b] = __ldcg(a.ws + 4 + b);
  if (tid < 2) a.state_out[tid] = __ldcg(a.ws + 1 + tid);
  if (tid == 0) a.ws[0] = 0;
}

cudaError_t launch_pool_resize(const PoolArgs &a, int sms, cudaStream_t stream) {
  const long long segs = (a.width + kTabSeg - 1) / kTabSeg;
  const long long want = (a.batch * segs + kTabWarps - 1) / kTabWarps;
  const int grid = static_cast<int>(want < 2ll * sms ? want : 2ll * sms);
  pool_resize_kernel<<<grid, kTabThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// ---- hyb_slot_map ----

__global__ void __launch_bounds__(kTabThreads) slot_map_kernel(const SlotArgs a) {
  __shared__ long long s_warp[kTabWarps];
  __shared__ int s_cu[kTabTile + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long sum = 0, all;
  bool neg = false;
  for (int b = tid; b < a.batch; b += kTabThreads) {
    const int n = a.n_tok[b];
    neg |= n < 0;
    sum += max(0, n);
  }
  cta_exclusive(sum, s_warp, &all);
  if (blockIdx.x == 0) {
    if (neg) set_status(a.status, HYB_STATUS_BAD_N_NEW);
    if (tid == 0 && all > a.max_total) set_status(a.status, HYB_STATUS_CAPACITY);
  }
  const long long total = min(all, static_cast<long long>(a.max_total));
  const long long o0 = total * blockIdx.x / gridDim.x, o1 = total * (blockIdx.x + 1) / gridDim.x;
  const int mask = (1 << a.bshift) - 1;
  bool bad = false;
  long long before = 0;  // tokens of the sequences before the tile
  for (int t0 = 0; t0 < a.batch; t0 += kTabTile) {
    if (before >= o1 && !(blockIdx.x == 0 && a.cu)) break;
    const int b0 = t0 + tid * kTabPer;
    int n[kTabPer];
    long long s = 0, tile;
#pragma unroll
    for (int k = 0; k < kTabPer; k++) {
      n[k] = b0 + k < a.batch ? max(0, a.n_tok[b0 + k]) : 0;
      s += n[k];
    }
    long long at = before + cta_exclusive(s, s_warp, &tile);
#pragma unroll
    for (int k = 0; k < kTabPer; k++) {
      const int v = static_cast<int>(min(at, total));
      s_cu[tid * kTabPer + k] = v;
      if (blockIdx.x == 0 && a.cu && b0 + k < a.batch) a.cu[b0 + k] = v;
      at += n[k];
    }
    const long long next = before + tile;
    if (tid == 0) s_cu[kTabTile] = static_cast<int>(min(next, total));
    __syncthreads();
    const long long ta = max(o0, before), tb = min(o1, next);
    for (long long w0 = ta + warp * kSlotChunk; w0 < tb; w0 += kTabWarps * kSlotChunk) {
      long long i = w0 + lane;
      const long long w1 = min(w0 + kSlotChunk, tb);
      if (i >= w1) continue;
      int lo = 0, hi = kTabTile;  // s_cu[lo] <= i < s_cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= i) lo = mid;
        else hi = mid;
      }
      int held = -1, len = 0, f = 0;
      for (; i < w1; i += 32) {
        while (s_cu[lo + 1] <= i) lo++;  // s_cu[kTabTile] = tokens up to the tile's end > i
        const int b = t0 + lo;
        if (b != held) {
          held = b;
          len = a.lens[b];
          f = a.first ? a.first[b] : 0;
        }
        const long long p = static_cast<long long>(f) + (i - s_cu[lo]);
        long long slot = HYB_SLOT_NONE;
        if (p >= 0 && p < len) {
          if (p >= static_cast<long long>(len) - a.hot) {
            slot = -2 - (static_cast<long long>(b) * a.hot + (p & (a.hot - 1)));
          } else {
            const long long col = p >> a.bshift;
            const int phys = col < a.width ? a.table[static_cast<size_t>(b) * a.width + col] : -1;
            if (phys < 0 || phys >= a.num_phys) bad = true;
            else slot = (static_cast<long long>(phys) << a.bshift) + (p & mask);
          }
        }
        a.slots[i] = slot;
      }
    }
    __syncthreads();  // s_cu is replaced
    before = next;
  }
  if (blockIdx.x == 0 && a.cu && tid == 0) a.cu[a.batch] = static_cast<int>(total);
  if (bad) set_status(a.status, HYB_STATUS_BAD_BLOCK);
}

cudaError_t launch_slot_map(const SlotArgs &a, int sms, cudaStream_t stream) {
  const long long per = kTabWarps * kSlotChunk;
  const long long want = (static_cast<long long>(a.max_total) + per - 1) / per;
  const int grid = static_cast<int>(want < 1 ? 1 : (want < 4ll * sms ? want : 4ll * sms));
  slot_map_kernel<<<grid, kTabThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace hyb
