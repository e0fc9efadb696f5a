// tree.cu -- hyb_tree_attn: attention of drafted tree nodes over the cache, on
// the fifth-generation tensor cores.
//
// Mathematics.  The nt nodes of a sequence and the G query heads of a kv head
// make M = nt G query rows that share their keys, up to the tree's mask.  Per
// 128-key tile: S = Q K^T, the online softmax (running maximum m, sum l) and
// O += P V.  INT8 / INT4 codes are integers that FP16 holds exactly, so K and
// V enter the products as codes: a tile's K scale multiplies its logits, its V
// scale the weights, both in FP32.  The weights p s_v / r are rounded once to
// FP16 (half a step, 2^-11 relative; the tensor core takes no FP32 operand),
// r being one of the V scales met, so that the FP16 range serves weights, not
// scales: O holds the sum in units of r.  m may lag behind the maximum by
// kLagLog2 (weights up to 2^6) and r behind the scales by kLagScale, so that O
// is rescaled when they grow by much only; a weight stays below 2^14.  Products
// are exact, sums FP32 in TMEM and registers.
//
// Work split.  A unit is (sequence, kv head, group of 128 * MT rows).  Its
// tiles -- cold tiles of 128 positions, then the hot ring and the drafted
// nodes as rows of FP16 tiles -- follow each other in one list over the batch,
// cut into one run of equal length per CTA (one CTA per SM): no SM idles
// whatever the lengths are, and nothing on the host depends on them.  A unit
// inside one run is finished there; the others leave (O, m, l) per CTA, and
// tree_combine_kernel merges them in the order of the tiles.
//
// Inside a CTA: eight producer warps bring codes or rows to FP16 in the
// 128-byte swizzled layout of the MMA's shared operands, one thread issues the
// MMAs, and four warps per 128 rows keep the softmax (one row per thread) and
// write the weights back over the logits in TMEM, where the second product
// reads them as its A operand.
#include "kernels.cuh"
#include "spec.cuh"
#include "tc05.cuh"

namespace hyb {

constexpr int kTK = 128;                     // keys per tile
constexpr int kTreeProducers = 8;            // producer warps
constexpr int kTreeStages = 2;               // K and V tiles in shared memory
constexpr int kTreeMeta = 4;                 // tile records (see the producers)
constexpr uint32_t kTreeOperand = 128 * 256; // bytes of a 128 x 128 FP16 operand
constexpr uint32_t kTreeSlab = kTreeOperand / 2;  // its halves of 64 columns
constexpr float kLagLog2 = 6.f;
constexpr float kLagScale = 256.f;

// What the softmax needs to know of a tile; four units of 32 keys.
struct TreeMeta {
  float k_scale[4];  // 1 for FP16 rows
  float v_scale[4];
  uint32_t ok[4];    // keys that every row attends
  uint32_t bad[kTreeProducers][4];  // FP16 rows of a tail tile with a V that is not finite
};

template <int MT>
struct TreeSmem {
  static constexpr int kQ = MT == 1 ? 2 : 1;  // Q buffers
  uint64_t kfull[kTreeStages], kempty[kTreeStages], vfull[kTreeStages], vempty[kTreeStages];
  uint64_t mfull[kTreeMeta];
  uint64_t qfull[kQ], qempty[kQ];
  uint64_t sfull[2], pfull[2];  // by S buffer (MT 1) or row tile (MT 2)
  uint64_t odone[2][2];         // by row tile and parity of its tile (a waiter may be two tiles behind)
  uint64_t ofree[2];            // by row tile
  uint64_t drain;
  TreeMeta meta[kTreeMeta];
  uint32_t tmem;
  volatile int abort;
  int start_b;
  long long start_base, total;
  long long warp_sum[32];
};

template <int MT>
struct TreeShape {
  static constexpr int kSoftWarps = 4 * MT;
  static constexpr int kThreads = 32 * (kSoftWarps + kTreeProducers + 1);
  static constexpr uint32_t kQBytes = TreeSmem<MT>::kQ * MT * kTreeOperand;
  static constexpr uint32_t kBytes = 1024 + kQBytes + 2 * kTreeStages * kTreeOperand + sizeof(TreeSmem<MT>);
};

// ---- the list of tiles ----

struct TreeSeq {
  int cold, hot, nt, keys;  // cold and ring tokens, nodes (rows), nodes that are keys
  int tiles, groups;        // per unit; row groups
  long long span;           // tiles of all its units
  int status;
};

template <int MT>
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs &a, int b) {
  TreeSeq s;
  const int L = a.seq_lens[b];
  s.nt = a.n_tree ? a.n_tree[b] : a.max_tree;
  s.status = 0;
  if (s.nt < 0 || s.nt > a.max_tree) {
    s.nt = 0;
    s.status = HYB_STATUS_BAD_TREE;
  }
  const bool bad = L < 0 || static_cast<long long>(L) - a.hot_tokens > (static_cast<long long>(a.max_blocks) << a.bshift);
  if (bad && s.nt > 0) s.status = HYB_STATUS_SEQ_LEN;
  s.cold = bad ? 0 : max(0, L - a.hot_tokens);
  s.hot = bad ? 0 : L - s.cold;
  s.keys = bad ? 0 : s.nt;
  s.tiles = max(1, (s.cold + kTK - 1) / kTK + (s.hot + s.keys + kTK - 1) / kTK);
  s.groups = (s.nt * (a.hq / a.hkv) + 128 * MT - 1) / (128 * MT);
  s.span = static_cast<long long>(s.tiles) * s.groups * a.hkv;
  return s;
}

// A run of tiles [w, w1) taken unit by unit.
template <int MT>
struct TreeWalk {
  long long w, w1, base;  // base: the list's index of sequence b's first tile
  int b;
  TreeSeq s;
  int hk, mg, t0, t1;     // the current segment: tiles [t0, t1) of unit (b, hk, mg)

  __device__ __forceinline__ void init(const TreeArgs &a, long long w_, long long w1_, long long base_, int b_) {
    w = w_;
    w1 = w1_;
    base = base_;
    b = b_;
    s = tree_seq<MT>(a, b);
  }
  __device__ __forceinline__ bool next(const TreeArgs &a) {
    if (w >= w1) return false;
    while (w >= base + s.span) {
      base += s.span;
      s = tree_seq<MT>(a, ++b);
    }
    const long long r = w - base;
    const int unit = static_cast<int>(r / s.tiles);
    t0 = static_cast<int>(r - static_cast<long long>(unit) * s.tiles);
    t1 = static_cast<int>(min(static_cast<long long>(s.tiles), t0 + (w1 - w)));
    hk = unit / s.groups;
    mg = unit - hk * s.groups;
    w += t1 - t0;
    return true;
  }
  // 128-row tiles of this unit that have a row
  __device__ __forceinline__ int m_tiles(const TreeArgs &a) const {
    const int rows = s.nt * (a.hq / a.hkv) - mg * 128 * MT;
    return MT == 1 ? 1 : min(MT, (rows + 127) / 128);
  }
};

// Wait for phase `parity`; false when the wait or the kernel gave up.
template <typename Sm>
__device__ __forceinline__ bool tree_wait(Sm &sm, uint64_t *bar, uint32_t parity, const TreeArgs &a) {
  if (mbar_test_wait(bar, parity)) return true;
  const bool quick = a.wait_cycles < kShortWaitCycles;
  const long long t0 = clock64();
  while (!(quick ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
    if (sm.abort) return false;
    if (clock64() - t0 > a.wait_cycles) {
      sm.abort = 1;
      set_status(a.status, HYB_STATUS_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The same for all lanes of a warp, with one answer.
template <typename Sm>
__device__ __forceinline__ bool tree_wait_warp(Sm &sm, uint64_t *bar, uint32_t parity, const TreeArgs &a) {
  return __all_sync(0xffffffffu, tree_wait(sm, bar, parity, a));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// ---- producers ----

// Eight codes (two words of four bytes, biased by 2^(bits-1)) as FP16: byte u
// under the exponent of 1024 is 1024 + u, and the subtraction is exact.
__device__ __forceinline__ uint4 f16_codes(uint32_t lo, uint32_t hi, uint32_t bias) {
  const __half2 off = __halves2half2(__ushort_as_half(static_cast<unsigned short>(bias)),
                                     __ushort_as_half(static_cast<unsigned short>(bias)));
  auto two = [&](uint32_t x, uint32_t sel) {
    const uint32_t h = __byte_perm(x, 0x64646464u, sel);
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&h), off);
    return *reinterpret_cast<const uint32_t *>(&d);
  };
  return make_uint4(two(lo, 0x4140), two(lo, 0x4342), two(hi, 0x4140), two(hi, 0x4342));
}
__device__ __forceinline__ uint4 f16_int8(uint32_t w0, uint32_t w1) {  // eight INT8 codes
  return f16_codes(w0 ^ 0x80808080u, w1 ^ 0x80808080u, 0x6480);        // 1024 + 128
}
__device__ __forceinline__ uint4 f16_int4(uint32_t w) {  // eight INT4 codes of a word
  return f16_codes((w & 0x0f0f0f0fu) ^ 0x08080808u, ((w >> 4) & 0x0f0f0f0fu) ^ 0x08080808u, 0x6408);  // 1024 + 8
}

__device__ __forceinline__ bool f16_not_finite(uint32_t h) { return (h & 0x7c00u) == 0x7c00u; }

// A producer thread's part of a tile: units u and u + 2 (u = thread / 128) of
// 32 keys.  K: key (thread % 128) / 4, 32 channels; V: INT8 / INT4 channel
// thread % 128, all 32 keys; FP16 channels 2 (thread % 64), + 1 and 16 keys.
template <bool kF16>
struct TreeRegs {
  uint4 k[2][kF16 ? 4 : 2];
  uint4 v[2][kF16 ? 4 : 2];
};

struct TreeTile {
  int b, hk, mg, ti;   // unit and tile; ti < 0: the list's end
  int cold, hot, keys, nt;
  bool first;          // of its segment
  int ent[2];          // block-table entries of the two units (-1: none)
};

template <int MT>
struct TreeFeed {
  TreeWalk<MT> walk;
  int t, unit0;  // next tile of the walk's segment; the thread's first unit
  bool live;

  __device__ __forceinline__ TreeTile next(const TreeArgs &a) {
    TreeTile x;
    bool first = false;
    if (live && t == walk.t1) {
      live = walk.next(a);
      t = walk.t0;
      first = true;
    }
    if (!live) {
      x.ti = -1;
      return x;
    }
    x.b = walk.b;
    x.hk = walk.hk;
    x.mg = walk.mg;
    x.cold = walk.s.cold;
    x.hot = walk.s.hot;
    x.keys = walk.s.keys;
    x.nt = walk.s.nt;
    x.first = first;
    x.ti = t++;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int p = x.ti * kTK + 32 * (unit0 + 2 * i);
      x.ent[i] = p < x.cold ? __ldg(a.block_table + static_cast<size_t>(x.b) * a.max_blocks + (p >> a.bshift)) : -1;
    }
    return x;
  }
};

// Where unit i of a cold tile lives: valid keys (0: nothing to read).
struct TreeUnit {
  int n;
  bool int4;
  const uint8_t *base;  // the 64-token tile pair, or (FP16) the unit's first row
  int half;             // slots 32 half .. of the tile pair
};

template <bool kF16>
__device__ __forceinline__ TreeUnit tree_unit(const TreeArgs &a, const TreeTile &x, int i, int u) {
  TreeUnit r;
  const int p = x.ti * kTK + 32 * (u + 2 * i);
  r.n = max(0, min(32, x.cold - p));
  const int phys = x.ent[i];
  if (r.n > 0 && (phys < 0 || phys >= a.num_phys)) {
    set_status(a.status, HYB_STATUS_BAD_BLOCK);
    r.n = 0;
  }
  const int slot = p & ((1 << a.bshift) - 1);
  const size_t pair = static_cast<size_t>(r.n > 0 ? phys : 0) * a.hkv + x.hk;
  if (kF16) {
    r.int4 = false;
    r.half = 0;
    r.base = a.cold + (((pair << a.bshift) + slot) * kHotTokenBytes);
  } else {
    r.int4 = a.quant_bits == 4 || (a.n_int4 != nullptr && (p >> a.bshift) < a.n_int4[x.b]);
    r.half = (slot >> 5) & 1;
    r.base = a.cold + ((pair << a.lsub) + (slot >> 6)) * kTilePairBytes;
  }
  return r;
}

__device__ __forceinline__ uint4 ldg_nc(const void *p) { return __ldg(static_cast<const uint4 *>(p)); }

// FP16 rows: 32 channels of the thread's key (K) ...
__device__ __forceinline__ void rows_k(const __half *row, bool valid, int tid, uint4 (&k)[4]) {
#pragma unroll
  for (int j = 0; j < 4; j++)
    k[j] = valid ? ldg_nc(row + 32 * (tid & 3) + 8 * j) : make_uint4(0, 0, 0, 0);
}

// ... and two channels of 16 keys (V); row(j) is the V row of key j or null.
template <typename Row>
__device__ __forceinline__ void rows_v(Row row, int tid, uint4 (&v)[4]) {
  uint32_t *w = reinterpret_cast<uint32_t *>(v);
  const int k0 = 16 * ((tid >> 6) & 1), c = 2 * (tid & 63);
#pragma unroll
  for (int j = 0; j < 16; j++) {
    const __half *r = row(k0 + j);
    w[j] = r ? __ldg(reinterpret_cast<const uint32_t *>(r + c)) : 0u;
  }
}

template <bool kF16>
__device__ __forceinline__ void load_cold_k(const TreeUnit &n, int tid, uint4 (&k)[kF16 ? 4 : 2]) {
  const int key = (tid & 127) >> 2;
  if constexpr (kF16) {
    rows_k(reinterpret_cast<const __half *>(n.base) + key * 2 * kDim, key < n.n, tid, k);
  } else {
    k[0] = k[1] = make_uint4(0, 0, 0, 0);
    if (n.n == 0) return;
    const int slot = 32 * n.half + key;
    if (n.int4) {
      k[0] = ldg_nc(n.base + slot * 64 + 16 * (tid & 3));
    } else {
      k[0] = ldg_nc(n.base + slot * 128 + 32 * (tid & 3));
      k[1] = ldg_nc(n.base + slot * 128 + 32 * (tid & 3) + 16);
    }
  }
}

template <bool kF16>
__device__ __forceinline__ void load_cold_v(const TreeUnit &n, int tid, uint4 (&v)[kF16 ? 4 : 2]) {
  if constexpr (kF16) {
    const __half *base = reinterpret_cast<const __half *>(n.base) + kDim;
    rows_v([&](int j) { return j < n.n ? base + j * 2 * kDim : nullptr; }, tid, v);
  } else {
    v[0] = v[1] = make_uint4(0, 0, 0, 0);
    if (n.n == 0) return;
    // the unit's two 16-slot chunks are one aligned pair, swapped where the
    // swizzle's lowest bit is set: v[0] is slots 0..15, v[1] 16..31 (INT4:
    // words 0, 1 and 2, 3 of v[0])
    const int c = tid & 127;
    const uint8_t *t = n.base + kTileBytes;
    if (n.int4) {
      const int x = (c >> 2) & 3;
      const uint4 y = ldg_nc(t + c * 32 + 8 * ((2 * n.half) ^ (x & 2)));
      v[0] = x & 1 ? make_uint4(y.z, y.w, y.x, y.y) : y;
    } else {
      const int x = (c >> 1) & 3;
      const uint8_t *p = t + c * 64 + 16 * ((2 * n.half) ^ (x & 2));
      const uint4 y = ldg_nc(p), z = ldg_nc(p + 16);
      v[0] = x & 1 ? z : y;
      v[1] = x & 1 ? y : z;
    }
  }
}

// K of one unit into the operand: row = key, 32 channels = four 16-byte chunks
// of a 64-channel slab.  Eight lanes are two rows of four threads; threads 2
// and 3 of a row write their chunks in the order k ^ 2, which spreads the
// eight over the banks.
__device__ __forceinline__ void store_k16(uint32_t st, int u, int tid, const uint4 (&k)[4]) {
  const int row = 32 * u + ((tid & 127) >> 2), i = tid & 3;
  const uint32_t base = st + (i >> 1) * kTreeSlab + row * 128;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const uint4 x = i & 2 ? k[j ^ 2] : k[j];
    const int c = 4 * (i & 1) + (i & 2 ? j ^ 2 : j);
    sts128(base + ((c ^ (row & 7)) << 4), x);
  }
}

__device__ __forceinline__ void store_k8(uint32_t st, int u, int tid, bool int4, const uint4 (&k)[2]) {
  uint4 f[4];
  if (int4) {
    f[0] = f16_int4(k[0].x);
    f[1] = f16_int4(k[0].y);
    f[2] = f16_int4(k[0].z);
    f[3] = f16_int4(k[0].w);
  } else {
    f[0] = f16_int8(k[0].x, k[0].y);
    f[1] = f16_int8(k[0].z, k[0].w);
    f[2] = f16_int8(k[1].x, k[1].y);
    f[3] = f16_int8(k[1].z, k[1].w);
  }
  store_k16(st, u, tid, f);
}

// V of one unit: row = channel, the unit's 32 keys = four chunks of a 64-key
// slab; eight lanes are eight rows, all banks.
__device__ __forceinline__ void store_v8(uint32_t st, int u, int tid, bool int4, const uint4 (&v)[2]) {
  const int row = tid & 127;
  const uint32_t base = st + (u >> 1) * kTreeSlab + row * 128;
  const int c = 4 * (u & 1), x = row & 7;
  if (int4) {
    sts128(base + (((c + 0) ^ x) << 4), f16_int4(v[0].x));
    sts128(base + (((c + 1) ^ x) << 4), f16_int4(v[0].y));
    sts128(base + (((c + 2) ^ x) << 4), f16_int4(v[0].z));
    sts128(base + (((c + 3) ^ x) << 4), f16_int4(v[0].w));
  } else {
    sts128(base + (((c + 0) ^ x) << 4), f16_int8(v[0].x, v[0].y));
    sts128(base + (((c + 1) ^ x) << 4), f16_int8(v[0].z, v[0].w));
    sts128(base + (((c + 2) ^ x) << 4), f16_int8(v[1].x, v[1].y));
    sts128(base + (((c + 3) ^ x) << 4), f16_int8(v[1].z, v[1].w));
  }
}

// FP16 V of one unit: the thread's two channels are two rows, its 16 keys two
// chunks of each.  Lanes 4..7 of eight write their odd row first, so that the
// eight rows differ modulo 8.
__device__ __forceinline__ void store_v16(uint32_t st, int u, int tid, const uint4 (&v)[4]) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
  const int p = tid & 63, odd = (p >> 2) & 1;
  const int c0 = 4 * (u & 1) + 2 * ((tid >> 6) & 1);
#pragma unroll
  for (int s = 0; s < 2; s++) {
    const int hi = s ^ odd, row = 2 * p + hi;
    const uint32_t base = st + (u >> 1) * kTreeSlab + row * 128;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; e++)
        o[e] = __byte_perm(w[8 * j + 2 * e], w[8 * j + 2 * e + 1], hi ? 0x7632 : 0x5410);
      sts128(base + (((c0 + j) ^ (row & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

// Row r of the tail (ring rows in the order of their positions, then nodes):
// its K row (V row: + add), or null.
__device__ __forceinline__ const __half *tail_row(const TreeArgs &a, const TreeTile &x, int r, int kv) {
  if (r < x.hot) {
    const int slot = (x.cold + r) & (a.hot_tokens - 1);
    return reinterpret_cast<const __half *>(a.hot) +
           (((static_cast<size_t>(x.b) * a.hkv + x.hk) * a.hot_tokens + slot) * 2 + kv) * kDim;
  }
  r -= x.hot;
  if (r >= x.keys) return nullptr;
  return (kv ? a.v_tree : a.k_tree) + ((static_cast<size_t>(x.b) * a.max_tree + r) * a.hkv + x.hk) * kDim;
}

// The query rows of a unit into its Q operand(s); rows beyond the tree are 0.
template <int MT>
__device__ __forceinline__ void load_q(const TreeArgs &a, const TreeTile &x, uint32_t st, int tid) {
  const int G = a.hq / a.hkv, rows = x.nt * G;
#pragma unroll 4
  for (int i = tid; i < 128 * MT * 16; i += 32 * kTreeProducers) {
    const int r = i >> 4, c = i & 15, row = x.mg * 128 * MT + r;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < rows) {
      const int t = row / G;
      v = ldg_nc(a.q + ((static_cast<size_t>(x.b) * a.max_tree + t) * a.hq + x.hk * G + row - t * G) * kDim + 8 * c);
    }
    sts128(st + (r >> 7) * kTreeOperand + (c >> 3) * kTreeSlab + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4), v);
  }
}

__device__ __forceinline__ void producer_arrive(uint64_t *bar, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

template <int MT, bool kF16>
__device__ __forceinline__ void tree_produce(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t q_s, uint32_t k_s,
                                             uint32_t v_s, long long w0, long long w1) {
  const int tid = threadIdx.x - 32 * TreeShape<MT>::kSoftWarps, lane = tid & 31, warp = tid >> 5;
  const int u = tid >> 7;
  constexpr int kQ = TreeSmem<MT>::kQ;
  TreeFeed<MT> feed;
  feed.walk.init(a, w0, w1, sm.start_base, sm.start_b);
  feed.walk.t1 = 0;
  feed.t = 0;
  feed.unit0 = u;
  feed.live = true;
  TreeTile cur = feed.next(a), nxt = feed.next(a);
  TreeRegs<kF16> regs;
  TreeUnit un[2];
  float2 sc[2];  // the units' scales (thread 0 of each half writes the records)
  const bool scribe = (tid & 127) == 0;

  auto is_cold = [&](const TreeTile &x) { return x.ti >= 0 && x.ti * kTK < x.cold; };
  auto units = [&](const TreeTile &x) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      un[i] = tree_unit<kF16>(a, x, i, u);
      sc[i] = kF16 ? make_float2(1.f, 1.f) : make_float2(0.f, 0.f);
      if (!kF16 && scribe && un[i].n > 0)
        sc[i] = __ldg(reinterpret_cast<const float2 *>(a.scales) + static_cast<size_t>(x.ent[i]) * a.hkv + x.hk);
    }
  };
  if (is_cold(cur)) {
    units(cur);
#pragma unroll
    for (int i = 0; i < 2; i++) load_cold_k<kF16>(un[i], tid, regs.k[i]);
#pragma unroll
    for (int i = 0; i < 2; i++) load_cold_v<kF16>(un[i], tid, regs.v[i]);
  }
  int seg = -1;
  for (int j = 0; cur.ti >= 0; j++) {
    const int s = j % kTreeStages;
    const uint32_t ph = (j / kTreeStages) & 1;
    const TreeTile nn = feed.next(a);
    if (cur.first) {
      seg++;
      if (!tree_wait_warp(sm, &sm.qempty[seg % kQ], ((seg / kQ) & 1) ^ 1, a)) return;
      load_q<MT>(a, cur, q_s + (seg % kQ) * MT * kTreeOperand, tid);
      producer_arrive(&sm.qfull[seg % kQ], lane);
    }
    const uint32_t kst = k_s + s * kTreeOperand, vst = v_s + s * kTreeOperand;
    TreeMeta &m = sm.meta[j % kTreeMeta];
    if (is_cold(cur)) {
      if (!tree_wait_warp(sm, &sm.kempty[s], ph ^ 1, a)) return;
      const bool int4[2] = {un[0].int4, un[1].int4};
      if (scribe) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
          m.k_scale[u + 2 * i] = sc[i].x;
          m.v_scale[u + 2 * i] = sc[i].y;
          m.ok[u + 2 * i] = un[i].n >= 32 ? 0xffffffffu : (1u << un[i].n) - 1;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; i++) {
        if constexpr (kF16) store_k16(kst, u + 2 * i, tid, regs.k[i]);
        else store_k8(kst, u + 2 * i, tid, int4[i], regs.k[i]);
      }
      producer_arrive(&sm.kfull[s], lane);
      if (lane == 0) mbar_arrive(&sm.mfull[j % kTreeMeta]);
      if (is_cold(nxt)) {
        units(nxt);
#pragma unroll
        for (int i = 0; i < 2; i++) load_cold_k<kF16>(un[i], tid, regs.k[i]);
      }
      if (!tree_wait_warp(sm, &sm.vempty[s], ph ^ 1, a)) return;
#pragma unroll
      for (int i = 0; i < 2; i++) {
        if constexpr (kF16) store_v16(vst, u + 2 * i, tid, regs.v[i]);
        else store_v8(vst, u + 2 * i, tid, int4[i], regs.v[i]);
      }
      producer_arrive(&sm.vfull[s], lane);
      if (is_cold(nxt)) {
#pragma unroll
        for (int i = 0; i < 2; i++) load_cold_v<kF16>(un[i], tid, regs.v[i]);
      }
    } else {
      // ring rows and nodes: at most two of a unit's tiles
      const int r0 = (cur.ti - (cur.cold + kTK - 1) / kTK) * kTK;
      uint4 tk[2][4], tv[2][4];
      uint32_t bad[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int ru = r0 + 32 * (u + 2 * i);
        const __half *row = tail_row(a, cur, ru + ((tid & 127) >> 2), 0);
        rows_k(row, row != nullptr, tid, tk[i]);
        rows_v([&](int k) { return tail_row(a, cur, ru + k, 1); }, tid, tv[i]);
        // a V that is not finite must not meet the zero weight of a row that
        // does not attend it: it becomes 0 here, and the rows that do attend
        // the node add it at the end
        uint32_t *w = reinterpret_cast<uint32_t *>(tv[i]);
#pragma unroll
        for (int k = 0; k < 16; k++) {
          const int r = 16 * ((tid >> 6) & 1) + k;
          if (ru + r < cur.hot) continue;
          const bool lo = f16_not_finite(w[k]), hi = f16_not_finite(w[k] >> 16);
          if (lo) w[k] &= 0xffff0000u;
          if (hi) w[k] &= 0x0000ffffu;
          if (lo || hi) bad[i] |= 1u << r;
        }
        bad[i] = __reduce_or_sync(0xffffffffu, bad[i]);
      }
      if (!tree_wait_warp(sm, &sm.kempty[s], ph ^ 1, a)) return;
      if (lane < 4) m.bad[warp][lane] = (lane & 1) == u ? bad[lane >> 1] : 0u;
      if (scribe) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const int n = max(0, min(32, cur.hot - (r0 + 32 * (u + 2 * i))));
          m.k_scale[u + 2 * i] = 1.f;
          m.v_scale[u + 2 * i] = 1.f;
          m.ok[u + 2 * i] = n >= 32 ? 0xffffffffu : (1u << n) - 1;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; i++) store_k16(kst, u + 2 * i, tid, tk[i]);
      producer_arrive(&sm.kfull[s], lane);
      if (lane == 0) mbar_arrive(&sm.mfull[j % kTreeMeta]);
      if (!tree_wait_warp(sm, &sm.vempty[s], ph ^ 1, a)) return;
#pragma unroll
      for (int i = 0; i < 2; i++) store_v16(vst, u + 2 * i, tid, tv[i]);
      producer_arrive(&sm.vfull[s], lane);
      if (is_cold(nxt)) {
        units(nxt);
#pragma unroll
        for (int i = 0; i < 2; i++) load_cold_k<kF16>(un[i], tid, regs.k[i]);
#pragma unroll
        for (int i = 0; i < 2; i++) load_cold_v<kF16>(un[i], tid, regs.v[i]);
      }
    }
    cur = nxt;
    nxt = nn;
  }
}

// ---- the MMA thread ----
// TMEM columns: MT 1: S buffers 0 and 128, O 256.  MT 2: S of row tile m at
// 128 m, O at 256 + 128 m.  The weights of a tile replace its S (FP16, the
// first 64 columns).

template <int MT>
__device__ __forceinline__ void tree_mma(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t q_s, uint32_t k_s, uint32_t v_s,
                                         uint32_t tmem, long long w0, long long w1) {
  constexpr uint32_t idesc = tc_idesc_f16(128);
  constexpr int kQ = TreeSmem<MT>::kQ;
  TreeWalk<MT> wq, wp;  // the walks of Q K^T (one tile ahead) and of P V
  wq.init(a, w0, w1, sm.start_base, sm.start_b);
  wp.init(a, w0, w1, sm.start_base, sm.start_b);
  const int n = static_cast<int>(w1 - w0);
  int seg_q = -1, left_q = 0, mt_q = 0, jq = 0;  // jq: tiles whose Q K^T is issued
  int used[2] = {0, 0};                          // tiles of row tile m issued (MT 2), for its barriers' phases
  int seg_o[2] = {0, 0};                         // segments of row tile m begun

  // make tile jq ready: its segment's Q and its K
  auto open = [&]() -> bool {
    if (left_q == 0) {
      wq.next(a);
      seg_q++;
      left_q = wq.t1 - wq.t0;
      mt_q = wq.m_tiles(a);
      if (!tree_wait(sm, &sm.qfull[seg_q % kQ], (seg_q / kQ) & 1, a)) return false;
    }
    return tree_wait(sm, &sm.kfull[jq % kTreeStages], (jq / kTreeStages) & 1, a);
  };
  auto qk = [&](int m) {
    tc_fence_after();
    const uint32_t q = q_s + ((seg_q % kQ) * MT + m) * kTreeOperand, k = k_s + (jq % kTreeStages) * kTreeOperand;
    const int buf = MT == 1 ? jq & 1 : m;
    const uint64_t dq = tc_desc_sw128(q), dk = tc_desc_sw128(k);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint64_t o = (i >> 2) * (kTreeSlab >> 4) + 2 * (i & 3);
      tc_mma_ss(tmem + 128 * buf, dq + o, dk + o, idesc, i > 0);
    }
    tc_commit(&sm.sfull[buf]);
  };
  auto close = [&]() {
    tc_commit(&sm.kempty[jq % kTreeStages]);
    if (--left_q == 0) tc_commit(&sm.qempty[seg_q % kQ]);
    jq++;
  };
  auto pv = [&](int j, int m, bool first) -> bool {
    const int buf = MT == 1 ? j & 1 : m;
    const uint32_t ph = MT == 1 ? (j >> 1) & 1 : used[m] & 1;
    if (first) {
      if (!tree_wait(sm, &sm.ofree[m], (seg_o[m] & 1) ^ 1, a)) return false;
      seg_o[m]++;
    }
    if (!tree_wait(sm, &sm.pfull[buf], ph, a)) return false;
    if (!tree_wait(sm, &sm.vfull[j % kTreeStages], (j / kTreeStages) & 1, a)) return false;
    tc_fence_after();
    const uint64_t dv = tc_desc_sw128(v_s + (j % kTreeStages) * kTreeOperand);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint64_t o = (i >> 2) * (kTreeSlab >> 4) + 2 * (i & 3);
      tc_mma_ts(tmem + 256 + 128 * m, tmem + 128 * buf + 8 * i, dv + o, idesc, !first || i > 0);
    }
    tc_commit(&sm.odone[m][used[m] & 1]);
    used[m]++;
    return true;
  };

  if (n > 0) {
    if (!open()) return;
    for (int m = 0; m < mt_q; m++) qk(m);
    close();
  }
  int left_p = 0, mt_p = 0;
  bool first = false;
  for (int j = 0; j < n; j++) {
    if (left_p == 0) {
      wp.next(a);
      left_p = wp.t1 - wp.t0;
      mt_p = wp.m_tiles(a);
      first = true;
    }
    const bool more = j + 1 < n;
    if (MT == 1) {
      if (more) {
        if (!open()) return;
        qk(0);
        close();
      }
      if (!pv(j, 0, first)) return;
    } else {
      // the next tile's S of a row tile follows that row tile's P V, whose
      // weights it overwrites; a row tile idle in this segment is free at once
      bool opened = false;
      for (int m = 0; m < MT; m++) {
        if (m < mt_p && !pv(j, m, first)) return;
        if (more) {
          if (!opened && !open()) return;
          opened = true;
          if (m < mt_q) qk(m);
        }
      }
      if (more) close();
    }
    tc_commit(&sm.vempty[j % kTreeStages]);
    left_p--;
    first = false;
  }
}

// ---- softmax ----

__device__ __forceinline__ float max32(const uint32_t (&v)[32]) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; k++) m[k] = __uint_as_float(v[k]);
#pragma unroll
  for (int k = 4; k < 32; k++) m[k & 3] = fmaxf(m[k & 3], __uint_as_float(v[k]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

template <int MT>
__device__ __forceinline__ void tree_softmax(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t tmem, long long w0,
                                             long long w1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt = warp >> 2, row_in = threadIdx.x & 127;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t t_o = tmem + lanes + 256 + 128 * mt;
  const int G = a.hq / a.hkv, groups_max = (a.max_tree * G + 128 * MT - 1) / (128 * MT);
  TreeWalk<MT> walk;
  walk.init(a, w0, w1, sm.start_base, sm.start_b);
  int j = 0;      // tiles of the CTA so far
  int mine = 0;   // tiles of this row tile so far
  while (walk.next(a)) {
    const int n = walk.t1 - walk.t0;
    if (MT > 1 && mt >= walk.m_tiles(a)) {
      j += n;
      continue;
    }
    const int row = walk.mg * 128 * MT + mt * 128 + row_in;
    const bool live = row < walk.s.nt * G;
    const bool warp_live = row - lane < walk.s.nt * G;
    const int t = live ? row / G : 0;
    uint64_t nodes = 0;  // nodes this row attends
    if (live && walk.s.keys > 0) {
      nodes = a.mask ? a.mask[static_cast<size_t>(walk.b) * a.max_tree + t] : (~0ull >> (63 - t));
      if (walk.s.keys < 64) nodes &= (1ull << walk.s.keys) - 1;
    }
    const int cold_tiles = (walk.s.cold + kTK - 1) / kTK;
    float m = -INFINITY, l = 0.f, ref = 1.f;
    uint64_t odd = 0;    // attended nodes whose V is not finite
    for (int ti = walk.t0; ti < walk.t1; ti++, j++, mine++) {
      const int buf = MT == 1 ? mine & 1 : mt;
      const uint32_t ph = MT == 1 ? (mine >> 1) & 1 : mine & 1;
      const uint32_t t_s = tmem + lanes + 128 * buf;
      // (a row tile that sat out a segment may have missed phases of mfull: S
      // first, whose phases are its own)
      if (!tree_wait_warp(sm, &sm.sfull[buf], ph, a)) return;
      if (!tree_wait_warp(sm, &sm.mfull[j % kTreeMeta], (j / kTreeMeta) & 1, a)) return;
      tc_fence_after();
      if (warp_live) {
        const TreeMeta &me = sm.meta[j % kTreeMeta];
        uint32_t ok[4];
#pragma unroll
        for (int c = 0; c < 4; c++) ok[c] = me.ok[c];
        if (ti >= cold_tiles) {
          const int r0 = (ti - cold_tiles) * kTK - walk.s.hot;  // first row of the tile, as a node
#pragma unroll
          for (int c = 0; c < 4; c++) {
            const int k = r0 + 32 * c;  // node of the unit's first key
            uint32_t own = 0;
            if (k >= 0) own = k < 64 ? static_cast<uint32_t>(nodes >> k) : 0u;
            else if (k > -32) own = static_cast<uint32_t>(nodes << -k);
            ok[c] |= own;
            uint32_t bad = 0;
#pragma unroll
            for (int w = 0; w < kTreeProducers; w++) bad |= me.bad[w][c];
            bad &= own;
            if (bad) odd |= k >= 0 ? static_cast<uint64_t>(bad) << k : static_cast<uint64_t>(bad) >> -k;
          }
        }
        float ks[4], vs[4];
        float vmax = 0.f;
#pragma unroll
        for (int c = 0; c < 4; c++) {
          ks[c] = me.k_scale[c] * a.qk_scale;
          vs[c] = me.v_scale[c];
          vmax = fmaxf(vmax, fabsf(vs[c]));
        }
        const bool full = __all_sync(0xffffffffu, (ok[0] & ok[1] & ok[2] & ok[3]) == 0xffffffffu);
        // the tile's maximum
        float top = -INFINITY;
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 4; c++) {
          tc_ld32(t_s + 32 * c, v);
          tc_wait_ld(v);
          if (!full || ks[c] < 0.f) {
#pragma unroll
            for (int k = 0; k < 32; k++) {
              const float z = __uint_as_float(v[k]) * ks[c];
              top = fmaxf(top, ok[c] >> k & 1 ? z : -INFINITY);
            }
          } else {
            top = fmaxf(top, max32(v) * ks[c]);
          }
        }
        // m and r follow when they lag too far behind; O and l follow them
        const bool first = ti == walk.t0;
        float r_new = ref;
        if (first || vmax > kLagScale * ref) r_new = vmax > 0.f ? vmax : ref;
        const bool move = first || top > m + kLagLog2;
        const float m_new = move ? fmaxf(m, top) : m;
        if (!first && __any_sync(0xffffffffu, m_new != m || r_new != ref)) {
          if (!tree_wait_warp(sm, &sm.odone[mt][(mine - 1) & 1], ((mine - 1) >> 1) & 1, a)) return;
          tc_fence_after();
          const float f = m == -INFINITY ? 0.f : ex2(m - m_new);
          l *= f;
          const float g = f * __fdividef(ref, r_new);
#pragma unroll
          for (int c = 0; c < 4; c++) {
            tc_ld32(t_o + 32 * c, v);
            tc_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 32; k++) v[k] = __float_as_uint(__uint_as_float(v[k]) * g);
            tc_st32(t_o + 32 * c, v);
          }
        }
        m = m_new;
        ref = r_new;
        const float base = m == -INFINITY ? 0.f : m;
        const float inv = __fdividef(1.f, ref);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; c++) {
          tc_ld32(t_s + 32 * c, v);
          tc_wait_ld(v);
          const float f = vs[c] * inv;
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float x = ex2(fmaf(__uint_as_float(v[k]), ks[c], -base));
            float y = ex2(fmaf(__uint_as_float(v[k + 1]), ks[c], -base));
            if (!full) {
              x = ok[c] >> k & 1 ? x : 0.f;
              y = ok[c] >> (k + 1) & 1 ? y : 0.f;
            }
            sum[(k >> 1) & 3] += x + y;
            const __half2 h = __floats2half2_rn(x * f, y * f);
            p[k >> 1] = *reinterpret_cast<const uint32_t *>(&h);
          }
          tc_st16(t_s + 16 * c, p);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tc_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.pfull[buf]);
    }
    // the segment's end: O of the last tile
    if (!tree_wait_warp(sm, &sm.odone[mt][(mine - 1) & 1], ((mine - 1) >> 1) & 1, a)) return;
    tc_fence_after();
    if (warp_live) {
      const bool whole = walk.t0 == 0 && walk.t1 == walk.s.tiles;
      const float o_scale = whole ? (l != 0.f ? ref / l : 0.f) : ref;
      const int hq = walk.hk * G + row - t * G;
      const size_t out_row = (static_cast<size_t>(walk.b) * a.max_tree + t) * a.hq + hq;
      const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (walk.t0 == 0 ? 1 : 0);
      const int pr = mt * 128 + row_in;
#pragma unroll 1
      for (int c = 0; c < 4; c++) {
        uint32_t v[32];
        tc_ld32(t_o + 32 * c, v);
        tc_wait_ld(v);
        float o[32];
#pragma unroll
        for (int k = 0; k < 32; k++) o[k] = (l != 0.f ? __uint_as_float(v[k]) : 0.f) * o_scale;
        if (odd) {
          for (uint64_t rest = odd; rest; rest &= rest - 1) {
            const int node = __ffsll(static_cast<long long>(rest)) - 1;
            const __half *vr = a.v_tree + ((static_cast<size_t>(walk.b) * a.max_tree + node) * a.hkv + walk.hk) * kDim;
#pragma unroll
            for (int k = 0; k < 32; k++) {
              const __half h = vr[32 * c + k];
              if (f16_not_finite(__half_as_ushort(h))) o[k] += __half2float(h);
            }
          }
        }
        if (!live) continue;
        if (whole) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const __half2 x = __floats2half2_rn(o[k + 2 * e], o[k + 2 * e + 1]);
              h[e] = *reinterpret_cast<const uint32_t *>(&x);
            }
            *reinterpret_cast<uint4 *>(a.out + out_row * kDim + 32 * c + k) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        } else {
          float4 *dst = reinterpret_cast<float4 *>(a.part_o) + slot * 32 * 128 * MT;
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            dst[(8 * c + (k >> 2)) * (128 * MT) + pr] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
      }
      if (live) {
        if (whole) {
          if (a.lse_out) a.lse_out[out_row] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
        } else {
          float2 *ml = reinterpret_cast<float2 *>(a.part_ml) + slot * 128 * MT;
          ml[pr] = make_float2(m, l);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.ofree[mt]);
    // who has the unit's tiles, from the CTA with its first
    if (threadIdx.x == 0 && walk.t0 == 0) {
      const long long ctas = min(static_cast<long long>(a.ctas), sm.total);
      const long long u0 = walk.w - walk.t1;  // the list's index of the unit's first tile
      const int last = static_cast<int>(((u0 + walk.s.tiles) * ctas - 1) / sm.total);
      a.unit_ctas[(static_cast<size_t>(walk.b) * a.hkv + walk.hk) * groups_max + walk.mg] =
          make_int2(static_cast<int>(blockIdx.x), last);
    }
  }
}

template <int MT, bool kF16>
__global__ void __launch_bounds__(TreeShape<MT>::kThreads, 1) tree_kernel(const __grid_constant__ TreeArgs a) {
  using Shape = TreeShape<MT>;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const uint32_t q_s = base, k_s = q_s + Shape::kQBytes, v_s = k_s + kTreeStages * kTreeOperand;
  TreeSmem<MT> &sm = *reinterpret_cast<TreeSmem<MT> *>(raw + (base - smem_addr(raw)) + Shape::kQBytes +
                                                       2 * kTreeStages * kTreeOperand);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge waits for this grid's end
  constexpr int kMmaWarp = Shape::kSoftWarps + kTreeProducers;

  // the list's length and where this CTA's run starts: every thread sums a
  // range of sequences, a scan over the threads places them
  const int per = (a.batch + Shape::kThreads - 1) / Shape::kThreads;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; b++) {
    const TreeSeq s = tree_seq<MT>(a, b);
    mine += s.span;
    if (blockIdx.x == 0 && s.status) set_status(a.status, s.status);
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sm.warp_sum[warp] = inc;
  if (tid == 0) {
    sm.abort = 0;
    for (int i = 0; i < kTreeStages; i++) {
      mbar_init(&sm.kfull[i], kTreeProducers);
      mbar_init(&sm.kempty[i], 1);
      mbar_init(&sm.vfull[i], kTreeProducers);
      mbar_init(&sm.vempty[i], 1);
    }
    for (int i = 0; i < kTreeMeta; i++) mbar_init(&sm.mfull[i], kTreeProducers);
    for (int i = 0; i < TreeSmem<MT>::kQ; i++) {
      mbar_init(&sm.qfull[i], kTreeProducers);
      mbar_init(&sm.qempty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.pfull[i], 4);
      mbar_init(&sm.odone[i][0], 1);
      mbar_init(&sm.odone[i][1], 1);
      mbar_init(&sm.ofree[i], 4);
    }
    mbar_init(&sm.drain, 1);
    mbar_fence_init();
  }
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w <= kMmaWarp; w++) {
    const long long v = sm.warp_sum[w];
    if (w < warp) before += v;
    total += v;
  }
  const long long ctas = min(static_cast<long long>(gridDim.x), total);
  if (static_cast<long long>(blockIdx.x) >= ctas) return;  // the whole CTA: nothing to do
  const long long w0 = total * blockIdx.x / ctas, w1 = total * (blockIdx.x + 1) / ctas;
  long long at = before + inc - mine;
  if (w0 >= at && w0 < at + mine) {
    for (int b = b0; b < b1; b++) {
      const long long span = tree_seq<MT>(a, b).span;
      if (w0 < at + span) {
        sm.start_b = b;
        sm.start_base = at;
        sm.total = total;
        break;
      }
      at += span;
    }
  }
  if (warp == kMmaWarp) tc_alloc(&sm.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp < Shape::kSoftWarps) {
    tree_softmax<MT>(a, sm, tmem, w0, w1);
  } else if (warp < kMmaWarp) {
    tree_produce<MT, kF16>(a, sm, q_s, k_s, v_s, w0, w1);
  } else {
    if (lane == 0) {
      tree_mma<MT>(a, sm, q_s, k_s, v_s, tmem, w0, w1);
      // no MMA is in flight when TMEM is given back
      tc_commit(&sm.drain);
      if (!mbar_wait_bounded(&sm.drain, 0, kDefaultWaitCycles)) set_status(a.status, HYB_STATUS_TIMEOUT);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tc_dealloc(tmem, 512);
}

// ---- the merge of units that several CTAs share ----
// CTA = (unit, 32 rows): thread = row (lane) and 16 channels (warp); parts in
// the order of the tiles.
template <int MT>
__global__ void __launch_bounds__(256) tree_combine_kernel(const __grid_constant__ TreeArgs a, int groups_max) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int unit = blockIdx.x;
  const int mg = unit % groups_max, hk = unit / groups_max % a.hkv, b = unit / groups_max / a.hkv;
  const int G = a.hq / a.hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nt = a.n_tree ? a.n_tree[b] : a.max_tree;
  if (nt < 0 || nt > a.max_tree) return;
  const int r = 32 * blockIdx.y + lane, row = mg * 128 * MT + r;
  if (row - lane >= nt * G) return;
  const int2 c = a.unit_ctas[unit];
  // (out of range: a call that gave up before it wrote them)
  if (c.x < 0 || c.x >= c.y || c.y >= a.ctas || row >= nt * G) return;
  const int t = row / G;
  const size_t out_row = (static_cast<size_t>(b) * a.max_tree + t) * a.hq + hk * G + row - t * G;
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
  const float4 *po = reinterpret_cast<const float4 *>(a.part_o);
  float top = -INFINITY;
  for (int i = c.x; i <= c.y; i++) top = fmaxf(top, ml[(2 * static_cast<size_t>(i) + (i == c.x)) * 128 * MT + r].x);
  float sum = 0.f;
  float4 o[4];
#pragma unroll
  for (int k = 0; k < 4; k++) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = c.x; i <= c.y; i++) {
    const size_t slot = 2 * static_cast<size_t>(i) + (i == c.x);
    const float2 x = ml[slot * 128 * MT + r];
    const float w = x.x == top ? 1.f : ex2(x.x - top);
    if (x.y == 0.f || w == 0.f) continue;
    sum = fmaf(w, x.y, sum);
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float4 y = po[(slot * 32 + 4 * warp + k) * 128 * MT + r];
      o[k].x = fmaf(w, y.x, o[k].x);
      o[k].y = fmaf(w, y.y, o[k].y);
      o[k].z = fmaf(w, y.z, o[k].z);
      o[k].w = fmaf(w, y.w, o[k].w);
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  uint32_t h[8];
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const __half2 x = __floats2half2_rn(o[k].x * inv, o[k].y * inv), y = __floats2half2_rn(o[k].z * inv, o[k].w * inv);
    h[2 * k] = *reinterpret_cast<const uint32_t *>(&x);
    h[2 * k + 1] = *reinterpret_cast<const uint32_t *>(&y);
  }
  uint4 *dst = reinterpret_cast<uint4 *>(a.out + out_row * kDim + 16 * warp);
  dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
  dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
  if (warp == 0 && a.lse_out) a.lse_out[out_row] = sum != 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

template <int MT, bool kF16>
static cudaError_t launch_tree(const TreeArgs &a, cudaStream_t stream) {
  using Shape = TreeShape<MT>;
  static int configured_dev_mask = 0;  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 31 || !(configured_dev_mask & (1 << dev))) {
    e = cudaFuncSetAttribute(tree_kernel<MT, kF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(Shape::kBytes));
    if (e != cudaSuccess) return e;
    if (dev < 31) configured_dev_mask |= 1 << dev;
  }
  tree_kernel<MT, kF16><<<a.ctas, Shape::kThreads, Shape::kBytes, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int G = a.hq / a.hkv, groups = tree_groups(a.max_tree, G);
  const int rows = a.max_tree * G < 128 * MT ? a.max_tree * G : 128 * MT;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch * a.hkv * groups, (rows + 31) / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_combine_kernel<MT>, a, groups);
}

cudaError_t launch_tree_attn(const TreeArgs &a, cudaStream_t stream) {
  const bool two = tree_m_tiles(a.max_tree, a.hq / a.hkv) == 2;
  if (a.quant_bits == 0) return two ? launch_tree<2, true>(a, stream) : launch_tree<1, true>(a, stream);
  return two ? launch_tree<2, false>(a, stream) : launch_tree<1, false>(a, stream);
}

}  // namespace hyb
