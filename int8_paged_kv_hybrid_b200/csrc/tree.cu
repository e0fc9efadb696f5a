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
// Inside a CTA (18 warps): a scout warp looks the tiles up (block table, scales,
// segment ends) some tiles ahead, writes their records and starts their way
// into L2; two groups of four producer warps take turns at the tiles and bring
// codes or rows to FP16 in the 128-byte swizzled layout of the
// MMA's shared operands; one thread issues the MMAs; two groups of four softmax
// warps (one query row per thread) keep two softmax streams and write the
// weights back over the logits in TMEM, where the second product reads them as
// its A operand.  The streams are the two row tiles (MT 2), or the even and the
// odd tiles of the run (MT 1), which are merged at a unit's end: either way a
// stream's softmax has the time of two tiles' MMAs.
#include "kernels.cuh"
#include "spec.cuh"
#include "tc05.cuh"

namespace hyb {

constexpr int kTK = 128;                     // keys per tile
constexpr int kTreeStages = 2;               // K and V tiles in shared memory
constexpr int kTreeBatch = 4;                // tiles the scout looks up at once
constexpr int kTreeRecs = 2 * kTreeBatch;    // tile records
constexpr uint32_t kTreeOperand = 128 * 256; // bytes of a 128 x 128 FP16 operand
constexpr uint32_t kTreeSlab = kTreeOperand / 2;  // its halves of 64 columns
constexpr float kLagLog2 = 6.f;
constexpr float kLagScale = 256.f;

// Warps: softmax, producers, MMA, scout.  A launch gives every thread 96
// registers (65536 / 20 warps); the producers, which hold a tile's codes, take 8
// of each softmax thread's.
constexpr int kTreeSoft = 8, kTreeProd = 8, kTreeGroups = 2;
constexpr int kTreeThreads = 32 * (kTreeSoft + kTreeProd + 2);
constexpr int kTreeSoftRegs = 88, kTreeProdRegs = 104;

// TreeRec::flags: the first, the second and the last tile of its segment; every
// key attended by every row and no negative scale; cold (not ring and nodes);
// the unit's row tiles; the segment's number modulo 4
constexpr uint32_t kTileFirst = 1, kTileSecond = 2, kTileLast = 4, kTilePlain = 8, kTileCold = 16;
constexpr int kTileRowsShift = 5, kTileSegShift = 7;

// A tile of 128 keys in four units of 32, as the scout found it.
struct TreeRec {
  const uint8_t *at[4];  // cold: the unit's 64-token tile pair (FP16: its first row); null: no keys
  float k_scale[4];      // 1 for FP16 rows
  float v_scale[4];
  uint32_t ok[4];        // keys that every row attends
  uint32_t bad[4][4];    // [warp][unit]: rows of a tail tile with a V that is not finite (by the producers)
  uint32_t fmt;          // bit c: unit c is INT4; bit 4 + c: it is the second half of its slots
  uint32_t flags;
  float v_max;           // largest |v_scale|
  int b, hk, mg;         // the unit's sequence, kv head and row group
  int cold, hot, keys;   // tail: cold and ring tokens, nodes
  int row0;              // tail: its first row (ring rows, then nodes)
};

// A stream's row at a segment's end (MT 1).
struct TreeStat {
  float m, l, ref;
  uint64_t odd;
};

template <int MT>
struct TreeSmem {
  static constexpr int kQ = MT == 1 ? 2 : 1;  // Q buffers
  uint64_t kfull[kTreeStages], kempty[kTreeStages], vfull[kTreeStages], vempty[kTreeStages];
  uint64_t rfull[2], rfree[2];  // records, by batch parity
  uint64_t mfull[kTreeRecs];    // a record's tile is in shared memory
  uint64_t qfull[kQ], qempty[kQ];
  uint64_t sfull[2], pfull[2], odone[2];  // by stream
  uint64_t ofree[2];                      // by stream (MT 1: one for both)
  uint64_t xfull;                         // MT 1: the streams' rows are in `stat`
  uint64_t drain;
  TreeRec rec[kTreeRecs];
  uint32_t tmem;
  volatile int abort;
  int start_b;
  long long start_pos, total;  // the run's start within sequence start_b, the list's length
  long long warp_sum[32];
  TreeStat stat[MT == 1 ? 2 : 1][MT == 1 ? 2 : 1][MT == 1 ? 128 : 1];  // [segment parity][stream][row]
};

template <int MT>
struct TreeShape {
  static constexpr uint32_t kQBytes = TreeSmem<MT>::kQ * MT * kTreeOperand;
  static constexpr uint32_t kBytes = 1024 + kQBytes + 2 * kTreeStages * kTreeOperand + sizeof(TreeSmem<MT>);
};

// ---- the list of tiles ----

struct TreeSeq {
  int cold, hot, nt, keys;  // cold and ring tokens, nodes (rows), nodes that are keys
  int tiles, groups;        // per unit; row groups
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
  return s;
}

// A run of `left` tiles from tile `pos` of sequence b on, taken unit by unit.
template <int MT>
struct TreeWalk {
  long long pos;
  int left, b;
  int cold, tiles, groups, nt;
  int hk, mg, t0, t1;  // the current segment: tiles [t0, t1) of unit (b, hk, mg)

  __device__ __forceinline__ void enter(const TreeArgs &a) {
    const TreeSeq s = tree_seq<MT>(a, b);
    cold = s.cold;
    tiles = s.tiles;
    groups = s.groups;
    nt = s.nt;
  }
  __device__ __forceinline__ bool next(const TreeArgs &a) {
    if (left == 0) return false;
    for (;;) {
      const long long span = static_cast<long long>(tiles) * groups * a.hkv;
      if (pos < span) break;
      pos -= span;
      b++;
      enter(a);
    }
    const int unit = static_cast<int>(pos / tiles);
    t0 = static_cast<int>(pos - static_cast<long long>(unit) * tiles);
    t1 = min(tiles, t0 + left);
    hk = unit / groups;
    mg = unit - hk * groups;
    pos += t1 - t0;
    left -= t1 - t0;
    return true;
  }
  // 128-row tiles of this unit that have a row
  __device__ __forceinline__ int m_tiles(const TreeArgs &a) const {
    return MT == 1 ? 1 : min(MT, (nt * (a.hq / a.hkv) - mg * 128 * MT + 127) / 128);
  }
};

// Wait for phase `parity`; false when the wait or the kernel gave up.
template <typename Sm>
__device__ __forceinline__ bool tree_wait(Sm &sm, uint64_t *bar, uint32_t parity, const TreeArgs &a) {
  const bool quick = a.wait_cycles < kShortWaitCycles;
  const uint32_t t0 = static_cast<uint32_t>(clock());
  while (!(quick ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
    if (sm.abort) return false;
    if (static_cast<uint32_t>(clock()) - t0 > a.wait_cycles) {
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

// A thread of a producer group has a part of each of a tile's four units of 32
// keys: K of key tid / 4, 32 channels; V of INT8 / INT4 channel tid, all 32
// keys, of FP16 rows channels 2 (tid % 64), + 1 and 16 keys.

// [p, p + bytes) on its way into L2; 16-byte aligned.
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Codes are read once: no place in L1.
__device__ __forceinline__ uint4 ldg16(const void *p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ void ldg32(const void *p, uint4 &x, uint4 &y) {  // 32-byte aligned
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w), "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
               : "l"(p));
}

// Codes of a unit: the thread's 32 bytes (INT4: 16) of K or V of the 64-token
// tile pair at `pair` that holds the unit as slots 32 half ...
__device__ __forceinline__ void load_codes(const TreeArgs &a, const uint8_t *p, uint4 (&r)[2]) {
  if (a.wide) {
    ldg32(p, r[0], r[1]);
  } else {
    r[0] = ldg16(p);
    r[1] = ldg16(p + 16);
  }
}

__device__ __forceinline__ void load_k(const TreeArgs &a, const uint8_t *pair, int half, bool int4, int tid, uint4 (&k)[2]) {
  const int slot = 32 * half + (tid >> 2);
  if (int4) k[0] = ldg16(pair + slot * 64 + 16 * (tid & 3));
  else load_codes(a, pair + slot * 128 + 32 * (tid & 3), k);
}

// (V: the unit's two 16-slot chunks are one aligned pair, swapped where the
// swizzle's lowest bit is set; store_v8 puts them right)
__device__ __forceinline__ void load_v(const TreeArgs &a, const uint8_t *pair, int half, bool int4, int tid, uint4 (&v)[2]) {
  const uint8_t *t = pair + kTileBytes;
  if (int4) v[0] = ldg16(t + tid * 32 + 8 * ((2 * half) ^ ((tid >> 2) & 2)));
  else load_codes(a, t + tid * 64 + 16 * ((2 * half) ^ ((tid >> 1) & 2)), v);
}

// K of one unit into the operand: row = key, 32 channels = four 16-byte chunks
// of a 64-channel slab.  Eight lanes are two rows of four threads; threads 2
// and 3 of a row write their chunks in the order k ^ 2, which spreads the
// eight over the banks.
__device__ __forceinline__ void store_k16(uint32_t st, int u, int tid, const uint4 (&k)[4]) {
  const int row = 32 * u + (tid >> 2), i = tid & 3;
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
  const int row = tid;
  const uint32_t base = st + (u >> 1) * kTreeSlab + row * 128;
  const int c = 4 * (u & 1);
  if (int4) {
    // the swap, as a bit of the chunk
    const int x = (row & 7) ^ ((row >> 2 & 1) << 1);
    sts128(base + (((c + 0) ^ x) << 4), f16_int4(v[0].x));
    sts128(base + (((c + 1) ^ x) << 4), f16_int4(v[0].y));
    sts128(base + (((c + 2) ^ x) << 4), f16_int4(v[0].z));
    sts128(base + (((c + 3) ^ x) << 4), f16_int4(v[0].w));
  } else {
    // (here that would leave eight rows four places: the words swap)
    const int x = row & 7;
    const bool swap = row & 2;
    const uint4 y = swap ? v[1] : v[0], z = swap ? v[0] : v[1];
    sts128(base + (((c + 0) ^ x) << 4), f16_int8(y.x, y.y));
    sts128(base + (((c + 1) ^ x) << 4), f16_int8(y.z, y.w));
    sts128(base + (((c + 2) ^ x) << 4), f16_int8(z.x, z.y));
    sts128(base + (((c + 3) ^ x) << 4), f16_int8(z.z, z.w));
  }
}

// FP16 V of one unit: the thread's two channels are two rows, its 16 keys two
// chunks of each.  Lanes 4..7 of eight write their odd row first, so that the
// eight rows differ modulo 8.
__device__ __forceinline__ void store_v16(uint32_t st, int u, int tid, const uint32_t (&w)[16]) {
  const int p = tid & 63, odd = (p >> 2) & 1;
  const int c0 = 4 * (u & 1) + 2 * (tid >> 6);
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

// FP16 rows as units: the rows of an FP16 cold block, or of the tail (the
// ring's in the order of their positions, then the nodes).
struct TreeRows {
  const TreeRec *rec;
  const __half *base;  // cold rows; null: the tail
  int n, r0;           // valid cold rows; the unit's first tail row

  __device__ __forceinline__ TreeRows(const TreeRec &r, int c) : rec(&r) {
    const bool cold = r.flags & kTileCold;
    base = cold ? reinterpret_cast<const __half *>(r.at[c]) : nullptr;
    n = cold ? __popc(r.ok[c]) : -1;
    r0 = r.row0 + 32 * c;
  }
  // the K row (kv 1: V row) of key k of the unit, or null
  __device__ __forceinline__ const __half *row(const TreeArgs &a, int k, int kv) const {
    if (n >= 0) return k < n ? base + (2 * k + kv) * kDim : nullptr;
    int r = r0 + k;
    if (r < rec->hot)
      return reinterpret_cast<const __half *>(a.hot) + (((static_cast<size_t>(rec->b) * a.hkv + rec->hk) * a.hot_tokens +
                                                         ((rec->cold + r) & (a.hot_tokens - 1))) * 2 + kv) * kDim;
    r -= rec->hot;
    if (r >= rec->keys) return nullptr;
    return (kv ? a.v_tree : a.k_tree) + ((static_cast<size_t>(rec->b) * a.max_tree + r) * a.hkv + rec->hk) * kDim;
  }
};

__device__ __forceinline__ void rows_k(const TreeArgs &a, const TreeRows &x, int tid, uint4 (&k)[4]) {
  const __half *row = x.row(a, tid >> 2, 0);
#pragma unroll
  for (int j = 0; j < 4; j++) k[j] = row ? ldg16(row + 32 * (tid & 3) + 8 * j) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ void rows_v(const TreeArgs &a, const TreeRows &x, int tid, uint32_t (&w)[16]) {
  const int k0 = 16 * (tid >> 6), c = 2 * (tid & 63);
#pragma unroll
  for (int j = 0; j < 16; j++) {
    const __half *r = x.row(a, k0 + j, 1);
    w[j] = r ? __ldg(reinterpret_cast<const uint32_t *>(r + c)) : 0u;
  }
}

// The query rows of a unit into its Q operand(s); rows beyond the tree are 0.
template <int MT>
__device__ __forceinline__ void load_q(const TreeArgs &a, const TreeRec &x, uint32_t st, int tid) {
  const int G = a.hq / a.hkv, mg = x.mg;
  const int rows = (a.n_tree ? a.n_tree[x.b] : a.max_tree) * G;
#pragma unroll 4
  for (int i = tid; i < 128 * MT * 16; i += 128) {
    const int r = i >> 4, c = i & 15, row = mg * 128 * MT + r;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < rows) {
      const int t = row / G;
      v = ldg16(a.q + ((static_cast<size_t>(x.b) * a.max_tree + t) * a.hq + x.hk * G + row - t * G) * kDim + 8 * c);
    }
    sts128(st + (r >> 7) * kTreeOperand + (c >> 3) * kTreeSlab + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4), v);
  }
}

// (The MMA thread orders these writes before its MMAs with one proxy fence: a
// fence here would wait for the thread's loads in flight.)
__device__ __forceinline__ void producer_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

template <int MT, bool kF16>
__device__ __forceinline__ void tree_produce(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t q_s, uint32_t k_s,
                                             uint32_t v_s, int n) {
  const int tid = threadIdx.x & 127, lane = tid & 31, group = (threadIdx.x >> 7) & 1;
  constexpr int kQ = TreeSmem<MT>::kQ;
  // a group's tiles have one stage of their own
  static_assert(kTreeStages == kTreeGroups, "one stage per producer group");
  const uint32_t kst = k_s + group * kTreeOperand, vst = v_s + group * kTreeOperand;
  uint4 rk[4][2], rv[4][2];  // the codes of the group's next tile
  uint32_t fmt = 0;

  // one round per tile of the group, and one before the first that only loads
  for (int j = group - kTreeGroups; j < n; j += kTreeGroups) {
    const uint32_t ph = (j / kTreeStages) & 1;
    if (j >= 0) {
      TreeRec &r = sm.rec[j & (kTreeRecs - 1)];
      const uint32_t flags = r.flags;
      if (flags & kTileFirst) {
        const uint32_t seg = flags >> kTileSegShift;
        if (!tree_wait_warp(sm, &sm.qempty[seg % kQ], ((seg / kQ) & 1) ^ 1, a)) return;
        load_q<MT>(a, r, q_s + (seg % kQ) * MT * kTreeOperand, tid);
        producer_arrive(&sm.qfull[seg % kQ], lane);
      }
      if (!tree_wait_warp(sm, &sm.kempty[group], ph ^ 1, a)) return;
      if (kF16 || !(flags & kTileCold)) {
        // FP16 rows.  V first: the record names the nodes whose V is not
        // finite.  Such a value must not meet the zero weight of a row that
        // does not attend its node: it becomes 0 here, and the rows that do
        // attend the node add it at the end
        if (!tree_wait_warp(sm, &sm.vempty[group], ph ^ 1, a)) return;
#pragma unroll
        for (int c = 0; c < 4; c++) {
          const TreeRows x(r, c);
          uint32_t w[16];
          rows_v(a, x, tid, w);
          if (!kF16 || x.n < 0) {
            const int k0 = 16 * (tid >> 6);
            uint32_t b = 0;
#pragma unroll
            for (int k = 0; k < 16; k++) {
              const bool lo = f16_not_finite(w[k]), hi = f16_not_finite(w[k] >> 16);
              if ((lo || hi) && x.r0 + k0 + k >= r.hot) {
                if (lo) w[k] &= 0xffff0000u;
                if (hi) w[k] &= 0x0000ffffu;
                b |= 1u << (k0 + k);
              }
            }
            b = __reduce_or_sync(0xffffffffu, b);
            if (lane == 0) r.bad[tid >> 5][c] = b;
          }
          store_v16(vst, c, tid, w);
        }
        producer_arrive(&sm.vfull[group], lane);
#pragma unroll
        for (int c = 0; c < 4; c++) {
          uint4 k[4];
          rows_k(a, TreeRows(r, c), tid, k);
          store_k16(kst, c, tid, k);
        }
        producer_arrive(&sm.kfull[group], lane);
        if (lane == 0) mbar_arrive(&sm.mfull[j & (kTreeRecs - 1)]);
      } else if constexpr (!kF16) {
#pragma unroll
        for (int c = 0; c < 4; c++) store_k8(kst, c, tid, fmt >> c & 1, rk[c]);
        producer_arrive(&sm.kfull[group], lane);
        if (lane == 0) mbar_arrive(&sm.mfull[j & (kTreeRecs - 1)]);
        if (!tree_wait_warp(sm, &sm.vempty[group], ph ^ 1, a)) return;
#pragma unroll
        for (int c = 0; c < 4; c++) store_v8(vst, c, tid, fmt >> c & 1, rv[c]);
        producer_arrive(&sm.vfull[group], lane);
      }
    }
    // the group's next tile: its codes have the time of two tiles to come
    const int next = j + kTreeGroups;
    if (next >= n) break;
    if (next % kTreeBatch < kTreeGroups) {
      const int batch = next / kTreeBatch;
      if (!tree_wait_warp(sm, &sm.rfull[batch & 1], (batch >> 1) & 1, a)) return;
    }
    const TreeRec &r = sm.rec[next & (kTreeRecs - 1)];
    if (!kF16) {
      const bool cold = r.flags & kTileCold;
      fmt = r.fmt;
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const uint8_t *pair = cold ? r.at[c] : nullptr;
        if (pair) {
          load_k(a, pair, fmt >> (4 + c) & 1, fmt >> c & 1, tid, rk[c]);
          load_v(a, pair, fmt >> (4 + c) & 1, fmt >> c & 1, tid, rv[c]);
        } else {  // code 0
          rk[c][0] = rk[c][1] = rv[c][0] = rv[c][1] = make_uint4(0, 0, 0, 0);
        }
      }
    }
  }
}

// ---- the scout ----
// Lane 4 k + c looks up unit c of tile k of a batch.
template <int MT, bool kF16>
__device__ __forceinline__ void tree_scout(const TreeArgs &a, TreeSmem<MT> &sm, int n) {
  const int lane = threadIdx.x & 31, k = (lane >> 2) & (kTreeBatch - 1), c = lane & 3;
  const bool on = lane < 4 * kTreeBatch;
  int b = sm.start_b, segs = 0;     // segments begun before the batch
  TreeSeq q = tree_seq<MT>(a, b);
  long long pos = sm.start_pos + k; // the lane's tile within sequence b
  for (int j0 = 0, batch = 0; j0 < n; j0 += kTreeBatch, batch++) {
    const int j = j0 + k;
    const bool have = on && j < n;
    int unit = 0, t = 0;
    if (have) {
      for (;;) {
        const long long span = static_cast<long long>(q.tiles) * q.groups * a.hkv;
        if (pos < span) break;
        pos -= span;
        q = tree_seq<MT>(a, ++b);
      }
      unit = static_cast<int>(pos / q.tiles);
      t = static_cast<int>(pos - static_cast<long long>(unit) * q.tiles);
    }
    const int in = min(t, j);  // tiles of the segment before this one
    const uint32_t firsts = __ballot_sync(0xffffffffu, have && in == 0 && c == 0);
    const int seg = segs + __popc(firsts & (0xffffffffu >> (31 - (4 * k)))) - 1;
    segs += __popc(firsts);
    const int hk = unit / q.groups, mg = unit - hk * q.groups;
    const int p = t * kTK + 32 * c;  // the unit's first position
    const bool cold = t * kTK < q.cold;
    int valid = cold ? max(0, min(32, q.cold - p)) : 0;
    const uint8_t *at = nullptr;
    float2 sc = make_float2(1.f, 1.f);
    uint32_t fmt = 0;
    const int block = p >> a.bshift, slot = p & ((1 << a.bshift) - 1);
    if (have && valid > 0) {
      const int phys = __ldg(a.block_table + static_cast<size_t>(b) * a.max_blocks + block);
      if (phys < 0 || phys >= a.num_phys) {
        set_status(a.status, HYB_STATUS_BAD_BLOCK);
        valid = 0;
      } else {
        const size_t i = static_cast<size_t>(phys) * a.hkv + hk;
        if (kF16) {
          at = a.cold + ((i << a.bshift) + slot) * kHotTokenBytes;
          prefetch_l2(at, 32 * kHotTokenBytes);
        } else {
          at = a.cold + ((i << a.lsub) + (slot >> 6)) * kTilePairBytes;
          if (a.quant_bits == 4 || (a.n_int4 != nullptr && block < a.n_int4[b])) fmt |= 1;
          if (slot & 32) fmt |= 16;
          sc = __ldg(reinterpret_cast<const float2 *>(a.scales) + i);
          if (!(slot & 32)) {  // the unit with the first slots brings the tile pair
            if (fmt & 1) {
              prefetch_l2(at, kTileBytes / 2);
              prefetch_l2(at + kTileBytes, kTileBytes / 2);
            } else {
              prefetch_l2(at, kTilePairBytes);
            }
          }
        }
      }
    }
    // (an empty unit has no say in the reference scale)
    if (!kF16 && cold && valid == 0) sc = make_float2(0.f, 0.f);
    const int row0 = (t - (q.cold + kTK - 1) / kTK) * kTK;
    if (!cold) valid = max(0, min(32, q.hot - row0 - 32 * c));
    const uint32_t ok = valid >= 32 ? 0xffffffffu : (1u << valid) - 1;
    bool plain = valid >= 32 && sc.x * a.qk_scale >= 0.f;
    float v_max = fabsf(sc.y);
    fmt <<= c;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      plain = __shfl_xor_sync(0xffffffffu, plain, o) && plain;
      v_max = fmaxf(v_max, __shfl_xor_sync(0xffffffffu, v_max, o));
      fmt |= __shfl_xor_sync(0xffffffffu, fmt, o);
    }
    if (!tree_wait_warp(sm, &sm.rfree[batch & 1], ((batch >> 1) & 1) ^ 1, a)) return;
    if (have) {
      TreeRec &r = sm.rec[j & (kTreeRecs - 1)];
      r.at[c] = at;
      r.k_scale[c] = sc.x;
      r.v_scale[c] = sc.y;
      r.ok[c] = ok;
      if (c == 0) {
        r.fmt = fmt;
        r.v_max = v_max;
        const int rows = MT == 1 ? 1 : min(MT, (q.nt * (a.hq / a.hkv) - mg * 128 * MT + 127) / 128);
        r.flags = (in == 0 ? kTileFirst : in == 1 ? kTileSecond : 0) |
                  (t == q.tiles - 1 || j == n - 1 ? kTileLast : 0) | (plain ? kTilePlain : 0) | (cold ? kTileCold : 0) |
                  static_cast<uint32_t>(rows) << kTileRowsShift | static_cast<uint32_t>(seg & 3) << kTileSegShift;
        r.b = b;
        r.hk = hk;
        r.mg = mg;
        r.cold = q.cold;
        r.hot = q.hot;
        r.keys = q.keys;
        r.row0 = row0;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.rfull[batch & 1]);
    pos += kTreeBatch;
  }
}

// ---- the MMA warp (one elected thread issues) ----
// TMEM columns: S of stream i at 128 i, its O at 256 + 128 i.  The weights of a
// tile replace its S (FP16, the first 64 columns).

// S of tile j for stream i; its Q operand is number `q`
template <int MT>
__device__ __forceinline__ void tree_qk(TreeSmem<MT> &sm, uint32_t q_s, uint32_t k_s, uint32_t tmem, int j, int i, int q) {
  const uint64_t dq = tc_desc_sw128(q_s + q * kTreeOperand);
  const uint64_t dk = tc_desc_sw128(k_s + (j & (kTreeStages - 1)) * kTreeOperand);
  if (tc_elect()) {
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const uint64_t o = (k >> 2) * (kTreeSlab >> 4) + 2 * (k & 3);
      tc_mma_ss(tmem + 128 * i, dq + o, dk + o, tc_idesc_f16(128), k > 0);
    }
    tc_commit(&sm.sfull[i]);
  }
  __syncwarp();
}

// O += P V of tile j for stream i, whose n-th tile it is
template <int MT>
__device__ __forceinline__ bool tree_pv(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t v_s, uint32_t tmem, int j, int i,
                                        int n, bool first) {
  if (!tree_wait_warp(sm, &sm.vfull[j & (kTreeStages - 1)], (j / kTreeStages) & 1, a)) return false;
  if (!tree_wait_warp(sm, &sm.pfull[i], n & 1, a)) return false;
  fence_proxy_async_smem();
  tc_fence_after();
  const uint64_t dv = tc_desc_sw128(v_s + (j & (kTreeStages - 1)) * kTreeOperand);
  if (tc_elect()) {
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const uint64_t o = (k >> 2) * (kTreeSlab >> 4) + 2 * (k & 3);
      tc_mma_ts(tmem + 256 + 128 * i, tmem + 128 * i + 8 * k, dv + o, tc_idesc_f16(128), !first || k > 0);
    }
    tc_commit(&sm.odone[i]);
  }
  __syncwarp();
  return true;
}

template <int MT>
__device__ __forceinline__ void tree_mma(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t q_s, uint32_t k_s, uint32_t v_s,
                                         uint32_t tmem, int n) {
  constexpr int kQ = TreeSmem<MT>::kQ;
  auto commit = [](uint64_t *bar) {
    if (tc_elect()) tc_commit(bar);
    __syncwarp();
  };
  auto two = [](uint32_t flags) { return MT == 2 && ((flags >> kTileRowsShift) & 3) == 2; };
  // tile j's K is there, and its segment's Q
  auto open = [&](int j, uint32_t &flags) -> bool {
    if (!tree_wait_warp(sm, &sm.kfull[j & (kTreeStages - 1)], (j / kTreeStages) & 1, a)) return false;
    flags = sm.rec[j & (kTreeRecs - 1)].flags;
    if (flags & kTileFirst) {
      const uint32_t seg = flags >> kTileSegShift;
      if (!tree_wait_warp(sm, &sm.qfull[seg % kQ], (seg / kQ) & 1, a)) return false;
    }
    fence_proxy_async_smem();
    tc_fence_after();
    return true;
  };
  auto close = [&](int j, uint32_t flags) {
    commit(&sm.kempty[j & (kTreeStages - 1)]);
    if (flags & kTileLast) commit(&sm.qempty[(flags >> kTileSegShift) % kQ]);
  };
  auto q_of = [](uint32_t flags) { return static_cast<int>((flags >> kTileSegShift) % kQ) * MT; };

  if (MT == 1) {
    // tile j belongs to stream j & 1; its Q K^T is issued as soon as the
    // stream's last P V, whose weights its S overwrites
    uint32_t f0 = 0, f1 = 0, f2 = 0;  // flags of tiles j, j + 1, j + 2
    int freed = 0;                    // segments whose O may be written
    if (!open(0, f0)) return;
    tree_qk<MT>(sm, q_s, k_s, tmem, 0, 0, q_of(f0));
    close(0, f0);
    if (n > 1) {
      if (!open(1, f1)) return;
      tree_qk<MT>(sm, q_s, k_s, tmem, 1, 1, q_of(f1));
      close(1, f1);
    }
    for (int j = 0; j < n; j++) {
      if (f0 & kTileFirst) {
        if (!tree_wait_warp(sm, &sm.ofree[0], (freed & 1) ^ 1, a)) return;
        freed++;
      }
      if (!tree_pv<MT>(a, sm, v_s, tmem, j, j & 1, j >> 1, f0 & (kTileFirst | kTileSecond))) return;
      commit(&sm.vempty[j & (kTreeStages - 1)]);
      if ((j + 1) % kTreeBatch == 0) commit(&sm.rfree[(j / kTreeBatch) & 1]);
      if (j + 2 < n) {
        if (!open(j + 2, f2)) return;
        tree_qk<MT>(sm, q_s, k_s, tmem, j + 2, j & 1, q_of(f2));
        close(j + 2, f2);
      }
      f0 = f1;
      f1 = f2;
    }
  } else {
    uint32_t fq = 0, fp;                       // of the tiles of Q K^T (one ahead) and of P V
    int used0 = 0, used1 = 0, o0 = 0, o1 = 0;  // tiles and segments of row tiles 0 and 1
    if (!open(0, fq)) return;
    tree_qk<MT>(sm, q_s, k_s, tmem, 0, 0, q_of(fq));
    if (two(fq)) tree_qk<MT>(sm, q_s, k_s, tmem, 0, 1, q_of(fq) + 1);
    close(0, fq);
    for (int j = 0; j < n; j++) {
      fp = fq;
      const bool more = j + 1 < n, first = fp & kTileFirst;
      if (first) {
        if (!tree_wait_warp(sm, &sm.ofree[0], (o0++ & 1) ^ 1, a)) return;
        if (two(fp) && !tree_wait_warp(sm, &sm.ofree[1], (o1++ & 1) ^ 1, a)) return;
      }
      // the next tile's S of a row tile follows that row tile's P V
      if (!tree_pv<MT>(a, sm, v_s, tmem, j, 0, used0++, first)) return;
      if (more) {
        if (!open(j + 1, fq)) return;
        tree_qk<MT>(sm, q_s, k_s, tmem, j + 1, 0, q_of(fq));
      }
      if (two(fp) && !tree_pv<MT>(a, sm, v_s, tmem, j, 1, used1++, first)) return;
      commit(&sm.vempty[j & (kTreeStages - 1)]);
      if ((j + 1) % kTreeBatch == 0) commit(&sm.rfree[(j / kTreeBatch) & 1]);
      if (more) {
        if (two(fq)) tree_qk<MT>(sm, q_s, k_s, tmem, j + 1, 1, q_of(fq) + 1);
        close(j + 1, fq);
      }
    }
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

// Two FP32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &x, float &y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// The nodes of unit c of a tail tile that the row attends (bits), k = the node
// of the unit's first key; `odd` collects those whose V is not finite.
__device__ __forceinline__ uint32_t tree_nodes(const TreeRec &me, int c, int k, uint64_t nodes, uint64_t &odd) {
  uint32_t own = 0, bad = 0;
  if (k >= 0) own = k < 64 ? static_cast<uint32_t>(nodes >> k) : 0u;
  else if (k > -32) own = static_cast<uint32_t>(nodes << -k);
#pragma unroll
  for (int w = 0; w < 4; w++) bad |= me.bad[w][c];
  bad &= own;
  if (bad) odd |= k >= 0 ? static_cast<uint64_t>(bad) << k : static_cast<uint64_t>(bad) >> -k;
  return own;
}

// 16 channels of a row, from channel c0 on: to the output, or to the CTA's part
// of a unit that several share.  v: the sums in units of `scale`.
template <int MT>
__device__ __forceinline__ void tree_store(const TreeArgs &a, uint32_t (&v)[16], float scale, uint64_t odd, int c0, int b,
                                           int hk, bool live, bool whole, size_t out_row, size_t slot, int part_row) {
#pragma unroll
  for (int k = 0; k < 16; k++) v[k] = __float_as_uint(__uint_as_float(v[k]) * scale);
  for (uint64_t rest = odd; rest; rest &= rest - 1) {
    const int node = __ffsll(static_cast<long long>(rest)) - 1;
    const __half *vr = a.v_tree + ((static_cast<size_t>(b) * a.max_tree + node) * a.hkv + hk) * kDim + c0;
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const __half2 x = *reinterpret_cast<const __half2 *>(vr + k);
      if (f16_not_finite(__half_as_ushort(x.x))) v[k] = __float_as_uint(__uint_as_float(v[k]) + __low2float(x));
      if (f16_not_finite(__half_as_ushort(x.y))) v[k + 1] = __float_as_uint(__uint_as_float(v[k + 1]) + __high2float(x));
    }
  }
  if (!live) return;
  if (whole) {
#pragma unroll
    for (int k = 0; k < 16; k += 8) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; e++)
        w[e] = half2_bits(__uint_as_float(v[k + 2 * e]), __uint_as_float(v[k + 2 * e + 1]));
      *reinterpret_cast<uint4 *>(a.out + out_row * kDim + c0 + k) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    uint4 *dst = reinterpret_cast<uint4 *>(a.part_o) + slot * 32 * 128 * MT;
#pragma unroll
    for (int k = 0; k < 16; k += 4)
      dst[(c0 / 4 + (k >> 2)) * (128 * MT) + part_row] = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
  }
}

template <int MT>
__device__ __forceinline__ void tree_softmax(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t tmem, int n_tiles) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stream = warp >> 2, row_in = threadIdx.x & 127;
  const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t t_s = lanes + 128 * stream, t_o = lanes + 256 + 128 * stream;
  const int G = a.hq / a.hkv;
  TreeWalk<MT> walk;
  walk.pos = sm.start_pos;
  walk.left = n_tiles;
  walk.b = sm.start_b;
  walk.enter(a);
  int j = 0;      // tiles of the CTA so far
  int mine = 0;   // tiles of this stream so far
  for (int seg = 0; walk.next(a); seg++) {
    const int j0 = j;
    j += walk.t1 - walk.t0;
    if (MT == 2 && stream >= walk.m_tiles(a)) continue;
    const int row = walk.mg * 128 * MT + (MT == 2 ? stream * 128 : 0) + row_in;
    const bool live = row < walk.nt * G;
    const bool warp_live = row - lane < walk.nt * G;
    const int t = live ? row / G : 0;
    const int cold_tiles = (walk.cold + kTK - 1) / kTK;
    uint64_t nodes = 0;  // nodes this row attends
    int node0 = 0;       // the node of the first tail row
    {
      const TreeSeq seq = tree_seq<MT>(a, walk.b);
      node0 = -seq.hot;
      if (live && seq.keys > 0) {
        nodes = a.mask ? a.mask[static_cast<size_t>(walk.b) * a.max_tree + t] : (~0ull >> (63 - t));
        if (seq.keys < 64) nodes &= (1ull << seq.keys) - 1;
      }
    }
    float m = -INFINITY, l = 0.f, ref = 1.f, inv = 1.f;
    uint64_t odd = 0;    // attended nodes whose V is not finite
    bool first = true;   // of this stream in the segment
    for (int i = MT == 2 ? j0 : j0 + ((j0 ^ stream) & 1); i < j; i += MT == 2 ? 1 : 2) {
      // (a row tile that sat out a segment may have missed phases of mfull: S
      // first, whose phases are its own)
      if (!tree_wait_warp(sm, &sm.sfull[stream], mine & 1, a)) return;
      if (!tree_wait_warp(sm, &sm.mfull[i & (kTreeRecs - 1)], (i / kTreeRecs) & 1, a)) return;
      tc_fence_after();
      if (warp_live) {
        const TreeRec &me = sm.rec[i & (kTreeRecs - 1)];
        const int ti = walk.t0 + i - j0;
        const bool tail = ti >= cold_tiles, plain = me.flags & kTilePlain;
        const int k0 = node0 + (ti - cold_tiles) * kTK;
        float top = -INFINITY;
        uint32_t v[32];
#pragma unroll 1
        for (int c = 0; c < 4; c++) {
          tc_ld32(t_s + 32 * c, v);
          const float s = me.k_scale[c] * a.qk_scale;
          tc_wait_ld(v);
          if (plain) {
            top = fmaxf(top, max32(v) * s);
          } else {
            uint32_t ok = me.ok[c];
            if (tail) ok |= tree_nodes(me, c, k0 + 32 * c, nodes, odd);
#pragma unroll
            for (int k = 0; k < 32; k++)
              if (ok >> k & 1) top = fmaxf(top, __uint_as_float(v[k]) * s);
          }
        }
        // m and r follow when they lag too far behind; O and l follow them (the
        // stream's last P V is done: this tile's S came after it)
        float r_new = ref;
        const float v_max = me.v_max;
        if (first || v_max > kLagScale * ref) r_new = v_max > 0.f ? v_max : ref;
        const float m_new = first || top > m + kLagLog2 ? fmaxf(m, top) : m;
        if (__any_sync(0xffffffffu, m_new != m || r_new != ref)) {
          if (!first) {
            const float f = m == -INFINITY ? 0.f : ex2(m - m_new);
            l *= f;
            const float g = f * __fdividef(ref, r_new);
#pragma unroll 1
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
          inv = __fdividef(1.f, ref);
        }
        const float base = m == -INFINITY ? 0.f : -m;
        uint64_t sum0 = 0, sum1 = 0;
#pragma unroll 1
        for (int c = 0; c < 4; c++) {
          tc_ld32(t_s + 32 * c, v);
          const float s = me.k_scale[c] * a.qk_scale, f = me.v_scale[c] * inv;
          const uint64_t s2 = pack2(s, s), b2 = pack2(base, base), f2 = pack2(f, f);
          uint32_t ok = 0xffffffffu;
          if (!plain) {
            ok = me.ok[c];
            if (tail) ok |= tree_nodes(me, c, k0 + 32 * c, nodes, odd);
          }
          tc_wait_ld(v);
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float x, y;
            unpack2(fma2(pack2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), s2, b2), x, y);
            x = ex2(x);
            y = ex2(y);
            if (!plain) {
              x = ok >> k & 1 ? x : 0.f;
              y = ok >> (k + 1) & 1 ? y : 0.f;
            }
            const uint64_t e = pack2(x, y);
            if (k & 2) sum1 = add2(sum1, e);
            else sum0 = add2(sum0, e);
            unpack2(mul2(e, f2), x, y);
            p[k >> 1] = half2_bits(x, y);
          }
          tc_st16(t_s + 16 * c, p);
        }
        float x, y;
        unpack2(add2(sum0, sum1), x, y);
        l += x + y;
        tc_wait_st();
      }
      first = false;
      mine++;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.pfull[stream]);
    }
    // the segment's end: O of the stream's last tile
    const bool whole = walk.t0 == 0 && walk.t1 == walk.tiles;
    const size_t out_row = (static_cast<size_t>(walk.b) * a.max_tree + t) * a.hq + walk.hk * G + row - t * G;
    const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (walk.t0 == 0 ? 1 : 0);
    const int part_row = (MT == 2 ? stream * 128 : 0) + row_in;
    if (!first) {
      if (!tree_wait_warp(sm, &sm.odone[stream], (mine - 1) & 1, a)) return;
      tc_fence_after();
    }
    if (MT == 2) {
      if (warp_live) {
#pragma unroll 1
        for (int c = 0; c < 8; c++) {
          uint32_t v[16];
          tc_ld16(t_o + 16 * c, v);
          tc_wait_ld(v);
          tree_store<MT>(a, v, whole ? (l != 0.f ? ref / l : 0.f) : ref, odd, 16 * c, walk.b, walk.hk, live, whole, out_row,
                         slot, part_row);
        }
      }
    } else {
      // both streams of a row meet: group i takes channels 64 i.. of the two
      TreeStat *st = &sm.stat[seg & 1][0][row_in];
      st[128 * stream] = TreeStat{m, l, ref, odd};
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.xfull);
      if (!tree_wait_warp(sm, &sm.xfull, seg & 1, a)) return;
      tc_fence_after();
      if (warp_live) {
        const TreeStat o = st[128 * (stream ^ 1)];
        const float top = fmaxf(m, o.m);
        const float f = m == top ? 1.f : ex2(m - top), fo = o.m == top ? 1.f : ex2(o.m - top);
        // (a stream without a tile has nothing in its O)
        const bool other = walk.t1 - walk.t0 > 1 || first;
        l = l * f + o.l * fo;
        m = top;
        const float scale = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
        const float g = first || f == 0.f ? 0.f : f * ref, go = !other || fo == 0.f ? 0.f : fo * o.ref;
        const uint32_t t_o2 = lanes + 256 + 128 * (stream ^ 1);
#pragma unroll 1
        for (int c = 4 * stream; c < 4 * stream + 4; c++) {
          uint32_t v[16];
          if (!first) {
            tc_ld16(t_o + 16 * c, v);
            tc_wait_ld(v);
          }
#pragma unroll
          for (int k = 0; k < 16; k++) v[k] = g == 0.f ? 0u : __float_as_uint(__uint_as_float(v[k]) * g);
          if (other) {
            uint32_t w[16];
            tc_ld16(t_o2 + 16 * c, w);
            tc_wait_ld(w);
#pragma unroll
            for (int k = 0; k < 16; k++)
              if (go != 0.f) v[k] = __float_as_uint(fmaf(__uint_as_float(w[k]), go, __uint_as_float(v[k])));
          }
          tree_store<MT>(a, v, scale, odd | o.odd, 16 * c, walk.b, walk.hk, live, whole, out_row, slot, part_row);
        }
      }
    }
    if (live && (MT == 2 || stream == 0)) {
      if (whole) {
        if (a.lse_out) a.lse_out[out_row] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
      } else {
        float2 *ml = reinterpret_cast<float2 *>(a.part_ml) + slot * 128 * MT;
        ml[part_row] = make_float2(m, l);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.ofree[MT == 2 ? stream : 0]);
    // who has the unit's tiles, from the CTA with its first
    if (threadIdx.x == 0 && walk.t0 == 0) {
      const long long ctas = min(static_cast<long long>(a.ctas), sm.total);
      // the list's index of the unit's last tile, and the run that has it
      const long long end = sm.total * blockIdx.x / ctas + j0 + walk.tiles;
      const int last = static_cast<int>((end * ctas - 1) / sm.total);
      const int groups_max = (a.max_tree * G + 128 * MT - 1) / (128 * MT);
      a.unit_ctas[(static_cast<size_t>(walk.b) * a.hkv + walk.hk) * groups_max + walk.mg] =
          make_int2(static_cast<int>(blockIdx.x), last);
    }
  }
}

template <int MT, bool kF16>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const __grid_constant__ TreeArgs a) {
  using Shape = TreeShape<MT>;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const uint32_t q_s = base, k_s = q_s + Shape::kQBytes, v_s = k_s + kTreeStages * kTreeOperand;
  TreeSmem<MT> &sm = *reinterpret_cast<TreeSmem<MT> *>(raw + (base - smem_addr(raw)) + Shape::kQBytes +
                                                       2 * kTreeStages * kTreeOperand);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge waits for this grid's end
  constexpr int kMmaWarp = kTreeSoft + kTreeProd;

  // the list's length and where this CTA's run starts: every thread sums a
  // range of sequences, a scan over the threads places them
  const int per = (a.batch + kTreeThreads - 1) / kTreeThreads;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; b++) {
    const TreeSeq s = tree_seq<MT>(a, b);
    mine += static_cast<long long>(s.tiles) * s.groups * a.hkv;
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
      mbar_init(&sm.kfull[i], kTreeProd / kTreeGroups);
      mbar_init(&sm.kempty[i], 1);
      mbar_init(&sm.vfull[i], kTreeProd / kTreeGroups);
      mbar_init(&sm.vempty[i], 1);
    }
    for (int i = 0; i < kTreeRecs; i++) mbar_init(&sm.mfull[i], kTreeProd / kTreeGroups);
    for (int i = 0; i < TreeSmem<MT>::kQ; i++) {
      mbar_init(&sm.qfull[i], kTreeProd / kTreeGroups);
      mbar_init(&sm.qempty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.pfull[i], 4);
      mbar_init(&sm.odone[i], 1);
      mbar_init(&sm.ofree[i], MT == 1 ? 8 : 4);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&sm.rfull[i], 1);
      mbar_init(&sm.rfree[i], 1);
    }
    mbar_init(&sm.xfull, 8);
    mbar_init(&sm.drain, 1);
    mbar_fence_init();
  }
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kTreeThreads / 32; w++) {
    const long long v = sm.warp_sum[w];
    if (w < warp) before += v;
    total += v;
  }
  const long long ctas = min(static_cast<long long>(gridDim.x), total);
  if (static_cast<long long>(blockIdx.x) >= ctas) return;  // the whole CTA: nothing to do
  const long long w0 = total * blockIdx.x / ctas;
  const int n_tiles = static_cast<int>(total * (blockIdx.x + 1) / ctas - w0);
  long long at = before + inc - mine;
  if (w0 >= at && w0 < at + mine) {
    for (int b = b0; b < b1; b++) {
      const TreeSeq s = tree_seq<MT>(a, b);
      const long long span = static_cast<long long>(s.tiles) * s.groups * a.hkv;
      if (w0 < at + span) {
        sm.start_b = b;
        sm.start_pos = w0 - at;
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

  if (warp < kTreeSoft) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTreeSoftRegs));
    tree_softmax<MT>(a, sm, tmem, n_tiles);
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTreeProdRegs));
    tree_produce<MT, kF16>(a, sm, q_s, k_s, v_s, n_tiles);
  } else if (warp > kMmaWarp) {
    tree_scout<MT, kF16>(a, sm, n_tiles);
  } else {
    tree_mma<MT>(a, sm, q_s, k_s, v_s, tmem, n_tiles);
    __syncwarp();
    // no MMA is in flight when TMEM is given back
    if (tc_elect()) tc_commit(&sm.drain);
    __syncwarp();
    if (!mbar_wait_bounded(&sm.drain, 0, kDefaultWaitCycles)) set_status(a.status, HYB_STATUS_TIMEOUT);
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
    // what the producers add the softmax warps give up, of the registers that
    // the launch really has
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, tree_kernel<MT, kF16>);
    if (e != cudaSuccess) return e;
    if (2 * at.numRegs < kTreeSoftRegs + kTreeProdRegs) return cudaErrorInvalidKernelImage;
    if (dev < 31) configured_dev_mask |= 1 << dev;
  }
  tree_kernel<MT, kF16><<<a.ctas, kTreeThreads, Shape::kBytes, stream>>>(a);
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
