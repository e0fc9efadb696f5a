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
constexpr int kTreeStages = 2;               // K and V tiles in shared memory
constexpr int kTreeMeta = 4;                 // tile records (see the producers)
constexpr uint32_t kTreeOperand = 128 * 256; // bytes of a 128 x 128 FP16 operand
constexpr uint32_t kTreeSlab = kTreeOperand / 2;  // its halves of 64 columns
constexpr float kLagLog2 = 6.f;
constexpr float kLagScale = 256.f;

// TreeMeta::flags and TreeTile::flags
constexpr uint32_t kTileFirst = 1, kTileLast = 2, kTileRowsShift = 2, kTileGroupShift = 4;

// What the softmax needs to know of a tile; four units of 32 keys.
struct TreeMeta {
  float k_scale[4];  // 1 for FP16 rows
  float v_scale[4];
  uint32_t ok[4];    // keys that every row attends
  uint32_t flags;    // kTileFirst, kTileLast (of its segment) and the unit's row tiles
  uint32_t bad[4][4];  // [warp of the unit][unit]: tail rows with a V that is not finite
};

// Producer warps: with one row tile the codes set the pace; with two the MMAs
// do, and four warps leave every thread 128 registers.
constexpr int tree_producers(int mt) { return mt == 1 ? 8 : 4; }

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
  long long start_pos, total;  // the run's start within sequence start_b, the list's length
  long long warp_sum[32];
};

template <int MT>
struct TreeShape {
  static constexpr int kSoftWarps = 4 * MT;
  static constexpr int kProducers = tree_producers(MT);
  static constexpr int kThreads = 32 * (kSoftWarps + kProducers + 1);
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

// A producer thread has units u, u + kStep, ... of 32 keys of every tile (u =
// thread / 128): K of key (thread % 128) / 4, 32 channels; V of INT8 / INT4
// channel thread % 128, all 32 keys, of FP16 rows channels 2 (thread % 64), + 1
// and 16 keys.
template <int MT>
struct TreePart {
  static constexpr int kStep = tree_producers(MT) / 4;
  static constexpr int kUnits = 4 / kStep;
};

template <int MT>
struct TreeTile {
  int b, hk, ti, cold;  // unit, tile (ti < 0: the list's end) and the sequence's cold tokens
  uint32_t flags;       // as TreeMeta's, and the row group from kTileGroupShift on
  int ent[TreePart<MT>::kUnits];  // block-table entries of the thread's units
};

template <int MT>
struct TreeFeed {
  TreeWalk<MT> walk;
  int t, u;  // next tile of the walk's segment; the thread's first unit

  __device__ __forceinline__ TreeTile<MT> next(const TreeArgs &a) {
    TreeTile<MT> x;
    x.flags = 0;
    if (t == walk.t1) {
      if (!walk.next(a)) {
        x.ti = -1;
        return x;
      }
      t = walk.t0;
      x.flags = kTileFirst;
    }
    x.b = walk.b;
    x.hk = walk.hk;
    x.cold = walk.cold;
    x.ti = t++;
    if (t == walk.t1) x.flags |= kTileLast;
    x.flags |= static_cast<uint32_t>(walk.m_tiles(a)) << kTileRowsShift;
    x.flags |= static_cast<uint32_t>(walk.mg) << kTileGroupShift;
#pragma unroll
    for (int i = 0; i < TreePart<MT>::kUnits; i++) {
      const int p = x.ti * kTK + 32 * (u + TreePart<MT>::kStep * i);
      x.ent[i] = p < x.cold ? __ldg(a.block_table + static_cast<size_t>(x.b) * a.max_blocks + (p >> a.bshift)) : -1;
    }
    return x;
  }
};

// Valid keys of the unit at position p of a cold tile (0: nothing to read).
__device__ __forceinline__ int unit_keys(const TreeArgs &a, int cold, int p, int ent) {
  const int n = max(0, min(32, cold - p));
  if (n > 0 && (ent < 0 || ent >= a.num_phys)) {
    set_status(a.status, HYB_STATUS_BAD_BLOCK);
    return 0;
  }
  return n;
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
  const int slot = 32 * half + ((tid & 127) >> 2);
  if (int4) k[0] = ldg16(pair + slot * 64 + 16 * (tid & 3));
  else load_codes(a, pair + slot * 128 + 32 * (tid & 3), k);
}

// (V: the unit's two 16-slot chunks are one aligned pair, swapped where the
// swizzle's lowest bit is set; store_v8 puts them right)
__device__ __forceinline__ void load_v(const TreeArgs &a, const uint8_t *pair, int half, bool int4, int tid, uint4 (&v)[2]) {
  const int c = tid & 127;
  const uint8_t *t = pair + kTileBytes;
  if (int4) v[0] = ldg16(t + c * 32 + 8 * ((2 * half) ^ ((c >> 2) & 2)));
  else load_codes(a, t + c * 64 + 16 * ((2 * half) ^ ((c >> 1) & 2)), v);
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

// FP16 rows as units: rows of an FP16 cold block (`base`, n of them valid), or
// rows r0.. of the tail (the ring's in the order of their positions, then the
// nodes).
struct TreeRows {
  const __half *base;  // null: the tail
  int n;
  int b, hk, cold, hot, keys, r0;

  // the K row (kv 1: V row) of key k of the unit, or null
  __device__ __forceinline__ const __half *row(const TreeArgs &a, int k, int kv) const {
    if (base) return k < n ? base + (2 * k + kv) * kDim : nullptr;
    int r = r0 + k;
    if (r < hot)
      return reinterpret_cast<const __half *>(a.hot) +
             (((static_cast<size_t>(b) * a.hkv + hk) * a.hot_tokens + ((cold + r) & (a.hot_tokens - 1))) * 2 + kv) * kDim;
    r -= hot;
    if (r >= keys) return nullptr;
    return (kv ? a.v_tree : a.k_tree) + ((static_cast<size_t>(b) * a.max_tree + r) * a.hkv + hk) * kDim;
  }
};

__device__ __forceinline__ void rows_k(const TreeArgs &a, const TreeRows &x, int tid, uint4 (&k)[4]) {
  const __half *row = x.row(a, (tid & 127) >> 2, 0);
#pragma unroll
  for (int j = 0; j < 4; j++) k[j] = row ? ldg16(row + 32 * (tid & 3) + 8 * j) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ void rows_v(const TreeArgs &a, const TreeRows &x, int tid, uint32_t (&w)[16]) {
  const int k0 = 16 * ((tid >> 6) & 1), c = 2 * (tid & 63);
#pragma unroll
  for (int j = 0; j < 16; j++) {
    const __half *r = x.row(a, k0 + j, 1);
    w[j] = r ? __ldg(reinterpret_cast<const uint32_t *>(r + c)) : 0u;
  }
}

// The query rows of a unit into its Q operand(s); rows beyond the tree are 0.
template <int MT>
__device__ __forceinline__ void load_q(const TreeArgs &a, const TreeTile<MT> &x, uint32_t st, int tid) {
  const int G = a.hq / a.hkv, mg = x.flags >> kTileGroupShift;
  const int rows = (a.n_tree ? a.n_tree[x.b] : a.max_tree) * G;
#pragma unroll 4
  for (int i = tid; i < 128 * MT * 16; i += 32 * tree_producers(MT)) {
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
  const int tid = threadIdx.x - 32 * TreeShape<MT>::kSoftWarps, lane = tid & 31;
  const int u = tid >> 7;
  constexpr int kQ = TreeSmem<MT>::kQ, kUnits = TreePart<MT>::kUnits, kStep = TreePart<MT>::kStep;
  TreeFeed<MT> feed;
  feed.walk.pos = sm.start_pos;
  feed.walk.left = n;
  feed.walk.b = sm.start_b;
  feed.walk.enter(a);
  feed.walk.t1 = feed.t = 0;
  feed.u = u;
  TreeTile<MT> cur, nxt = feed.next(a);
  cur.ti = -1;
  cur.cold = 0;
  const bool scribe = (tid & 127) == 0;
  // of the tile whose codes are in registers: codes, scales, valid keys, formats
  uint4 rk[kF16 ? 1 : kUnits][2], rv[kF16 ? 1 : kUnits][2];
  float2 sc[kUnits];
  int valid[kUnits];
  uint32_t fmt = 0, fmt_next = 0;  // bit i: unit i is INT4

  // one round per tile, and one before the first that only loads
  int seg = -1;
  for (int j = -1; j < n; j++) {
    const int s = j & (kTreeStages - 1);
    const uint32_t ph = (j / kTreeStages) & 1;
    const uint32_t kst = k_s + s * kTreeOperand, vst = v_s + s * kTreeOperand;
    const bool cold = j >= 0 && cur.ti * kTK < cur.cold;
    const TreeTile<MT> nn = feed.next(a);
    if (j >= 0) {
      if (cur.flags & kTileFirst) {
        seg++;
        if (!tree_wait_warp(sm, &sm.qempty[seg % kQ], ((seg / kQ) & 1) ^ 1, a)) return;
        load_q<MT>(a, cur, q_s + (seg % kQ) * MT * kTreeOperand, tid);
        producer_arrive(&sm.qfull[seg % kQ], lane);
      }
      TreeMeta &m = sm.meta[j & (kTreeMeta - 1)];
      uint32_t bad = 0;  // lane c < 4: unit c
      if (kF16 || !cold) {
        // FP16 rows.  V first: the record names the nodes whose V is not
        // finite.  Such a value must not meet the zero weight of a row that
        // does not attend its node: it becomes 0 here, and the rows that do
        // attend the node add it at the end
        const TreeSeq q = tree_seq<MT>(a, cur.b);
        const int tail0 = (cur.ti - (cur.cold + kTK - 1) / kTK) * kTK;
        auto rows = [&](int i) {
          const int c = u + kStep * i;
          TreeRows x{nullptr, 0, cur.b, cur.hk, cur.cold, q.hot, q.keys, tail0 + 32 * c};
          if (kF16 && cold) {
            const int p = cur.ti * kTK + 32 * c;
            x.n = unit_keys(a, cur.cold, p, cur.ent[i]);
            x.base = reinterpret_cast<const __half *>(
                a.cold + ((((static_cast<size_t>(x.n ? cur.ent[i] : 0) * a.hkv + cur.hk) << a.bshift) +
                           (p & ((1 << a.bshift) - 1))) * kHotTokenBytes));
          }
          return x;
        };
        if (!tree_wait_warp(sm, &sm.vempty[s], ph ^ 1, a)) return;
#pragma unroll
        for (int i = 0; i < kUnits; i++) {
          const int c = u + kStep * i, k0 = 16 * ((tid >> 6) & 1);
          const TreeRows x = rows(i);
          uint32_t w[16];
          rows_v(a, x, tid, w);
          if (!(kF16 && cold)) {
            uint32_t b = 0;
#pragma unroll
            for (int k = 0; k < 16; k++) {
              if (x.r0 + k0 + k < q.hot) continue;
              const bool lo = f16_not_finite(w[k]), hi = f16_not_finite(w[k] >> 16);
              if (lo) w[k] &= 0xffff0000u;
              if (hi) w[k] &= 0x0000ffffu;
              if (lo || hi) b |= 1u << (k0 + k);
            }
            b = __reduce_or_sync(0xffffffffu, b);
            if (lane == c) bad = b;
          }
          store_v16(vst, c, tid, w);
          sc[i] = make_float2(1.f, 1.f);
          valid[i] = kF16 && cold ? x.n : max(0, min(32, q.hot - x.r0));
        }
        producer_arrive(&sm.vfull[s], lane);
        if (!tree_wait_warp(sm, &sm.kempty[s], ph ^ 1, a)) return;
#pragma unroll
        for (int i = 0; i < kUnits; i++) {
          uint4 k[4];
          rows_k(a, rows(i), tid, k);
          store_k16(kst, u + kStep * i, tid, k);
        }
      } else {
        if (!tree_wait_warp(sm, &sm.kempty[s], ph ^ 1, a)) return;
        if constexpr (!kF16) {
#pragma unroll
          for (int i = 0; i < kUnits; i++) store_k8(kst, u + kStep * i, tid, fmt >> i & 1, rk[i]);
        }
      }
      if (lane < 4 && lane % kStep == u) m.bad[(tid >> 5) & 3][lane] = bad;
      if (scribe) {
#pragma unroll
        for (int i = 0; i < kUnits; i++) {
          const int c = u + kStep * i;
          m.k_scale[c] = sc[i].x;
          m.v_scale[c] = sc[i].y;
          m.ok[c] = valid[i] >= 32 ? 0xffffffffu : (1u << valid[i]) - 1;
        }
        if (u == 0) m.flags = cur.flags;
      }
      producer_arrive(&sm.kfull[s], lane);
      if (lane == 0) mbar_arrive(&sm.mfull[j & (kTreeMeta - 1)]);
    }
    // the next tile's codes are on their way while this one's V is stored
    const bool more = !kF16 && nxt.ti >= 0 && nxt.ti * kTK < nxt.cold;
    const uint8_t *pair[kUnits];
    if (!kF16 && more) {
      fmt_next = 0;
#pragma unroll
      for (int i = 0; i < kUnits; i++) {
        const int p = nxt.ti * kTK + 32 * (u + kStep * i);
        valid[i] = unit_keys(a, nxt.cold, p, nxt.ent[i]);
        const bool int4 = a.quant_bits == 4 || (a.n_int4 != nullptr && (p >> a.bshift) < a.n_int4[nxt.b]);
        if (int4) fmt_next |= 1u << i;
        const int slot = p & ((1 << a.bshift) - 1);
        const size_t at = static_cast<size_t>(valid[i] ? nxt.ent[i] : 0) * a.hkv + nxt.hk;
        pair[i] = a.cold + ((at << a.lsub) + (slot >> 6)) * kTilePairBytes;
        // (an empty unit has code 0 and no say in the reference scale)
        sc[i] = make_float2(0.f, 0.f);
        rk[i][0] = rk[i][1] = make_uint4(0, 0, 0, 0);
        if (valid[i]) {
          load_k(a, pair[i], (slot >> 5) & 1, int4, tid, rk[i]);
          if (scribe) sc[i] = __ldg(reinterpret_cast<const float2 *>(a.scales) + at);
        }
      }
    }
    if (!kF16 && cold) {
      if (!tree_wait_warp(sm, &sm.vempty[s], ph ^ 1, a)) return;
#pragma unroll
      for (int i = 0; i < kUnits; i++) store_v8(vst, u + kStep * i, tid, fmt >> i & 1, rv[i]);
      producer_arrive(&sm.vfull[s], lane);
    }
    if (!kF16 && more) {
#pragma unroll
      for (int i = 0; i < kUnits; i++) {
        const int p = nxt.ti * kTK + 32 * (u + kStep * i);
        rv[i][0] = rv[i][1] = make_uint4(0, 0, 0, 0);
        if (valid[i]) load_v(a, pair[i], (p & ((1 << a.bshift) - 1)) >> 5 & 1, fmt_next >> i & 1, tid, rv[i]);
      }
      fmt = fmt_next;
    }
    cur = nxt;
    nxt = nn;
  }
}

// ---- the MMA thread ----
// TMEM columns: MT 1: S buffers 0 and 128, O 256.  MT 2: S of row tile m at
// 128 m, O at 256 + 128 m.  The weights of a tile replace its S (FP16, the
// first 64 columns).

// S of tile j, row tile m
template <int MT>
__device__ __forceinline__ void tree_qk(TreeSmem<MT> &sm, uint32_t q_s, uint32_t k_s, uint32_t tmem, int j, int seg, int m) {
  const int buf = MT == 1 ? j & 1 : m;
  const uint64_t dq = tc_desc_sw128(q_s + ((seg % TreeSmem<MT>::kQ) * MT + m) * kTreeOperand);
  const uint64_t dk = tc_desc_sw128(k_s + (j & (kTreeStages - 1)) * kTreeOperand);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint64_t o = (i >> 2) * (kTreeSlab >> 4) + 2 * (i & 3);
    tc_mma_ss(tmem + 128 * buf, dq + o, dk + o, tc_idesc_f16(128), i > 0);
  }
  tc_commit(&sm.sfull[buf]);
}

// O += P V of tile j, row tile m, whose n-th tile it is
template <int MT>
__device__ __forceinline__ bool tree_pv(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t v_s, uint32_t tmem, int j, int m,
                                        int n, bool first) {
  const int buf = MT == 1 ? n & 1 : m;
  if (!tree_wait(sm, &sm.pfull[buf], (MT == 1 ? n >> 1 : n) & 1, a)) return false;
  if (!tree_wait(sm, &sm.vfull[j & (kTreeStages - 1)], (j / kTreeStages) & 1, a)) return false;
  fence_proxy_async_smem();
  tc_fence_after();
  const uint64_t dv = tc_desc_sw128(v_s + (j & (kTreeStages - 1)) * kTreeOperand);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint64_t o = (i >> 2) * (kTreeSlab >> 4) + 2 * (i & 3);
    tc_mma_ts(tmem + 256 + 128 * m, tmem + 128 * buf + 8 * i, dv + o, tc_idesc_f16(128), !first || i > 0);
  }
  tc_commit(&sm.odone[m][n & 1]);
  return true;
}

template <int MT>
__device__ __forceinline__ void tree_mma(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t q_s, uint32_t k_s, uint32_t v_s,
                                         uint32_t tmem, int n) {
  constexpr int kQ = TreeSmem<MT>::kQ;
  int seg = -1;                           // of the last tile opened
  uint32_t flags_q = 0, flags_p;          // of the tiles of Q K^T (one ahead) and of P V
  int used0 = 0, used1 = 0, o0 = 0, o1 = 0;  // tiles and segments of row tiles 0 and 1

  // tile j's K is there, and its segment's Q
  auto open = [&](int j) -> bool {
    if (!tree_wait(sm, &sm.kfull[j & (kTreeStages - 1)], (j / kTreeStages) & 1, a)) return false;
    flags_q = sm.meta[j & (kTreeMeta - 1)].flags;
    if (flags_q & kTileFirst) {
      seg++;
      if (!tree_wait(sm, &sm.qfull[seg % kQ], (seg / kQ) & 1, a)) return false;
    }
    fence_proxy_async_smem();
    tc_fence_after();
    return true;
  };
  auto close = [&](int j) {
    tc_commit(&sm.kempty[j & (kTreeStages - 1)]);
    if (flags_q & kTileLast) tc_commit(&sm.qempty[seg % kQ]);
  };
  auto two = [](uint32_t flags) { return MT == 2 && ((flags >> kTileRowsShift) & 3) == 2; };

  if (!open(0)) return;
  tree_qk<MT>(sm, q_s, k_s, tmem, 0, seg, 0);
  if (two(flags_q)) tree_qk<MT>(sm, q_s, k_s, tmem, 0, seg, 1);
  close(0);
  for (int j = 0; j < n; j++) {
    flags_p = flags_q;
    const bool more = j + 1 < n, first = flags_p & kTileFirst;
    if (first) {
      if (!tree_wait(sm, &sm.ofree[0], (o0++ & 1) ^ 1, a)) return;
      if (two(flags_p) && !tree_wait(sm, &sm.ofree[1], (o1++ & 1) ^ 1, a)) return;
    }
    if (MT == 1) {
      if (more) {
        if (!open(j + 1)) return;
        tree_qk<MT>(sm, q_s, k_s, tmem, j + 1, seg, 0);
        close(j + 1);
      }
      if (!tree_pv<MT>(a, sm, v_s, tmem, j, 0, used0++, first)) return;
    } else {
      // the next tile's S of a row tile follows that row tile's P V, whose
      // weights it overwrites
      if (!tree_pv<MT>(a, sm, v_s, tmem, j, 0, used0++, first)) return;
      if (more) {
        if (!open(j + 1)) return;
        tree_qk<MT>(sm, q_s, k_s, tmem, j + 1, seg, 0);
      }
      if (two(flags_p) && !tree_pv<MT>(a, sm, v_s, tmem, j, 1, used1++, first)) return;
      if (more) {
        if (two(flags_q)) tree_qk<MT>(sm, q_s, k_s, tmem, j + 1, seg, 1);
        close(j + 1);
      }
    }
    tc_commit(&sm.vempty[j & (kTreeStages - 1)]);
  }
}

// ---- softmax ----

template <int N>
__device__ __forceinline__ float max_of(const uint32_t *v) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; k++) m[k] = __uint_as_float(v[k]);
#pragma unroll
  for (int k = 4; k < N; k++) m[k & 3] = fmaxf(m[k & 3], __uint_as_float(v[k]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Keys of unit c of a tile that the row attends (bits): the record's, and in a
// tail tile the nodes the row's mask names; `odd` collects the attended nodes
// whose V is not finite.  k: the node of the unit's first key.
__device__ __forceinline__ uint32_t tree_ok(const TreeMeta &me, int c, bool tail, int k, uint64_t nodes, uint64_t &odd) {
  uint32_t ok = me.ok[c];
  if (tail) {
    uint32_t own = 0, bad = 0;
    if (k >= 0) own = k < 64 ? static_cast<uint32_t>(nodes >> k) : 0u;
    else if (k > -32) own = static_cast<uint32_t>(nodes << -k);
#pragma unroll
    for (int w = 0; w < 4; w++) bad |= me.bad[w][c];
    bad &= own;
    if (bad) odd |= k >= 0 ? static_cast<uint64_t>(bad) << k : static_cast<uint64_t>(bad) >> -k;
    ok |= own;
  }
  return ok;
}

template <int MT>
__device__ __forceinline__ void tree_softmax(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t tmem, int n_tiles) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt = warp >> 2, row_in = threadIdx.x & 127;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t t_o = tmem + lanes + 256 + 128 * mt;
  const int G = a.hq / a.hkv;
  TreeWalk<MT> walk;
  walk.pos = sm.start_pos;
  walk.left = n_tiles;
  walk.b = sm.start_b;
  walk.enter(a);
  int j = 0;      // tiles of the CTA so far
  int mine = 0;   // tiles of this row tile so far
  while (walk.next(a)) {
    if (MT > 1 && mt >= walk.m_tiles(a)) {
      j += walk.t1 - walk.t0;
      continue;
    }
    const int row = walk.mg * 128 * MT + mt * 128 + row_in;
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
    float m = -INFINITY, l = 0.f, ref = 1.f;
    uint64_t odd = 0;    // attended nodes whose V is not finite
    for (int ti = walk.t0; ti < walk.t1; ti++, j++, mine++) {
      const int buf = MT == 1 ? mine & 1 : mt;
      const uint32_t t_s = tmem + lanes + 128 * buf;
      // (a row tile that sat out a segment may have missed phases of mfull: S
      // first, whose phases are its own)
      if (!tree_wait_warp(sm, &sm.sfull[buf], (MT == 1 ? mine >> 1 : mine) & 1, a)) return;
      if (!tree_wait_warp(sm, &sm.mfull[j & (kTreeMeta - 1)], (j / kTreeMeta) & 1, a)) return;
      tc_fence_after();
      if (warp_live) {
        const TreeMeta &me = sm.meta[j & (kTreeMeta - 1)];
        const bool tail = ti >= cold_tiles;
        const int k0 = node0 + (ti - cold_tiles) * kTK;
        bool plain = true;  // every key attended, no negative scale: the maximum of S times the scale
        float vmax = 0.f;
#pragma unroll
        for (int c = 0; c < 4; c++) {
          plain &= tree_ok(me, c, tail, k0 + 32 * c, nodes, odd) == 0xffffffffu && me.k_scale[c] * a.qk_scale >= 0.f;
          vmax = fmaxf(vmax, fabsf(me.v_scale[c]));
        }
        plain = __all_sync(0xffffffffu, plain);
        float top = -INFINITY;
        uint32_t v[64];
#pragma unroll 1
        for (int h = 0; h < 2; h++) {
          tc_ld64(t_s + 64 * h, v);
          tc_wait_ld(v);
          const float s0 = me.k_scale[2 * h] * a.qk_scale, s1 = me.k_scale[2 * h + 1] * a.qk_scale;
          if (plain) {
            top = fmaxf(top, fmaxf(max_of<32>(v) * s0, max_of<32>(v + 32) * s1));
          } else {
            const uint32_t ok0 = tree_ok(me, 2 * h, tail, k0 + 64 * h, nodes, odd);
            const uint32_t ok1 = tree_ok(me, 2 * h + 1, tail, k0 + 64 * h + 32, nodes, odd);
#pragma unroll
            for (int k = 0; k < 32; k++) {
              if (ok0 >> k & 1) top = fmaxf(top, __uint_as_float(v[k]) * s0);
              if (ok1 >> k & 1) top = fmaxf(top, __uint_as_float(v[k + 32]) * s1);
            }
          }
        }
        // m and r follow when they lag too far behind; O and l follow them
        const bool first = ti == walk.t0;
        float r_new = ref;
        if (first || vmax > kLagScale * ref) r_new = vmax > 0.f ? vmax : ref;
        const float m_new = first || top > m + kLagLog2 ? fmaxf(m, top) : m;
        if (!first && __any_sync(0xffffffffu, m_new != m || r_new != ref)) {
          if (!tree_wait_warp(sm, &sm.odone[mt][(mine - 1) & 1], ((mine - 1) >> 1) & 1, a)) return;
          tc_fence_after();
          const float f = m == -INFINITY ? 0.f : ex2(m - m_new);
          l *= f;
          const float g = f * __fdividef(ref, r_new);
#pragma unroll 1
          for (int h = 0; h < 2; h++) {
            tc_ld64(t_o + 64 * h, v);
            tc_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 64; k++) v[k] = __float_as_uint(__uint_as_float(v[k]) * g);
            tc_st64(t_o + 64 * h, v);
          }
        }
        m = m_new;
        ref = r_new;
        const float base = m == -INFINITY ? 0.f : m;
        const float inv = __fdividef(1.f, ref);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int h = 0; h < 2; h++) {
          tc_ld64(t_s + 64 * h, v);
          tc_wait_ld(v);
          const float s0 = me.k_scale[2 * h] * a.qk_scale, s1 = me.k_scale[2 * h + 1] * a.qk_scale;
          const float f0 = me.v_scale[2 * h] * inv, f1 = me.v_scale[2 * h + 1] * inv;
#pragma unroll
          for (int k = 0; k < 64; k++)
            v[k] = __float_as_uint(ex2(fmaf(__uint_as_float(v[k]), k < 32 ? s0 : s1, -base)));
          if (!plain) {
            const uint32_t ok0 = tree_ok(me, 2 * h, tail, k0 + 64 * h, nodes, odd);
            const uint32_t ok1 = tree_ok(me, 2 * h + 1, tail, k0 + 64 * h + 32, nodes, odd);
#pragma unroll
            for (int k = 0; k < 32; k++) {
              if (!(ok0 >> k & 1)) v[k] = 0;
              if (!(ok1 >> k & 1)) v[k + 32] = 0;
            }
          }
          uint32_t p[32];
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            const float x = __uint_as_float(v[k]), y = __uint_as_float(v[k + 1]), f = k < 32 ? f0 : f1;
            sum[(k >> 1) & 3] += x + y;
            const __half2 w = __floats2half2_rn(x * f, y * f);
            p[k >> 1] = *reinterpret_cast<const uint32_t *>(&w);
          }
          tc_st32(t_s + 32 * h, p);
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
      const bool whole = walk.t0 == 0 && walk.t1 == walk.tiles;
      const float o_scale = whole ? (l != 0.f ? ref / l : 0.f) : ref;
      const size_t out_row = (static_cast<size_t>(walk.b) * a.max_tree + t) * a.hq + walk.hk * G + row - t * G;
      const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (walk.t0 == 0 ? 1 : 0);
      const int pr = mt * 128 + row_in;
#pragma unroll 1
      for (int h = 0; h < 2; h++) {
        uint32_t v[64];
        tc_ld64(t_o + 64 * h, v);
        tc_wait_ld(v);
#pragma unroll
        for (int k = 0; k < 64; k++) v[k] = __float_as_uint((l != 0.f ? __uint_as_float(v[k]) : 0.f) * o_scale);
        for (uint64_t rest = odd; rest; rest &= rest - 1) {
          const int node = __ffsll(static_cast<long long>(rest)) - 1;
          const __half *vr =
              a.v_tree + ((static_cast<size_t>(walk.b) * a.max_tree + node) * a.hkv + walk.hk) * kDim + 64 * h;
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            const __half2 x = *reinterpret_cast<const __half2 *>(vr + k);
            if (f16_not_finite(__half_as_ushort(x.x))) v[k] = __float_as_uint(__uint_as_float(v[k]) + __low2float(x));
            if (f16_not_finite(__half_as_ushort(x.y)))
              v[k + 1] = __float_as_uint(__uint_as_float(v[k + 1]) + __high2float(x));
          }
        }
        if (!live) continue;
        if (whole) {
#pragma unroll
          for (int k = 0; k < 64; k += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const __half2 x = __floats2half2_rn(__uint_as_float(v[k + 2 * e]), __uint_as_float(v[k + 2 * e + 1]));
              w[e] = *reinterpret_cast<const uint32_t *>(&x);
            }
            *reinterpret_cast<uint4 *>(a.out + out_row * kDim + 64 * h + k) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          uint4 *dst = reinterpret_cast<uint4 *>(a.part_o) + slot * 32 * 128 * MT;
#pragma unroll
          for (int k = 0; k < 64; k += 4)
            dst[(16 * h + (k >> 2)) * (128 * MT) + pr] = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
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
      // the list's index of the unit's last tile, and the run that has it
      const long long end = sm.total * blockIdx.x / ctas + j - (walk.t1 - walk.t0) + walk.tiles;
      const int last = static_cast<int>((end * ctas - 1) / sm.total);
      const int groups_max = (a.max_tree * G + 128 * MT - 1) / (128 * MT);
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
  constexpr int kMmaWarp = Shape::kSoftWarps + Shape::kProducers;

  // the list's length and where this CTA's run starts: every thread sums a
  // range of sequences, a scan over the threads places them
  const int per = (a.batch + Shape::kThreads - 1) / Shape::kThreads;
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
      mbar_init(&sm.kfull[i], Shape::kProducers);
      mbar_init(&sm.kempty[i], 1);
      mbar_init(&sm.vfull[i], Shape::kProducers);
      mbar_init(&sm.vempty[i], 1);
    }
    for (int i = 0; i < kTreeMeta; i++) mbar_init(&sm.mfull[i], Shape::kProducers);
    for (int i = 0; i < TreeSmem<MT>::kQ; i++) {
      mbar_init(&sm.qfull[i], Shape::kProducers);
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

  if (warp < Shape::kSoftWarps) {
    tree_softmax<MT>(a, sm, tmem, n_tiles);
  } else if (warp < kMmaWarp) {
    tree_produce<MT, kF16>(a, sm, q_s, k_s, v_s, n_tiles);
  } else {
    if (lane == 0) {
      tree_mma<MT>(a, sm, q_s, k_s, v_s, tmem, n_tiles);
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
