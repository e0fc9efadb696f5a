// tree.cu -- hyb_tree_attn: attention of drafted tree nodes over the cache, on
// the fifth-generation tensor cores.
//
// Mathematics.  The nt nodes of a sequence and the G query heads of a kv head
// make M = nt G query rows that share their keys, up to the tree's mask.  Per
// 128-key tile: S = Q K^T, the online softmax (running maximum m, sum l) and
// O += P V.  INT8 / INT4 codes are integers that FP16 holds exactly, so K and
// V enter the products as codes: a tile's K scale multiplies its logits, its V
// scale the weights, both in FP32.  The weights p s_v / r are rounded once to
// FP16 (the tensor core takes no FP32 operand): half a step, 2^-11 relative, or
// 2^-25 where p s_v / r is below 2^-14.  r is the tile's largest V scale where it
// was set last (0 while all are 0), so that the FP16 range serves weights, not
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
// Inside a CTA (20 warps): a scout warp looks the tiles up (block table, scales,
// segment ends) some tiles ahead, writes their records and fetches the query
// rows; the lanes of a copy warp bring their bytes into rings in shared memory by
// bulk copies; four producer warps turn K, four V, from codes or rows into FP16 in
// the 128-byte swizzled layout of the MMA's shared operands; two MMA warps issue
// the products; two groups of four softmax warps (one query row per thread) keep
// two softmax streams and write the weights over the logits in TMEM, where the
// second product reads them as its A operand.  The streams are the two row tiles
// (MT 2, with an MMA warp each), or the two halves of every tile's keys (MT 1),
// merged at a unit's end: then a tile's softmax is 64 keys per thread, and S has
// two buffers, so that Q K^T of the next tile (one MMA warp) runs behind it and
// P V of the last one (the other).
//
// What bounds it (us with the L2 flushed before each call; "long": 4 sequences of
// 32768 .. 131072 tokens, 32 nodes, 32 heads, 8 kv heads: 242; "short trees": 64
// sequences of 256 .. 8192 tokens, 8 nodes: 314; "wide": 8 of 16384 tokens, 64
// nodes, 64 heads: 383).  No unit is busy most of the time: of long's 242 us the
// bytes need 101 and the products 103.  In SM cycles, by a clock read per tile (the
// SMs run at about 1840 MHz inside a call, at 1600 .. 1750 when long calls follow
// each other under the power limit):
//   a cold tile: 2450 (32 query rows) .. 2640 (128), with INT4 among them 2760, of
//   FP16 rows 4000, MT 2 5550.  The first is the softmax warps' path from one tile
//   to the next: two warps' powers of two take 1120, and the waits, records, the
//   TMEM round trip and the arrival about 1400 whatever the rows and keys are
//   the end of a unit: its tail tile 11000 .. 13500 (the ring and the nodes are
//   loaded when its turn has come), the next unit's first tile 5700 .. 6600
//   a call's begin: 4500 until the roles start, 15000 until the first weights
//   (18500 with the L2 flushed); the merge: 1 us behind the last CTA, 5 .. 9 us long
// Runs are cut by tiles, not by time: short trees' runs have 2 .. 16 ends of units,
// and half of the CTAs are done after 196 of the 297 us that the last one takes
// (long: 208 of 223).  Instruction supply bounded it before, as six roles share an
// SM's instruction cache: with 110 KB of unrolled code 31% of the requests missed and
// a stall for instructions was the commonest (long 372; as loops, 86 KB: 285).  What
// was tried:
//   a lane per ring piece issues the copies, instead of one thread: long 283 -> 261
//   64 logits stay in registers between maximum and weights (MT 1): long 262 -> 247
//   K and V producers share their code: short trees 354 -> 342
//   120 / 72 registers for softmax / producers, not 112 / 80: short trees 330 -> 315
//   four MMA steps per loop turn, not one: wide 450 -> 422
//   one test per tile whether maximum and reference may stay: long 248 -> 241
//   a quarter of the powers of two by a polynomial: long 248 -> 252, not kept
//   up to 64 rows twice in the tile, half the keys for each: short trees 289 -> 302
//   (the fixed part stays, the second Q buffer goes), not kept
//   rings of two pieces instead of three: codes the same, FP16 rows 85 -> 90
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
constexpr uint32_t kPiece = 8192;            // of the rings of codes or rows
constexpr float kLagLog2 = 6.f;
constexpr float kLagScale = 256.f;

// Warps: softmax, producers, MMA, scout, copies: 20 warps of 96 registers at
// launch; the softmax warps take what the producers do not need.
constexpr int kTreeSoft = 8, kTreeProd = 8, kTreeMma = 2;
constexpr int kTreeThreads = 32 * (kTreeSoft + kTreeProd + kTreeMma + 2);
constexpr int kTreeSoftRegs = 120, kTreeProdRegs = 72;

// TreeRec::flags: the first and the last tile of its segment (the part of a unit
// that this CTA has); every key attended by every row and no
// negative scale; cold (not ring and nodes); the segment has the unit's first,
// its last tile; the segment's number modulo 4
constexpr uint32_t kTileFirst = 1, kTileLast = 2, kTilePlain = 4, kTileCold = 8, kUnitStart = 16, kUnitEnd = 32;
constexpr int kTileSegShift = 6;

// A tile of 128 keys in four units of 32, as the scout found it.
struct TreeRec {
  const uint8_t *at[4];  // cold: the unit's 64-token tile pair (FP16: its first row); null: no keys
  float k_scale[4];      // 1 for FP16 rows
  float v_scale[4];
  uint32_t ok[4];        // keys that every row attends
  uint32_t bad[4][4];    // [V warp][unit]: keys of a tail tile with a V that is not finite (by the producers)
  uint32_t fmt;          // bit c: unit c is INT4; bit 4 + c: it is the second half of its slots
  uint32_t flags;
  float v_max;           // largest |v_scale|
  int rest;              // tiles of the unit after the segment
  int b, hk, mg;         // the unit's sequence, kv head and row group
  int rows;              // query rows of the sequence and kv head
  // tail: its first row (ring rows in the order of their positions, then
  // nodes), the cold and ring tokens and the nodes; the ring and the nodes' K, V
  int row0, cold, hot, keys;
  const __half *ring, *node[2];
};

// A stream's row at a segment's end (MT 1).
struct TreeStat {
  float m, l, ref;
  uint64_t odd;
};

template <int MT>
struct TreeSmem {
  // pieces of 8192 bytes: a ring of codes of K and one of V, or one of FP16 rows
  static constexpr int kPieces = MT == 1 ? 6 : 4;
  // MMA operands (MT 2: both MMA warps free a stage)
  uint64_t kfull[kTreeStages], kempty[kTreeStages], vfull[kTreeStages], vempty[kTreeStages];
  uint64_t cfull[kPieces], cempty[kPieces];
  uint64_t rfull[2], rfree[2];     // records, by batch parity
  uint64_t mfull[kTreeRecs];       // a record's tile is in shared memory
  uint64_t qfull[2], qempty[2];
  uint64_t sfull[2];               // MT 1: by S buffer; MT 2: by stream
  uint64_t pfull[2][2];            // by stream and (MT 1) S buffer
  uint64_t odone[2], ofree[2];     // by stream
  uint64_t xfull;                  // MT 1: both streams' rows are in `stat`
  uint64_t drain[2];
  TreeRec rec[kTreeRecs];
  uint32_t tmem;
  volatile int abort;
  int start_b;
  long long start_pos, total;      // the run's start within sequence start_b; the list's length
  long long warp_sum[32];
  TreeStat stat[MT == 1 ? 2 : 1][MT == 1 ? 2 : 1][MT == 1 ? 128 : 1];  // [parity][stream][row]
};

// Shared memory: Q, K stages, V stages, pieces, the rest.  MT 1: two buffers of
// 64 query rows or one of 128 (an MMA reads 128 rows from either: what follows
// in shared memory makes rows that nobody reads).
template <int MT>
struct TreeShape {
  static constexpr uint32_t kQBytes = MT * kTreeOperand;
  static constexpr uint32_t kTiles = kQBytes + 2 * kTreeStages * kTreeOperand;
  static constexpr uint32_t kBytes = kTiles + TreeSmem<MT>::kPieces * kPiece + sizeof(TreeSmem<MT>);
  static_assert(kBytes <= 232448, "shared memory of an SM");
};

// ---- the list of tiles ----

struct TreeSeq {
  int cold, hot, nt, keys;  // cold and ring tokens, nodes (rows), nodes that are keys
  int tiles, groups;        // per unit; row groups
  int status;
};

// ceil(tokens / 128), also where the sum with 127 would pass 32 bits
__device__ __forceinline__ int tiles_of(int tokens) { return tokens / kTK + (tokens % kTK != 0); }

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
  s.tiles = max(1, tiles_of(s.cold) + tiles_of(s.hot + s.keys));
  s.groups = (s.nt * a.group + 128 * MT - 1) / (128 * MT);
  return s;
}

// Wait for phase `parity`; false when the wait or the kernel gave up.  By a whole
// warp, with one answer.  Small, as it stands at many places.
template <typename Sm>
__device__ __forceinline__ bool tree_wait(Sm &sm, uint64_t *bar, uint32_t parity, const TreeArgs &a) {
  uint32_t t0 = 0;
#pragma unroll 1
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint32_t t = static_cast<uint32_t>(clock()) | 1;
    if (t0 == 0) t0 = t;
    if (__any_sync(0xffffffffu, sm.abort || t - t0 > a.wait_cycles)) break;
  }
  sm.abort = 1;
  return false;
}

// The node of a query row: row / (Hq / Hkv), by a multiplication that is exact
// for rows below 2^13 (there are at most 64 * 8).
__device__ __forceinline__ int row_node(const TreeArgs &a, int row) { return (row * a.group_recip) >> 16; }

__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
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

// Codes as FP16: a byte u = code + 2^(bits-1) under the exponent of 1024 is 1024
// + u, and the subtraction of 1024 + 2^(bits-1) is exact.  `flip` takes a code's
// byte to u.
struct TreeCodec {
  uint32_t flip, off;
  __device__ __forceinline__ explicit TreeCodec(bool int4)
      : flip(int4 ? 0x08080808u : 0x80808080u), off(int4 ? 0x64086408u : 0x64806480u) {}
  __device__ __forceinline__ uint32_t two(uint32_t x, uint32_t sel) const {
    const uint32_t h = __byte_perm(x, 0x64646464u, sel);
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&off));
    return *reinterpret_cast<const uint32_t *>(&d);
  }
  __device__ __forceinline__ uint4 eight(uint32_t w0, uint32_t w1) const {
    w0 ^= flip;
    w1 ^= flip;
    return make_uint4(two(w0, 0x4140), two(w0, 0x4342), two(w1, 0x4140), two(w1, 0x4342));
  }
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Sixteen codes, INT8 or (of eight bytes, code e of a word the low nibble of byte
// e, e + 4 the high nibble) INT4, to two neighbouring 16-byte chunks `to`, `to` ^ 16.
__device__ __forceinline__ void put16(const TreeCodec &f, uint4 x, uint32_t to) {
  sts128(to, f.eight(x.x, x.y));
  sts128(to ^ 16, f.eight(x.z, x.w));
}
__device__ __forceinline__ uint4 get16(bool int4, uint32_t from) {
  if (!int4) return lds128(from);
  const uint2 y = lds64(from);
  const uint32_t m = 0x0f0f0f0fu;
  return make_uint4(y.x & m, y.x >> 4 & m, y.y & m, y.y >> 4 & m);
}

// Rows are read once: no place in L1.
__device__ __forceinline__ uint4 ldg16(const void *p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ bool f16_not_finite(uint32_t h) { return (h & 0x7c00u) == 0x7c00u; }

// The K row (kv 1: V row) of row i of a tail tile (ring rows in the order of
// their positions, then nodes), or null.
__device__ __forceinline__ const __half *tail_row(const TreeArgs &a, const TreeRec &r, int i, int kv) {
  i += r.row0;
  if (i < r.hot) return r.ring + (2 * ((r.cold + i) & (a.hot_tokens - 1)) + kv) * kDim;
  return i - r.hot < r.keys ? r.node[kv] + static_cast<size_t>(i - r.hot) * a.hkv * kDim : nullptr;
}

// A tail tile's K: one row per thread; eight lanes are eight rows.
__device__ __forceinline__ void tail_k(const TreeArgs &a, const TreeRec &r, uint32_t kst, int tid) {
  const __half *p = tail_row(a, r, tid, 0);
#pragma unroll 1
  for (int q = 0; q < 4; q++) {
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] = p ? ldg16(p + 32 * q + 8 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; j++)
      sts128(kst + (q >> 1) * kTreeSlab + tid * 128 + (((4 * (q & 1) + j) ^ (tid & 7)) << 4), x[j]);
  }
}

// Two channels (2 pair, + 1) of eight keys (words w) to a chunk of the channels'
// rows.  Lanes 4..7 of eight write their odd row first, so that the eight rows
// differ modulo 8.
__device__ __forceinline__ void put_v(uint32_t vst, int pair, int key, const uint32_t *w) {
  const int odd = (pair >> 2) & 1;
#pragma unroll
  for (int s = 0; s < 2; s++) {
    const int hi = s ^ odd, row = 2 * pair + hi, sel = hi ? 0x7632 : 0x5410;
    sts128(vst + (key >> 6) * kTreeSlab + row * 128 + (((key >> 3 & 7) ^ (row & 7)) << 4),
           make_uint4(__byte_perm(w[0], w[1], sel), __byte_perm(w[2], w[3], sel), __byte_perm(w[4], w[5], sel),
                      __byte_perm(w[6], w[7], sel)));
  }
}

// A tail tile's V: two channels of 16 of every unit's keys per thread.  Lane k
// knows key k's row.
__device__ __forceinline__ void tail_v(const TreeArgs &a, TreeRec &r, uint32_t vst, int tid) {
  const int lane = tid & 31, k0 = 16 * (tid >> 6), pair = tid & 63;
#pragma unroll 1
  for (int u = 0; u < 4; u++) {
    const uint64_t mine = reinterpret_cast<uint64_t>(tail_row(a, r, 32 * u + lane, 1));
    uint32_t bad = 0;
#pragma unroll 1
    for (int k8 = k0; k8 < k0 + 16; k8 += 8) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const uint64_t p = __shfl_sync(0xffffffffu, mine, k8 + k);
        w[k] = p ? __ldg(reinterpret_cast<const uint32_t *>(reinterpret_cast<const __half *>(p) + 2 * pair)) : 0u;
      }
      // A node's V that is not finite must not meet the zero weight of a row that
      // does not attend the node: it becomes 0 here and the record names the
      // node; the rows that do attend it add it at the end
      const int ring = r.hot - (r.row0 + 32 * u + k8);  // ring rows among the eight
#pragma unroll
      for (int k = 0; k < 8; k++) {
        uint32_t nf = ((w[k] & 0x7fff7fffu) + 0x04000400u) & 0x80008000u;  // bit 15 of a half: its exponent is all ones
        if (k < ring) nf = 0;
        w[k] &= ~((nf >> 15) * 0xffffu);
        bad |= nf ? 1u << (k8 + k) : 0u;
      }
      put_v(vst, pair, 32 * u + k8, w);
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (lane == 0) r.bad[tid >> 5][u] = bad;
  }
}

// Both groups run the same code where they can (the instruction cache holds it
// once): kv 0 makes K, 1 makes V.
template <int MT, bool kF16>
__device__ __forceinline__ void tree_produce(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t st, uint32_t c_s, int kv, int n) {
  const int tid = threadIdx.x & 127, lane = tid & 31;
  uint64_t *full = kv ? sm.vfull : sm.kfull, *empty = kv ? sm.vempty : sm.kempty;
  const bool small = a.bshift == 5;
  // the pieces: of FP16 rows both groups take all, of codes each its ring's
  constexpr int kRing = kF16 ? TreeSmem<MT>::kPieces : TreeSmem<MT>::kPieces / 2;
  const int first = !kF16 && kv ? kRing : 0;
  int at = 0;
  uint32_t turn = 0;  // modulo 2
  auto piece_done = [&]() {
    warp_arrive(&sm.cempty[first + at], lane);
    if (++at == kRing) {
      at = 0;
      turn ^= 1;
    }
  };
  // K: the thread's keys (8 i and this one of a unit) and its 16 channels.
  // Eight lanes are channels 0..63 of one key and 64..127 of the next: all
  // banks of both the piece and (as neighbouring rows of different slabs) the
  // operand
  const int hi = (tid >> 2) & 1, key = 2 * (tid >> 4) + hi, ch16 = (tid & 3) + 4 * (hi ^ ((tid >> 3) & 1));
  // V: channel tid / 4 and 32, 64, 96 more, 16-slot chunk position tid % 4 of a
  // 64-token tile; eight lanes are two channels of four chunks
  const int v_ch = tid >> 2, v_pos = tid & 3;
  // INT8: where the thread's 16 codes are in a piece, and go in the operand
  // (the next: 2048 bytes on, and a quarter of the piece's part of the operand:
  // 64 keys of K, 64 columns of V)
  const uint32_t from8 = kv ? tid * 16 : key * 128 + ch16 * 16;
  const uint32_t to8 = kv ? v_ch * 128 + (((2 * (v_pos ^ (v_ch >> 1 & 3))) ^ (v_ch & 7)) << 4)
                          : (ch16 >> 2) * kTreeSlab + key * 128 + (((2 * (ch16 & 3)) ^ (key & 7)) << 4);
  const uint32_t part = kv ? kTreeSlab : kTreeSlab / 2;

#pragma unroll 1
  for (int j = 0; j < n; j++) {
    const int s = j & (kTreeStages - 1);
    const uint32_t ph = (j / kTreeStages) & 1, to = st + s * kTreeOperand;
    if (j % kTreeBatch == 0) {
      const int batch = j / kTreeBatch;
      if (!tree_wait(sm, &sm.rfull[batch & 1], (batch >> 1) & 1, a)) return;
    }
    TreeRec &r = sm.rec[j & (kTreeRecs - 1)];
    const bool cold = r.flags & kTileCold;
    const uint32_t fmt = r.fmt;
    if (!tree_wait(sm, &empty[s], ph ^ 1, a)) return;
    if (!cold) {
      if (kv) tail_v(a, r, to, tid);
      else tail_k(a, r, to, tid);
    } else {
      // FP16: pieces of 16 rows of K and V.  Codes: two pieces of two units; of
      // V with 32-token blocks four of one.
      const int pieces = kF16 ? 8 : kv && small ? 4 : 2;
#pragma unroll 1
      for (int p = 0; p < pieces; p++) {
        if (!tree_wait(sm, &sm.cfull[first + at], turn, a)) return;
        const uint32_t c = c_s + (first + at) * kPiece;
        if constexpr (kF16) {
          if (kv) {
            const int pair = tid & 63, rows = 8 * (tid >> 6);
            const uint32_t ok = r.ok[p >> 1] >> (16 * (p & 1) + rows);
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; k++) w[k] = lds32(c + (rows + k) * 512 + 256 + 4 * pair);
#pragma unroll
            for (int k = 0; k < 8; k++)  // (keys that are not there may hold anything)
              if (!(ok >> k & 1)) w[k] = 0;
            put_v(to, pair, 16 * p + rows, w);
          } else {
#pragma unroll
            for (int i = 0; i < 2; i++) {
              const int row = (tid >> 4) + 8 * i, c16 = tid & 15;
              sts128(to + (c16 >> 3) * kTreeSlab + (16 * p + row) * 128 + (((c16 & 7) ^ (row & 7)) << 4),
                     lds128(c + row * 512 + c16 * 16));
            }
          }
        } else if ((fmt & 15) == 0 && pieces == 2) {
          const TreeCodec f(false);
          uint4 x[4];
#pragma unroll
          for (int k = 0; k < 4; k++) x[k] = lds128(c + from8 + 2048 * k);
#pragma unroll
          for (int k = 0; k < 4; k++) put16(f, x[k], to + to8 + p * part + (k * part >> 2));
        } else {
#pragma unroll 1
          for (int i = 0; i < 4; i++) {
            uint32_t from, dst;
            bool int4, there = true;
            if (!kv) {
              int4 = fmt >> (2 * p + i / 2) & 1;
              from = 4096 * (i / 2) + (key + 16 * (i & 1)) * (int4 ? 64 : 128) + ch16 * (int4 ? 8 : 16);
              dst = to8 + p * part + i * (part >> 2);
            } else {
              // 64-slot tiles of a pair of units, or (32-token blocks) of one,
              // whose slots 0..31 are its tokens
              int4 = fmt >> (small ? p : 2 * p) & 1;
              const int ch = v_ch + 32 * i, chunk = v_pos ^ (ch >> (int4 ? 2 : 1) & 3);  // slots 16 chunk ..
              const int c8 = small ? 4 * (p & 1) + 2 * chunk : 2 * chunk;
              there = !small || chunk < 2;
              from = int4 ? ch * 32 + v_pos * 8 : ch * 64 + v_pos * 16;
              dst = (small ? p >> 1 : p) * kTreeSlab + ch * 128 + ((c8 ^ (ch & 7)) << 4);
            }
            if (there) put16(TreeCodec(int4), get16(int4, c + from), to + dst);
          }
        }
        piece_done();
      }
    }
    warp_arrive(&full[s], lane);
    // the record is ready for the softmax: with V's part of a tail tile
    if (kv == !cold && lane == 0) mbar_arrive(&sm.mfull[j & (kTreeRecs - 1)]);
  }
}

// ---- the copy warp ----

// (bulk_g2s of common.cuh with the shared address as a number)
__device__ __forceinline__ void bulk_to(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// Lane i of one warp fills piece i of the rings, over and over, as soon as it is
// free: per tile K of two units (4096 bytes apart) and of the other two in one
// ring, their V tiles (32-token blocks: one per unit) in the other; FP16 rows 16
// at a time in one ring.  Side by side, as a single thread takes longer to
// issue a copy (about 900 cycles with all it looks up) than the copies last.
template <int MT, bool kF16>
__device__ __forceinline__ void tree_copy(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t c_s, int n, int piece) {
  constexpr int kRing = kF16 ? TreeSmem<MT>::kPieces : TreeSmem<MT>::kPieces / 2;
  const uint64_t policy = l2_policy_evict_first();
  const bool is_v = piece >= kRing, small = a.bshift == 5;
  const int pieces = kF16 ? 8 : is_v && small ? 4 : 2;  // of the ring per tile
  const uint32_t to = c_s + piece * kPiece;
  uint64_t *full = &sm.cfull[piece], *empty = &sm.cempty[piece];
  int j = 0, p = is_v ? piece - kRing : piece;  // the tile and its piece to bring next
  uint32_t turn = 0, t0 = 0;                    // modulo 2; when the lane began to wait
#pragma unroll 1
  while (j < n) {
    const TreeRec &r = sm.rec[j & (kTreeRecs - 1)];
    const int batch = j / kTreeBatch;
    bool ready = mbar_test_wait(&sm.rfull[batch & 1], (batch >> 1) & 1);
    const bool skip = ready && (p >= pieces || !(r.flags & kTileCold));
    ready = ready && !skip && mbar_test_wait(empty, turn ^ 1);
    if (skip) {
      if (r.flags & kTileCold) p -= pieces;
      if (++j % kTreeBatch == 0) mbar_arrive(&sm.rfree[batch & 1]);
    }
    if (ready) {
      const uint8_t *src, *src1 = nullptr;
      uint32_t bytes, bytes1 = 0;
      if constexpr (kF16) {
        src = r.at[p >> 1];
        bytes = src ? kPiece : 0;
        src += (p & 1) * kPiece;
      } else {
        const int u = pieces == 4 ? p : 2 * p;
        const uint32_t f = r.fmt >> u;
        src = r.at[u];
        bytes = !src ? 0 : f & 1 ? 2048 : 4096;
        if (is_v) {  // the whole V tile
          src += kTileBytes;
          bytes *= 2;
        } else {     // K of units u and u + 1
          src1 = r.at[u + 1];
          bytes1 = !src1 ? 0 : f & 2 ? 2048 : 4096;
          if (src == src1 && bytes == 4096) {  // the two halves of an INT8 tile are one run
            bytes = kPiece;
            bytes1 = 0;
          } else {
            if (f & 16) src += bytes;
            if (f & 32) src1 += bytes1;
          }
        }
      }
      mbar_arrive_expect_tx(full, bytes + bytes1);
      if (bytes) bulk_to(to, src, bytes, full, policy);
      if (!kF16 && bytes1) bulk_to(to + 4096, src1, bytes1, full, policy);
      p += kRing;
      turn ^= 1;
    }
    if (ready || skip) {
      t0 = 0;
    } else {
      const uint32_t t = static_cast<uint32_t>(clock()) | 1;
      if (t0 == 0) t0 = t;
      if (sm.abort || t - t0 > a.wait_cycles) {
        sm.abort = 1;
        break;
      }
    }
  }
  // the copies in flight land before the CTA ends, also when nobody takes them
  // (before the first copy nothing is in flight, and parity 1 is done)
  mbar_wait_bounded(full, turn ^ 1, kDefaultWaitCycles);
}

// ---- the scout ----

// The query rows of a unit on their way into its Q operand(s) (rows beyond the
// tree keep what they were: nobody reads their results).
template <int MT>
__device__ __forceinline__ void fetch_q(const TreeArgs &a, int b, int hk, int mg, int rows, uint32_t st, int lane) {
  const int G = a.group, n = min(128 * MT, rows - mg * 128 * MT), c = lane & 15;
  const __half *q = a.q + (static_cast<size_t>(b) * a.max_tree * a.hq + hk * G) * kDim + 8 * c;
  const uint32_t slab = MT == 1 ? a.q_rows * 128 : kTreeSlab, to = st + (c >> 3) * slab;
#pragma unroll 2
  for (int r = lane >> 4; r < n; r += 2) {
    const int row = mg * 128 * MT + r, t = row_node(a, row);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     to + (r >> 7) * kTreeOperand + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4)),
                 "l"(q + (static_cast<size_t>(t) * a.hq + row - t * G) * kDim)
                 : "memory");
  }
}

// Lane 4 k + c looks up unit c of tile k of a batch.
template <int MT, bool kF16>
__device__ __forceinline__ void tree_scout(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t q_s, int n) {
  const int lane = threadIdx.x & 31, k = (lane >> 2) & (kTreeBatch - 1), c = lane & 3;
  const bool on = lane < 4 * kTreeBatch;
  int b = sm.start_b, segs = 0;     // segments begun before the batch
  TreeSeq q = tree_seq<MT>(a, b);
  // the lane's tile: tile t of row group mg of kv head hk
  int t = static_cast<int>(sm.start_pos % q.tiles), hk = static_cast<int>(sm.start_pos / q.tiles), mg = hk % q.groups;
  hk /= q.groups;
  t += k;

#pragma unroll 1
  for (int j0 = 0, batch = 0; j0 < n; j0 += kTreeBatch, batch++) {
    const int j = j0 + k;
    const bool have = on && j < n;
    if (have) {
#pragma unroll 1
      while (t >= q.tiles) {
        t -= q.tiles;
        if (++mg < q.groups) continue;
        mg = 0;
        if (++hk < a.hkv) continue;
        hk = 0;
#pragma unroll 1
        do q = tree_seq<MT>(a, ++b);
        while (q.groups == 0);
      }
    }
    const int in = min(t, j);                        // tiles of the segment before this one
    const int left = min(q.tiles - 1 - t, n - 1 - j);  // and after it
    const uint32_t firsts = __ballot_sync(0xffffffffu, have && in == 0 && c == 0);
    const int seg = segs + __popc(firsts & (0xffffffffu >> (31 - (4 * k)))) - 1;
    const int rows = q.nt * a.group;

    const int cold_tiles = tiles_of(q.cold);
    const bool cold = t < cold_tiles;
    const int p = cold ? t * kTK + 32 * c : 0;  // the unit's first position
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
        } else {
          at = a.cold + ((i << a.lsub) + (slot >> 6)) * kTilePairBytes;
          sc = __ldg(reinterpret_cast<const float2 *>(a.scales) + i);
          if (a.quant_bits == 4 || (a.n_int4 != nullptr && block < a.n_int4[b])) fmt |= 1;
          if (slot & 32) fmt |= 16;
        }
      }
    }
    // (an empty unit has no say in the reference scale)
    if (!kF16 && cold && valid == 0) sc = make_float2(0.f, 0.f);
    const int row0 = (t - cold_tiles) * kTK;
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
    if (!tree_wait(sm, &sm.rfree[batch & 1], ((batch >> 1) & 1) ^ 1, a)) return;
    if (have) {
      TreeRec &r = sm.rec[j & (kTreeRecs - 1)];
      r.at[c] = at;
      r.k_scale[c] = sc.x;
      r.v_scale[c] = sc.y;
      r.ok[c] = ok;
      if (c == 0) {
        r.fmt = fmt;
        r.v_max = v_max;
        r.flags = (in == 0 ? kTileFirst : 0) | (left == 0 ? kTileLast : 0) |
                  (plain ? kTilePlain : 0) | (cold ? kTileCold : 0) | (t <= j ? kUnitStart : 0) |
                  (left == q.tiles - 1 - t ? kUnitEnd : 0) | static_cast<uint32_t>(seg & 3) << kTileSegShift;
        r.rest = q.tiles - 1 - t - left;
        r.b = b;
        r.hk = hk;
        r.mg = mg;
        r.rows = rows;
        r.row0 = row0;
        r.cold = q.cold;
        r.hot = q.hot;
        r.keys = q.keys;
        r.ring = reinterpret_cast<const __half *>(a.hot) + (static_cast<size_t>(b) * a.hkv + hk) * a.hot_tokens * 2 * kDim;
        const size_t first_node = (static_cast<size_t>(b) * a.max_tree * a.hkv + hk) * kDim;
        r.node[0] = a.k_tree + first_node;
        r.node[1] = a.v_tree + first_node;
      }
    }
    warp_arrive(&sm.rfull[batch & 1], lane);
    // the segments that begin in this batch: their query rows
    for (uint32_t f = firsts; f; f &= f - 1, segs++) {
      const int s = segs;
      const int from = __ffs(f) - 1, i = a.q_bufs == 2 ? s & 1 : 0;
      const int fb = __shfl_sync(0xffffffffu, b, from), fhk = __shfl_sync(0xffffffffu, hk, from);
      const int fmg = __shfl_sync(0xffffffffu, mg, from), frows = __shfl_sync(0xffffffffu, rows, from);
      // (the buffer's last segment: a.q_bufs ago)
      const uint32_t turn = a.q_bufs == 2 ? s >> 1 : s;
      if (!tree_wait(sm, &sm.qempty[i], (turn & 1) ^ 1, a)) return;
      fetch_q<MT>(a, fb, fhk, fmg, frows, q_s + i * 256 * a.q_rows, lane);
      // one arrival per lane when its rows are there
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&sm.qfull[i])) : "memory");
    }
    t += kTreeBatch;
  }
}

// ---- the MMA warps (one elected thread issues) ----
// TMEM columns: O of stream i at 256 + 128 i.  MT 1: S of tile j at 128 (j % 2),
// its halves of 64 keys the streams'.  MT 2: S of stream i at 128 i.  The weights
// (FP16) replace the first half of the stream's columns of S.

// (Four steps at a time: all eight do not pay for their code.)
__device__ __forceinline__ void issue_qk(uint32_t t_s, uint32_t q, uint32_t q_slab, uint32_t k) {
  uint32_t dq = tc_desc_low(q), dk = tc_desc_low(k);
#pragma unroll 4
  for (int i = 0; i < 8; i++) {
    tc_mma_ss(t_s, dq, dk, tc_idesc_f16(128), i > 0);
    dq += i == 3 ? (q_slab >> 4) - 6 : 2;
    dk += i == 3 ? (kTreeSlab >> 4) - 6 : 2;
  }
}

// 64 keys
__device__ __forceinline__ void issue_pv(uint32_t t_o, uint32_t t_p, uint32_t v, bool first) {
  const uint32_t dv = tc_desc_low(v);
#pragma unroll
  for (int i = 0; i < 4; i++) tc_mma_ts(t_o, t_p + 8 * i, dv + 2 * i, tc_idesc_f16(128), !first || i > 0);
}

// MT 1: a warp for Q K^T and one for P V.
__device__ __forceinline__ void tree_mma_qk(const TreeArgs &a, TreeSmem<1> &sm, uint32_t q_s, uint32_t k_s, uint32_t tmem,
                                            int n) {
#pragma unroll 1
  for (int j = 0; j < n; j++) {
    const int s = j & 1;
    const uint32_t ph = (j >> 1) & 1;
    if (!tree_wait(sm, &sm.kfull[s], ph, a)) return;
    const uint32_t flags = sm.rec[j & (kTreeRecs - 1)].flags, seg = flags >> kTileSegShift & 3;
    const int qb = a.q_bufs == 2 ? seg & 1 : 0;
    if ((flags & kTileFirst) && !tree_wait(sm, &sm.qfull[qb], (a.q_bufs == 2 ? seg >> 1 : seg) & 1, a)) return;
    // S replaces the weights of tile j - 2: their P V is done
    if (!tree_wait(sm, &sm.vempty[s], ph ^ 1, a)) return;
    fence_proxy_async_smem();
    tc_fence_after();
    if (tc_elect()) {
      issue_qk(tmem + 128 * s, q_s + qb * 256 * a.q_rows, a.q_rows * 128, k_s + s * kTreeOperand);
      tc_commit(&sm.sfull[s]);
      tc_commit(&sm.kempty[s]);
      if (flags & kTileLast) tc_commit(&sm.qempty[qb]);
      if ((j + 1) % kTreeBatch == 0) mbar_arrive(&sm.rfree[(j / kTreeBatch) & 1]);
    }
    __syncwarp();
  }
}

__device__ __forceinline__ void tree_mma_pv(const TreeArgs &a, TreeSmem<1> &sm, uint32_t v_s, uint32_t tmem, int n) {
  int begun = 0;  // segments
#pragma unroll 1
  for (int j = 0; j < n; j++) {
    const int s = j & 1;
    const uint32_t ph = (j >> 1) & 1;
    if (!tree_wait(sm, &sm.vfull[s], ph, a)) return;
    const uint32_t flags = sm.rec[j & (kTreeRecs - 1)].flags;
    const bool first = flags & kTileFirst;
#pragma unroll 1
    for (int i = 0; i < 2; i++) {
      if (first && !tree_wait(sm, &sm.ofree[i], (begun & 1) ^ 1, a)) return;
      if (!tree_wait(sm, &sm.pfull[i][s], ph, a)) return;
      fence_proxy_async_smem();
      tc_fence_after();
      if (tc_elect()) {
        issue_pv(tmem + 256 + 128 * i, tmem + 128 * s + 64 * i, v_s + s * kTreeOperand + i * kTreeSlab, first);
        if (flags & kTileLast) tc_commit(&sm.odone[i]);
        if (i == 1) {
          tc_commit(&sm.vempty[s]);
          if ((j + 1) % kTreeBatch == 0) tc_commit(&sm.rfree[(j / kTreeBatch) & 1]);
        }
      }
      __syncwarp();
    }
    if (first) begun++;
  }
}

// MT 2: a warp for each row tile i; S of the next tile replaces the weights of
// this one.
__device__ __forceinline__ void tree_mma2(const TreeArgs &a, TreeSmem<2> &sm, uint32_t q_s, uint32_t k_s, uint32_t v_s,
                                          uint32_t tmem, int n, int i) {
  const uint32_t t_s = tmem + 128 * i, t_o = tmem + 256 + 128 * i;
  int begun = 0;  // segments
  for (int j = 0; j < n; j++) {
    const int s = j & 1;
    const uint32_t ph = (j >> 1) & 1;
    if (!tree_wait(sm, &sm.kfull[s], ph, a)) return;
    const uint32_t flags = sm.rec[j & (kTreeRecs - 1)].flags;
    const bool first = flags & kTileFirst;
    if (first && !tree_wait(sm, &sm.qfull[0], begun & 1, a)) return;
    fence_proxy_async_smem();
    tc_fence_after();
    if (tc_elect()) {
      issue_qk(t_s, q_s + i * kTreeOperand, kTreeSlab, k_s + s * kTreeOperand);
      tc_commit(&sm.sfull[i]);
      tc_commit(&sm.kempty[s]);
      if (flags & kTileLast) tc_commit(&sm.qempty[0]);
    }
    __syncwarp();
    if (first) {
      if (!tree_wait(sm, &sm.ofree[i], (begun & 1) ^ 1, a)) return;
      begun++;
    }
    if (!tree_wait(sm, &sm.vfull[s], ph, a)) return;
    if (!tree_wait(sm, &sm.pfull[i][0], j & 1, a)) return;
    fence_proxy_async_smem();
    tc_fence_after();
    if (tc_elect()) {
#pragma unroll 1
      for (int h = 0; h < 2; h++) issue_pv(t_o, t_s + 32 * h, v_s + s * kTreeOperand + h * kTreeSlab, first && h == 0);
      tc_commit(&sm.vempty[s]);
      if (flags & kTileLast) tc_commit(&sm.odone[i]);
      if ((j + 1) % kTreeBatch == 0) tc_commit(&sm.rfree[(j / kTreeBatch) & 1]);
    }
    __syncwarp();
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
__device__ __forceinline__ uint32_t tree_nodes(const TreeRec &r, int c, int k, uint64_t nodes, uint64_t &odd) {
  uint32_t own = 0, bad = 0;
  if (k >= 0) own = k < 64 ? static_cast<uint32_t>(nodes >> k) : 0u;
  else if (k > -32) own = static_cast<uint32_t>(nodes << -k);
  bad = (r.bad[0][c] | r.bad[1][c] | r.bad[2][c] | r.bad[3][c]) & own;
  if (bad) odd |= k >= 0 ? static_cast<uint64_t>(bad) << k : static_cast<uint64_t>(bad) >> -k;
  return own;
}

// 16 channels of a row, from channel c0 on: to the output, or to the CTA's part
// of a unit that several share.
template <int MT>
__device__ __forceinline__ void tree_store(const TreeArgs &a, const uint32_t (&v)[16], int c0, bool whole, size_t out_row,
                                           size_t slot, int part_row) {
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

// The values of V that are not finite, of the attended nodes `odd`, join the
// channels [c0, c1) that tree_store wrote: rare, and small rather than fast.
template <int MT>
__device__ __forceinline__ void tree_store_odd(const TreeArgs &a, uint64_t odd, int c0, int c1, int b, int hk, bool whole,
                                            size_t out_row, size_t slot, int part_row) {
  for (; odd; odd &= odd - 1) {
    const int node = __ffsll(static_cast<long long>(odd)) - 1;
    const __half *v = a.v_tree + ((static_cast<size_t>(b) * a.max_tree + node) * a.hkv + hk) * kDim;
#pragma unroll 1
    for (int c = c0; c < c1; c++) {
      if (!f16_not_finite(__half_as_ushort(v[c]))) continue;
      __half *o = a.out + out_row * kDim + c;
      float *p = a.part_o + ((slot * 32 + c / 4) * 128 * MT + part_row) * 4 + c % 4;
      if (whole) *o = __float2half_rn(__half2float(*o) + __half2float(v[c]));
      else *p += __half2float(v[c]);
    }
  }
}

// The weights of a unit: exp2(logit - m), summed, and times the V scale over the
// reference in FP16 to TMEM at `at`.
__device__ __forceinline__ void tree_weights(const uint32_t (&v)[32], float scale, float factor, float minus_m, uint32_t at,
                                             uint64_t &sum0, uint64_t &sum1) {
  const uint64_t s2 = pack2(scale, scale), f2 = pack2(factor, factor), b2 = pack2(minus_m, minus_m);
  uint32_t p[16];
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    float x, y;
    unpack2(fma2(pack2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), s2, b2), x, y);
    const uint64_t e = pack2(ex2(x), ex2(y));
    if (k & 2) sum1 = add2(sum1, e);
    else sum0 = add2(sum0, e);
    unpack2(mul2(e, f2), x, y);
    p[k >> 1] = half2_bits(x, y);
  }
  tc_st16(at, p);
}

template <int MT>
__device__ __forceinline__ void tree_softmax(const TreeArgs &a, TreeSmem<MT> &sm, uint32_t tmem, int n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stream = warp >> 2, row_in = threadIdx.x & 127;
  const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t t_o = lanes + 256 + 128 * stream;
  const int part_row = (MT == 2 ? stream * 128 : 0) + row_in;
  // the row's state in the segment
  uint64_t odd = 0;  // attended nodes whose V is not finite
  float m = -INFINITY, l = 0.f, ref = 0.f;
  float inv = 0.f, minus_m = 0.f;  // 1 / ref (0 while ref is 0), -m (0 while m is -inf)
  int ends = 0;      // segments

  for (int j = 0; j < n; j++) {
    const int buf = MT == 1 ? j & 1 : stream;
    if (!tree_wait(sm, &sm.mfull[j & (kTreeRecs - 1)], (j / kTreeRecs) & 1, a)) return;
    const TreeRec &r = sm.rec[j & (kTreeRecs - 1)];
    const uint32_t flags = r.flags, t_s = lanes + 128 * buf;
    const bool first = flags & kTileFirst;
    const int row = r.mg * 128 * MT + part_row;  // of the sequence and kv head
    const bool live = row < r.rows, warp_live = row - lane < r.rows;
    const float v_max = r.v_max;
    float ks0 = 1.f, ks1 = 1.f, vs0 = 1.f, vs1 = 1.f;  // MT 1: the scales of the stream's two units
    if (MT == 1) {
      if (flags & kTilePlain) {
        ks0 = r.k_scale[2 * stream] * a.qk_scale;
        ks1 = r.k_scale[2 * stream + 1] * a.qk_scale;
      }
      vs0 = r.v_scale[2 * stream];
      vs1 = r.v_scale[2 * stream + 1];
    }
    if (!tree_wait(sm, &sm.sfull[buf], (MT == 1 ? j >> 1 : j) & 1, a)) return;
    tc_fence_after();
    if (first) {
      m = -INFINITY;
      l = 0.f;
      odd = 0;
    }
    if (warp_live) {
      const bool tail = !(flags & kTileCold), plain = flags & kTilePlain;
      uint64_t nodes = 0;  // nodes that the row attends
      if (tail && live && r.keys > 0) {
        const int t = row_node(a, row);
        nodes = a.mask ? a.mask[static_cast<size_t>(r.b) * a.max_tree + t] : (~0ull >> (63 - t));
        if (r.keys < 64) nodes &= (1ull << r.keys) - 1;
      }
      // m and r follow the maxima when they lag too far behind; O and l follow
      // them.  Rows without a query have no say, and where m and r stay the factors
      // are exactly 1: a row's bits do not depend on its neighbours, nor on what
      // shared memory held
      auto follow = [&](float top) -> bool {
        if (__builtin_expect(__any_sync(0xffffffffu, first || (live && top > m + kLagLog2) || v_max > kLagScale * ref), 0)) {
          const float ref_new = first || v_max > kLagScale * ref ? v_max : ref;
          const float m_new = first || top > m + kLagLog2 ? fmaxf(m, top) : m;
          if (!first) {
            // (MT 2: the stream's last P V is done, as this tile's S came after it)
            if (MT == 1 && !tree_wait(sm, &sm.vempty[(j - 1) & 1], ((j - 1) >> 1) & 1, a)) return false;
            if (MT == 1) tc_fence_after();
            const float f = m == -INFINITY ? 0.f : ex2(m - m_new);
            l *= f;
            const float g = ref_new == ref ? f : f * __fdividef(ref, ref_new);  // (O is 0 while ref is)
#pragma unroll 1
            for (int c = 0; c < 8; c++) {
              uint32_t o[16];
              tc_ld16(t_o + 16 * c, o);
              tc_wait_ld(o);
#pragma unroll
              for (int k = 0; k < 16; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * g);
              tc_st16(t_o + 16 * c, o);
            }
          }
          m = m_new;
          ref = ref_new;
          inv = ref > 0.f ? __fdividef(1.f, ref) : 0.f;
          minus_m = m == -INFINITY ? 0.f : -m;
        }
        return true;
      };
      uint64_t sum0 = 0, sum1 = 0;
      constexpr int kUnits = MT == 1 ? 2 : 4;
      const int u0 = MT == 1 ? 2 * stream : 0;
      const uint32_t t_p = t_s + 32 * u0;
      if (!plain) {
        // some keys are masked (or a scale is negative): the logits, -inf where
        // masked, replace S
#pragma unroll 1
        for (int u = u0; u < u0 + kUnits; u++) {
          uint32_t v[32];
          tc_ld32(t_s + 32 * u, v);
          const float scale = r.k_scale[u] * a.qk_scale;
          uint32_t ok = r.ok[u];
          if (tail) ok |= tree_nodes(r, u, r.row0 - r.hot + 32 * u, nodes, odd);
          tc_wait_ld(v);
#pragma unroll
          for (int k = 0; k < 32; k++) v[k] = ok >> k & 1 ? __float_as_uint(__uint_as_float(v[k]) * scale) : 0xff800000u;
          tc_st32(t_s + 32 * u, v);
        }
        tc_wait_st();
      }
      auto k_scale = [&](int u) { return plain ? r.k_scale[u] * a.qk_scale : 1.f; };
      // the maximum, then the weights, by units of 32 keys; MT 1 keeps its 64 logits
      // in registers, MT 2 reads its 128 twice
      if constexpr (MT == 1) {
        uint32_t v[2][32];
        tc_ld32(t_p, v[0]);
        tc_ld32(t_p + 32, v[1]);
        tc_wait_ld(v[0]);
        tc_wait_ld(v[1]);
        if (!follow(fmaxf(max_of<32>(v[0]) * ks0, max_of<32>(v[1]) * ks1))) return;
        tree_weights(v[0], ks0, vs0 * inv, minus_m, t_p, sum0, sum1);
        tree_weights(v[1], ks1, vs1 * inv, minus_m, t_p + 16, sum0, sum1);
      } else {
        float top = -INFINITY;
#pragma unroll 1
        for (int u = 0; u < kUnits; u++) {
          uint32_t v[32];
          tc_ld32(t_s + 32 * u, v);
          tc_wait_ld(v);
          top = fmaxf(top, max_of<32>(v) * k_scale(u));
        }
        if (!follow(top)) return;
#pragma unroll 1
        for (int u = 0; u < kUnits; u++) {
          uint32_t v[32];
          tc_ld32(t_s + 32 * u, v);
          tc_wait_ld(v);
          tree_weights(v, k_scale(u), r.v_scale[u] * inv, minus_m, t_s + 16 * u, sum0, sum1);
        }
      }
      float x, y;
      unpack2(add2(sum0, sum1), x, y);
      l += x + y;
      tc_wait_st();
    }
    // what the segment's end needs of the record, which may be gone after pfull
    int b = 0, hk = 0, mg = 0, rest = 0;
    if (flags & kTileLast) {
      b = r.b;
      hk = r.hk;
      mg = r.mg;
      rest = r.rest;
    }
    tc_fence_before();
    warp_arrive(&sm.pfull[stream][MT == 1 ? buf : 0], lane);
    if (!(flags & kTileLast)) continue;

    // O of the segment's last tile
    const bool whole = (flags & kUnitStart) && (flags & kUnitEnd);
    const int t = row_node(a, row);
    const size_t out_row = (static_cast<size_t>(b) * a.max_tree + t) * a.hq + hk * a.group + row - t * a.group;
    const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (flags & kUnitStart ? 1 : 0);
    if (!tree_wait(sm, &sm.odone[stream], ends & 1, a)) return;
    tc_fence_after();
    // both streams of a row meet: stream i takes channels 64 i.. of the two
    float g = ref, gx = 0.f;  // factors of this stream's O and of the other's
    int c0 = 0, c1 = kDim;
    if constexpr (MT == 1) {
      TreeStat *st = &sm.stat[ends & 1][0][row_in];
      st[128 * stream] = TreeStat{m, l, ref, odd};
      tc_fence_before();
      warp_arrive(&sm.xfull, lane);
      if (!tree_wait(sm, &sm.xfull, ends & 1, a)) return;
      tc_fence_after();
      const TreeStat x = st[128 * (stream ^ 1)];
      const float top = fmaxf(m, x.m);
      const float f = m == top ? 1.f : ex2(m - top), fx = x.m == top ? 1.f : ex2(x.m - top);
      l = l * f + x.l * fx;
      m = top;
      odd |= x.odd;
      g *= f;
      gx = fx * x.ref;
      c0 = 64 * stream;
      c1 = c0 + 64;
    }
    const bool writer = c0 == 0;
    if (warp_live) {
      const float scale = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
      g *= scale;
      gx *= scale;
#pragma unroll 1
      for (int c = c0; c < c1; c += 16) {
        uint32_t o[16];
        tc_ld16(t_o + c, o);
        tc_wait_ld(o);
#pragma unroll
        for (int k = 0; k < 16; k++) o[k] = g != 0.f ? __float_as_uint(__uint_as_float(o[k]) * g) : 0u;
        if (MT == 1) {
          uint32_t w[16];
          tc_ld16(lanes + 256 + 128 * (stream ^ 1) + c, w);
          tc_wait_ld(w);
#pragma unroll
          for (int k = 0; k < 16; k++)
            if (gx != 0.f) o[k] = __float_as_uint(fmaf(__uint_as_float(w[k]), gx, __uint_as_float(o[k])));
        }
        if (live) tree_store<MT>(a, o, c, whole, out_row, slot, part_row);
      }
      if (live && odd) tree_store_odd<MT>(a, odd, c0, c1, b, hk, whole, out_row, slot, part_row);
    }
    // O is free (MT 1: both groups read both)
    ends++;
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sm.ofree[stream]);
      if (MT == 1) mbar_arrive(&sm.ofree[stream ^ 1]);
    }
    if (live && writer) {
      if (whole) {
        if (a.lse_out) a.lse_out[out_row] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
      } else {
        float2 *ml = reinterpret_cast<float2 *>(a.part_ml) + slot * 128 * MT;
        ml[part_row] = make_float2(m, l);
      }
    }
    // the run's last unit goes on in later CTAs: the merge finds it here
    if (row_in == 0 && (MT == 1 || stream == 0) && writer && (flags & kUnitStart) && !(flags & kUnitEnd)) {
      const long long ctas = min(static_cast<long long>(a.ctas), sm.total);
      const long long end = sm.total * (blockIdx.x + 1) / ctas + rest;  // of the unit, in the list
      a.shared_units[blockIdx.x] = make_int4(b, hk, mg, static_cast<int>((end * ctas - 1) / sm.total - blockIdx.x));
    }
  }
}

template <int MT, bool kF16>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const __grid_constant__ TreeArgs a) {
  using Shape = TreeShape<MT>;
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t base = smem_addr(raw);
  if (base & 1023) {  // (the operands' swizzle is one of addresses)
    set_status(a.status, HYB_STATUS_TIMEOUT);
    return;
  }
  const uint32_t q_s = base, k_s = q_s + Shape::kQBytes, v_s = k_s + kTreeStages * kTreeOperand, c_s = base + Shape::kTiles;
  TreeSmem<MT> &sm = *reinterpret_cast<TreeSmem<MT> *>(raw + Shape::kTiles + TreeSmem<MT>::kPieces * kPiece);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge waits for this grid's end
  constexpr int kMmaWarp = kTreeSoft + kTreeProd, kScoutWarp = kMmaWarp + kTreeMma;

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
    a.shared_units[blockIdx.x] = make_int4(0, 0, 0, 0);
    sm.abort = 0;
    for (int i = 0; i < 2; i++) {
      mbar_init(&sm.kfull[i], kTreeProd / 2);
      mbar_init(&sm.vfull[i], kTreeProd / 2);
      mbar_init(&sm.kempty[i], MT);
      mbar_init(&sm.vempty[i], MT);
      mbar_init(&sm.rfull[i], 1);
      mbar_init(&sm.rfree[i], kTreeMma + TreeSmem<MT>::kPieces);
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.pfull[i][0], 4);
      mbar_init(&sm.pfull[i][1], 4);
      mbar_init(&sm.odone[i], 1);
      mbar_init(&sm.ofree[i], MT == 1 ? 8 : 4);
      mbar_init(&sm.drain[i], 1);
    }
    for (int i = 0; i < kTreeRecs; i++) mbar_init(&sm.mfull[i], kTreeProd / 2);
    for (int i = 0; i < 2; i++) {
      mbar_init(&sm.qfull[i], 32);
      mbar_init(&sm.qempty[i], MT);
    }
    for (int i = 0; i < TreeSmem<MT>::kPieces; i++) {
      mbar_init(&sm.cfull[i], 1);
      mbar_init(&sm.cempty[i], kF16 ? kTreeProd : kTreeProd / 2);
    }
    mbar_init(&sm.xfull, 8);
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTreeSoftRegs));
    tree_softmax<MT>(a, sm, tmem, n_tiles);
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTreeProdRegs));
    const int kv = (warp - kTreeSoft) / (kTreeProd / 2);
    tree_produce<MT, kF16>(a, sm, kv ? v_s : k_s, c_s, kv, n_tiles);
  } else if (warp < kScoutWarp) {
    const int i = warp - kMmaWarp;
    if constexpr (MT == 2) tree_mma2(a, sm, q_s, k_s, v_s, tmem, n_tiles, i);
    else if (i == 0) tree_mma_qk(a, sm, q_s, k_s, tmem, n_tiles);
    else tree_mma_pv(a, sm, v_s, tmem, n_tiles);
    __syncwarp();
    // no MMA is in flight when TMEM is given back
    if (tc_elect()) tc_commit(&sm.drain[i]);
    __syncwarp();
    if (!mbar_wait_bounded(&sm.drain[i], 0, kDefaultWaitCycles)) sm.abort = 1;
    __syncwarp();
  } else if (warp > kScoutWarp) {
    if (lane < TreeSmem<MT>::kPieces) tree_copy<MT, kF16>(a, sm, c_s, n_tiles, lane);
    __syncwarp();
  } else {
    tree_scout<MT, kF16>(a, sm, q_s, n_tiles);
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tc_dealloc(tmem, 512);
  if (tid == 0 && sm.abort) set_status(a.status, HYB_STATUS_TIMEOUT);
}

// ---- the merge of units that several CTAs share ----
// CTA = (the CTA with a shared unit's first tile, 32 rows): thread = row (lane)
// and 16 channels (warp); parts in the order of the tiles.
template <int MT>
__global__ void __launch_bounds__(256) tree_combine_kernel(const __grid_constant__ TreeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = blockIdx.x;
  const int4 unit = a.shared_units[c0];  // sequence, kv head, row group, tiles of the unit in later CTAs
  if (unit.w <= 0) return;
  const int b = unit.x, hk = unit.y, mg = unit.z;
  const int G = a.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nt = a.n_tree ? a.n_tree[b] : a.max_tree;
  const int r = 32 * blockIdx.y + lane, row = mg * 128 * MT + r;
  if (row >= nt * G) return;
  const int t = row / G;
  const size_t out_row = (static_cast<size_t>(b) * a.max_tree + t) * a.hq + hk * G + row - t * G;
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
  const float4 *po = reinterpret_cast<const float4 *>(a.part_o);
  // the later CTAs' parts: all but the last hold nothing else
  float top = ml[(2 * static_cast<size_t>(c0) + 1) * 128 * MT + r].x;
  const int c1 = c0 + unit.w;
  for (int i = c0 + 1; i <= c1; i++) top = fmaxf(top, ml[2 * static_cast<size_t>(i) * 128 * MT + r].x);
  float sum = 0.f;
  float4 o[4];
#pragma unroll
  for (int k = 0; k < 4; k++) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = c0; i <= c1; i++) {
    const size_t slot = 2 * static_cast<size_t>(i) + (i == c0);
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
    h[2 * k] = half2_bits(o[k].x * inv, o[k].y * inv);
    h[2 * k + 1] = half2_bits(o[k].z * inv, o[k].w * inv);
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
    // the softmax warps' registers come from the producers', of what the launch
    // really has
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, tree_kernel<MT, kF16>);
    if (e != cudaSuccess) return e;
    if (2 * at.numRegs < kTreeSoftRegs + kTreeProdRegs) return cudaErrorInvalidKernelImage;
    if (dev < 31) configured_dev_mask |= 1 << dev;
  }
  tree_kernel<MT, kF16><<<a.ctas, kTreeThreads, Shape::kBytes, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int G = a.group;
  const int rows = a.max_tree * G < 128 * MT ? a.max_tree * G : 128 * MT;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas, (rows + 31) / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_combine_kernel<MT>, a);
}

cudaError_t launch_tree_attn(const TreeArgs &a, cudaStream_t stream) {
  const bool two = tree_m_tiles(a.max_tree, a.group) == 2;
  if (a.quant_bits == 0) return two ? launch_tree<2, true>(a, stream) : launch_tree<1, true>(a, stream);
  return two ? launch_tree<2, false>(a, stream) : launch_tree<1, false>(a, stream);
}

}  // namespace hyb
