// Attention of a tree of T drafted tokens per sequence over the committed cache
// and the drafted tokens themselves (verification of a speculative step).
//
// Draft t of sequence b sits at position n_b + depth_t, n_b = lens[b] committed
// tokens before it.  It attends
//   - committed keys: all of them; with a window W those at positions >
//     n_b + depth_t - W; with a selection those whose bit is set;
//   - drafted keys j with bit j of its tree row set (and, with a window,
//     depth_j > depth_t - W),
// and o = sum_j softmax_j(scale * q.k_j) v_j over them (0 when there are none).
// The committed rows lie by position, or in a ring: position p in row p mod N.
//
// Bound: HBM (each committed row once per KV head) up to about 128 query rows
// per KV head (G heads x T drafts), the tensor cores above.
//
// Design (B200, tcgen05).  The query rows of a KV head go on the N side of both
// products and the KEYS (then the head dims) on the M side, so that a tile
// always fills the tensor core's 128 lanes however few drafts there are:
//   S^T = K Q^T      [128 keys x NR rows], A = K tile, B = Q, both K-major
//   O^T += V^T P^T   [128 dims x NR rows], A = V tile, B = P, both MN-major
// With the rows on M, 64 rows would waste half of every instruction.
// P and its rounding error go into one product as 128 columns (hi | lo).
//   softmax  a thread holds one key and 32 query rows.  Exponentials are taken
//            against a reference per row that is not the running maximum: the
//            logit of the first tile's first key, attended or not, raised every
//            8 tiles where a sum has grown past 2^40.  fp32 and bf16 share their
//            exponent range, so any reference within 2^60 above and 2^80 below
//            the row's maximum gives the same precision, and a tile needs no
//            reduction over keys and no exchange between warps.  A row outside
//            that range shows in its sum and goes the scalar way below.
//   O        is summed in TMEM over an epoch of 8 tiles (the tensor core
//            truncates, so a long sum would drift), then added to a second TMEM
//            tile by fp32 adds, and rescaled where references were raised.
//   streams  two groups of 8 softmax warps, each with its own S, P, O and
//            references for 64 rows, so that one exponentiates while the other
//            waits, loads or stores.  Up to 64 rows the streams take every other
//            tile of the same rows and their sums meet at the end; above, each
//            takes 64 of a CTA's 128 rows of every tile.
// Warps: 2 x 8 softmax, 4 loaders, 1 MMA issuer.  Interior tiles come by TMA
// (128-byte swizzle), tiles with rows to leave out (past the end, a ring's seam,
// drafts, selected keys) by 16-byte cp.async into the same layout, with zeros in
// the rows that hold no token.
//
// Work: the tiles of all (sequence, KV head) groups form one line, cut into
// equal ranges, one CTA each; a CTA's range may begin or end inside a group, and
// such pieces are joined by a second kernel (one warp or more per query row).
//
// With a selection a CTA reads the mask words of its rows, 512 keys at a time,
// queues the keys that any row selected (a ballot per key transposes the bits:
// the queue holds a key's row bits), and gathers only those, 128 to a tile.
//
// A row whose result is not finite, or whose sum has left its range, is computed
// again by a scalar pass over the keys it attends (0 * inf in a product with
// P = 0 must not reach it).
#include <math.h>

#include "launch.h"
#include "tc05.cuh"

namespace rtp {

namespace {

constexpr int kTrKeys = 128;                 // keys per tile
constexpr int kTrStages = 2;                 // K/V ring
constexpr int kTrHalf = kTrKeys * 128;       // 128 rows x 64 bf16, 128-byte swizzle
constexpr int kTrTile = 2 * kTrHalf;         // one K or V tile: 32 KB
constexpr int kTrLoadWarps = 4;
constexpr int kTrEpoch = 8;                  // tiles summed in TMEM before an fp32 add
constexpr float kTrHigh = 1.0995116e12f;     // 2^40: a sum above it raises the row's reference
constexpr float kTrLow = 8.6736174e-19f;     // 2^-60: a sum below it has lost the row's largest terms
constexpr float kTrTop = 1.2676506e30f;      // 2^100: a sum above it is past what a factor can scale down
constexpr float kTrNone = -3.0e38f;          // log2 of an empty sum
constexpr int kTrRound = 512;                // keys whose selection bits are read at a time
constexpr int kTrQueue = 640;                // 128 left over + one round
constexpr int kTrSms = 148;
constexpr int kTrStream = 64;                // query rows of a stream
constexpr int kTrSoft = 256;                 // threads of a stream
constexpr int kTrLoad = kTrLoadWarps * 32;
constexpr int kTrThreads = 2 * kTrSoft + kTrLoad + 128;  // (whole warpgroups; one warp issues the MMAs)
constexpr int kTrRing = 8;                   // tiles (and segments) described ahead
// registers per thread of each role; the launch's threads x registers hold them all
constexpr int kTrLaunchRegs = 80, kTrSoftRegs = 96, kTrLoadRegs = 56, kTrMmaRegs = 40;
static_assert(2 * kTrSoft * kTrSoftRegs + kTrLoad * kTrLoadRegs + 128 * kTrMmaRegs <= kTrThreads * kTrLaunchRegs,
              "register split");
constexpr int kBarLoad = 1;                  // named barrier
// TMEM columns of a stream: S, the epoch's O (hi | lo), the total O
constexpr uint32_t kTmemStream = 256, kTmemOe = 64, kTmemOt = 192, kTmemCols = 512;

// What the softmax needs to know of a segment (a CTA's share of a group's tiles).
struct TrSegInfo {
  int b, kvh, n, lo, draft_tiles, max_depth;
  int slot;   // where its partial result goes, or -1: the whole group
  int pad;
};

// NR query rows per CTA: 64 (the streams take tiles in turn) or 128 (64 rows each).
template <int NR>
struct TrSmem {
  static constexpr int kQueue = NR == 64 ? kTrQueue : 1, kMasks = NR == 64 ? 4 : 1;
  alignas(1024) uint8_t q[NR * 256];
  alignas(1024) uint8_t k[kTrStages][kTrTile];
  alignas(1024) uint8_t v[kTrStages][kTrTile];
  alignas(1024) uint8_t p[2][2][kTrKeys * kTrStream * 2];  // [stream][hi, lo]
  int row_at[NR];                        // each row's draft times 8 plus its head in the group
  alignas(16) float nref[2][kTrStream];  // minus the reference of each row (log2 units)
  alignas(16) float alpha[2][kTrStream];  // 2^(old - new reference) of the last raise; at a segment's end their scales or 1 / sum
  float sum[NR == 64 ? 2 : 1][NR == 64 ? kTrStream : 1];
  float wt[NR == 64 ? 2 : 1][2][NR == 64 ? kTrStream : 1];  // [stream writing][stream summed]: factors of its O
  uint32_t colmax[2][kTrStream];         // the largest sum of a row in any thread (float bits)
  uint64_t k_full[kTrStages], k_empty[kTrStages], v_full[kTrStages], v_empty[kTrStages];
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2], o_free[2], sum_full[2], sum_free[2], sync[2];
  uint64_t q_full, q_free, fin;
  int2 meta[kTrRing];            // per tile: its number in the group; 4 * segment + 2 * (CTA's last) + (segment's last)
  int4 cur[2];                   // each stream's scores: tile (-1: no more), and its meta
  int new_epoch[2];
  int raise[2][2];               // some sum has grown too large (alternating epochs)
  uint32_t seen[2][2];           // rows that attend a key of the segment
  int state[2];                  // at a segment's end: 1 the stream has an O, 2 and a total
  uint32_t tmem_base;
  int start_b;
  int start_base;
  int total, per;                // tiles of the whole line, and of a range
  int cnt[2][kTrLoadWarps];
  TrSegInfo seg[kTrRing];
  int qkey[kQueue];              // selected keys waiting for a tile (ring)
  uint2 qbits[kQueue];           // and which rows selected them
  uint32_t kmask[kMasks][2][NR == 64 ? kTrKeys : 1];  // row bits of a tile's keys
};

// ---- small helpers --------------------------------------------------------------
RTP_DEVICE void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
RTP_DEVICE void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
RTP_DEVICE void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }
RTP_DEVICE void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

template <int N>
RTP_DEVICE void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
RTP_DEVICE void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }

// mbar_wait, kept small: the code of a CTA has to stay in the instruction cache, and most of it runs once or twice.
RTP_DEVICE bool wait_bar(uint64_t* bar, uint32_t parity, bool& alive, const TreeAttnArgs& A) {
  if (!alive) return false;
  if (mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (!mbar_try(bar, parity))
    if (clock64() - t0 > A.budget) {
      atomicExch(A.err, kDevErrTimeout);
      alive = false;
      break;
    }
  return alive;
}

RTP_DEVICE void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// Barrier of n threads that also ORs a predicate.
RTP_DEVICE bool bar_or(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// Pairs of floats in one 64-bit word, and packed arithmetic on them.
RTP_DEVICE uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
RTP_DEVICE void unpack2(uint64_t x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(x)); }
RTP_DEVICE uint64_t add2u(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
RTP_DEVICE uint64_t sub2u(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// (a * s + c.lo, b * s + c.hi), c a pair of floats in one 64-bit word.
RTP_DEVICE void fma2c(uint32_t a, uint32_t b, uint64_t s, uint64_t c, float& ra, float& rb) {
  uint64_t x, r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(x) : "r"(a), "r"(b));
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(x), "l"(s), "l"(c));
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(ra), "=f"(rb) : "l"(r));
}

// Column c of every lane reduced over the 32 lanes, left in lane c (31 shuffles).
template <int O, typename F>
RTP_DEVICE float reduce_columns(float (&x)[2 * O], int lane, F op) {
  const bool up = lane & O;
  float y[O];
#pragma unroll
  for (int i = 0; i < O; ++i) {
    const float keep = up ? x[i + O] : x[i], send = up ? x[i] : x[i + O];
    y[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, O));
  }
  if constexpr (O == 1)
    return y[0];
  else
    return reduce_columns<O / 2>(y, lane, op);
}

// Bit c of lane k becomes bit k of lane c.
RTP_DEVICE uint32_t transpose32(uint32_t x, int lane) {
  uint32_t m = 0x0000ffffu;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
    x = lane & j ? (x & ~m) | ((y >> j) & m) : (x & m) | ((y & m) << j);
    m ^= m << (j >> 1);
  }
  return x;
}

// Waits for the loads that fill these registers (naming them keeps their uses behind it).
RTP_DEVICE void tmem_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
RTP_DEVICE void tmem_wait(float (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]));
}

// 32 lanes x 8 consecutive columns.
RTP_DEVICE void tmem_ld8(uint32_t taddr, float (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "r"(taddr));
}

// ---- what a sequence's rows attend -------------------------------------------------
// Committed tokens of sequence b.
RTP_DEVICE int committed(const TreeAttnArgs& A, int b) {
  const int n = A.lens ? max(A.lens[b], 0) : A.N;
  return A.ring ? n : min(n, A.N);
}

RTP_DEVICE int row_of(const TreeAttnArgs& A, uint32_t p) { return A.ring ? (int)(p % (uint32_t)A.N) : (int)p; }

// Tokens between a draft and the oldest committed key it attends, less the draft's own depth (W > 0).
RTP_DEVICE int draft_depth(const TreeAttnArgs& A, int b, int t) {
  return A.W > 0 ? max(__ldg(A.depth + (int64_t)b * A.T + t), 0) : 0;
}
RTP_DEVICE int oldest_age(const TreeAttnArgs& A, int depth) { return A.W - 2 - depth; }

RTP_DEVICE bool tree_bit(const TreeAttnArgs& A, int b, int t, int j) {
  return (__ldg(A.tree + ((int64_t)b * A.T + t) * A.tree_words + (j >> 5)) >> (j & 31)) & 1u;
}

// Tiles of one KV head of a sequence: its drafts first, then the committed keys from position lo on (with a
// selection: rounds of kTrRound keys, aligned).
struct TrSpan {
  int n, lo, draft_tiles, tiles;
};
template <bool SEL>
RTP_DEVICE TrSpan span_of(const TreeAttnArgs& A, int b) {
  constexpr uint32_t kStep = SEL ? kTrRound : kTrKeys;
  TrSpan s;
  s.n = committed(A, b);
  s.lo = A.W > 0 ? max(0, s.n - (A.W - 1)) : 0;
  if (SEL) s.lo = s.lo / kTrRound * kTrRound;
  s.draft_tiles = (A.T + kTrKeys - 1) / kTrKeys;
  s.tiles = s.draft_tiles + (int)(((uint32_t)(s.n - s.lo) + kStep - 1) / kStep);
  return s;
}

// One segment: the tiles [u0, u1) of a group (b, kvh) that a CTA works on.
struct TrSeg {
  int b, kvh;
  TrSpan span;
  int u0, u1;
  int base;  // the line's tile number of the group's tile 0
};

// Walks the segments of the range [lo, hi) of the line of tiles.
template <bool SEL>
struct TrWalk {
  int pos, hi, base_b;
  TrSeg s;
  RTP_DEVICE void start(const TreeAttnArgs& A, int lo, int end, int b, int base) {
    pos = lo;
    hi = end;
    base_b = base;
    s.b = b;
    s.span = span_of<SEL>(A, b);
    s.kvh = (lo - base) / s.span.tiles;
    fill();
  }
  RTP_DEVICE void fill() {
    s.base = base_b + s.kvh * s.span.tiles;
    s.u0 = pos - s.base;
    s.u1 = min(s.span.tiles, hi - s.base);
  }
  RTP_DEVICE bool next(const TreeAttnArgs& A) {
    pos = s.base + s.u1;
    if (pos >= hi) return false;
    if (++s.kvh == A.Hk) {
      base_b += A.Hk * s.span.tiles;
      s.kvh = 0;
      s.span = span_of<SEL>(A, ++s.b);
    }
    fill();
    return true;
  }
};

// ---- the scalar pass ------------------------------------------------------------------
// One warp computes one row from the definition.
__device__ __noinline__ void scalar_row(const TreeAttnArgs& A, int b, int h, int t, float4& out) {
  const int lane = threadIdx.x & 31, kvh = h / A.G;
  auto row = [&](const View4& x, int head, int64_t r) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(x.data) + b * x.sb +
                                                         head * x.sh + r * x.sn + 4 * lane));
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  };
  const float4 q = row(A.q, h, t);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto take = [&](const float4 k, const float4 v) {
    const float s = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w) * A.scale_log2;
    const float mn = fmaxf(m, s);
    const float al = mn == -INFINITY ? 1.f : ex2a(m - mn), p = mn == -INFINITY ? 0.f : ex2a(s - mn);
    m = mn;
    l = l * al + p;
    o = make_float4(o.x * al + p * v.x, o.y * al + p * v.y, o.z * al + p * v.z, o.w * al + p * v.w);
  };
  const int n = committed(A, b), depth = draft_depth(A, b, t);
  const int lo = A.W > 0 ? max(0, n - 1 - oldest_age(A, depth)) : 0;  // (past n when the window holds none)
  const uint32_t* sel = A.sel ? A.sel + ((int64_t)(b * A.Hq + h) * A.T + t) * A.sel_words : nullptr;
  if (A.W <= 0 || oldest_age(A, depth) >= 0)
#pragma unroll 1
    for (int p = lo; p < n; ++p) {
      if (sel && !((__ldg(sel + (p >> 5)) >> (p & 31)) & 1u)) continue;
      const int r = row_of(A, (uint32_t)p);
      take(row(A.k, kvh, r), row(A.v, kvh, r));
    }
#pragma unroll 1
  for (int j = 0; j < A.T; ++j) {
    if (!tree_bit(A, b, t, j)) continue;
    if (A.W > 0 && draft_depth(A, b, j) <= depth - A.W) continue;
    take(row(A.kn, kvh, j), row(A.vn, kvh, j));
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;  // (a NaN stays one)
  out = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

RTP_DEVICE void store4(const TreeAttnArgs& A, int64_t off, const float4& y) {
  if (A.o_bf16)
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(A.o.data) + off) =
        make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(A.o.data) + off) = y;
}

RTP_DEVICE bool finite4(const float4& y) {
  return isfinite(y.x) && isfinite(y.y) && isfinite(y.z) && isfinite(y.w);
}

// ---- layout of the workspace -------------------------------------------------------------
struct TrLayout {
  int nr, rbs, ranges;  // rows per CTA, row blocks per KV head, ranges of the line of tiles
  size_t table, o, ml;  // byte sizes
  size_t bytes() const { return table + o + ml; }
};

TrLayout tree_layout(int64_t B, int64_t Hq, int64_t T, int64_t Hk, bool sel) {
  TrLayout L;
  const int64_t rows = Hq / Hk * T;
  // (a selection's queue and masks take the shared memory of the larger form)
  L.nr = sel || rows <= 64 ? 64 : 128;
  L.rbs = (int)((rows + L.nr - 1) / L.nr);
  L.ranges = L.rbs >= kTrSms ? 1 : kTrSms / L.rbs;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  L.table = up((size_t)(B * Hk) * sizeof(int2));
  const size_t slots = (size_t)L.rbs * L.ranges * 2 * L.nr;
  L.o = up(slots * kHeadDim * sizeof(float));
  L.ml = up(slots * sizeof(float2));
  return L;
}

// What the kernels know of it.  A piece of a group lies in slot 2 range + (1 if it begins the group).
struct TrParts {
  int2* table;  // [B * Hk] first range and number of pieces
  float* o;     // [row block][2 * ranges][nr][128]
  float2* ml;   // [row block][2 * ranges][nr] m and l, the sum of 2^logit being 2^m l; o is normalised
  int nr, rbs, ranges;
};

struct TrMaps {
  CUtensorMap k, v;
};

// ---- the kernel --------------------------------------------------------------------------
template <int NR, bool SEL>
__global__ void __launch_bounds__(kTrThreads, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ TreeAttnArgs A, const __grid_constant__ TrParts W, int use_tma) {
  using Smem = TrSmem<NR>;
  constexpr bool kSplitRows = NR == 128;  // the streams share tiles (64 rows each), else they take tiles in turn
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(smem_raw);
  if (smem_addr(smem_raw) % 1024u) {  // (the swizzle and the descriptors rest on the alignment declared above)
    if (threadIdx.x == 0) atomicExch(A.err, kDevErrTimeout);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rb = blockIdx.x % W.rbs, range = blockIdx.x / W.rbs;
  const int rows = A.G * A.T, row0 = rb * NR, nrows = min(NR, rows - row0);

  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], 1);
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.v_full[i], 1);
      mbar_init(&S.v_empty[i], 1);
      mbar_init(&S.s_full[i], 2);  // the products' commit, and the issuer (for S.cur)
      mbar_init(&S.s_free[i], 8);
      mbar_init(&S.p_full[i], 8);
      mbar_init(&S.p_free[i], 1);
      mbar_init(&S.o_free[i], 8);
      mbar_init(&S.sum_full[i], 8);
      mbar_init(&S.sum_free[i], 8);
      mbar_init(&S.sync[i], 8);
      S.raise[i][0] = S.raise[i][1] = 0;
      S.seen[i][0] = S.seen[i][1] = 0u;
    }
    mbar_init(&S.q_full, 1);
    mbar_init(&S.q_free, 1);
    mbar_init(&S.fin, 1);
    mbar_fence_init();
  }
  if (tid < 2 * kTrStream) S.colmax[0][tid] = 0u;
  if (tid < NR) {
    const int r = min(row0 + tid, rows - 1), g = r / A.T;
    S.row_at[tid] = (r - g * A.T) * 8 + g;
  }
  if (use_tma && tid == kTrThreads - 1) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (warp == 0) tmem_alloc(&S.tmem_base, kTmemCols);
  // rows past the last one never get a P: zeros
  if (nrows < NR) {
    uint4* p = reinterpret_cast<uint4*>(&S.p[0][0][0]);
#pragma unroll 1
    for (int i = tid; i < (int)(sizeof(S.p) / 16); i += kTrThreads) p[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_async();
  }
  pdl_wait();
  pdl_release();

  // ---- this CTA's range of the line of tiles ----
  if (warp == 0) {
    int sum = 0;
    const int first = lane < A.B ? span_of<SEL>(A, lane).tiles : 0;
#pragma unroll 1
    for (int b = lane; b < A.B; b += 32) sum += b == lane ? first : span_of<SEL>(A, b).tiles;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int total = sum * A.Hk, per = (total + W.ranges - 1) / W.ranges, lo = range * per;
    if (lane == 0) {
      S.total = total;
      S.per = per;
    }
    int base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < A.B && lo < total; b0 += 32) {
      const int b = b0 + lane;
      const int mine = (b0 == 0 ? first : b < A.B ? span_of<SEL>(A, b).tiles : 0) * A.Hk;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, base + incl > lo);
      if (past) {
        if (lane == __ffs(past) - 1) {
          S.start_b = b;
          S.start_base = base + incl - mine;
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  const int per = S.per, lo = range * per, hi = min(lo + per, S.total);
  const bool work = lo < hi;

  bool alive = true;

  if (warp >= 2 * kTrSoft / 32 && warp < 2 * kTrSoft / 32 + kTrLoadWarps) {
    // ---------------- loaders ----------------
    regs_dec<kTrLoadRegs>();
    const int lt = tid - 2 * kTrSoft, lw = lt >> 5;
    const int chunk = lt & 15, r_first = lt >> 4;  // this thread's 16-byte column; rows r_first + 8 i
    // (8 rows on, the swizzle is the same)
    const uint32_t slot0 = (uint32_t)r_first * 128u + (uint32_t)(((chunk & 7) ^ r_first) << 4);
    const uint32_t slot_kv = slot0 + (uint32_t)(chunk >> 3) * (uint32_t)kTrHalf;
    uint32_t it = 0, k_loads = 0;  // tiles so far; tiles whose K has been sent for
    int segs = 0;
    bool q_due = false;
    // Waits for a free K or V stage; false (for all loaders alike) once any wait gave up.
    auto stage_free = [&](uint64_t* empty) {
      const bool ok = wait_bar(&empty[it & 1], ((it >> 1) & 1u) ^ 1u, alive, A);
      return !bar_or(kBarLoad, kTrLoad, !ok);
    };
    // 128 rows of K or V by cp.async: row_at(r, ok) gives the row of tile row r.
    auto copy_rows = [&](const View4& x, uint8_t* tile, const TrSeg& s, auto&& row_at) {
      const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(x.data) + s.b * x.sb + s.kvh * x.sh + chunk * 8;
      const uint32_t dst = smem_addr(tile) + slot_kv;
#pragma unroll 2
      for (int i = 0; i < 16; ++i) {
        bool ok;
        const int row = row_at(r_first + 8 * i, ok);
        cp16(dst + 1024u * i, ok ? (const void*)(base + row * x.sn) : A.q.data, ok);
      }
      cp_commit();
    };
    auto landed = [&](uint64_t* full) {  // (after a cp_wait) every loader's copies are there
      fence_async();
      named_sync(kBarLoad, kTrLoad);
      if (lt == 0) {
        if (q_due) mbar_arrive(&S.q_full);
        if (full) mbar_arrive(full);
      }
      q_due = false;
    };
    auto gather = [&](const View4& xk, const View4& xv, const TrSeg& s, int u, int flags, auto&& row_at) -> bool {
      const int st = it & 1;
      bool k_there = false;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        // K is handed on before a wait for V's stage, else with V on its way
        if (i == 1 && bar_or(kBarLoad, kTrLoad, !mbar_try(&S.v_empty[st], ((it >> 1) & 1u) ^ 1u))) {
          cp_wait<0>();
          landed(&S.k_full[st]);
          k_there = true;
        }
        if (!stage_free(i ? S.v_empty : S.k_empty)) return false;
        if (i == 0 && lt == 0) S.meta[it % kTrRing] = make_int2(u, flags);
        copy_rows(i ? xv : xk, i ? S.v[st] : S.k[st], s, row_at);
      }
      if (!k_there) {
        cp_wait<1>();
        landed(&S.k_full[st]);
      }
      cp_wait<0>();
      landed(&S.v_full[st]);
      k_loads = ++it;
      return true;
    };
    TrWalk<SEL> walk;
    bool more = work, ok = true;
    if (more) walk.start(A, lo, hi, S.start_b, S.start_base);
#pragma unroll 1
    while (more && ok) {
      const TrSeg s = walk.s;
      const int seg_flags = 4 * segs, last_flags = seg_flags + (s.base + s.u1 < hi ? 1 : 3);
      // ---- the query rows (the previous segment's products are done with the buffer) ----
      {
        const bool free = segs == 0 || wait_bar(&S.q_free, (segs - 1) & 1u, alive, A);
        if (bar_or(kBarLoad, kTrLoad, !free)) break;
        const __nv_bfloat16* qb =
            static_cast<const __nv_bfloat16*>(A.q.data) + s.b * A.q.sb + (int64_t)s.kvh * A.G * A.q.sh + chunk * 8;
#pragma unroll 4
        for (int i = 0; i < NR / 8; ++i) {
          const int r = r_first + 8 * i, at = S.row_at[r];
          cp16(smem_addr(S.q) + (uint32_t)(chunk >> 3) * (NR * 128u) + slot0 + 1024u * i,
               qb + (at & 7) * A.q.sh + (at >> 3) * A.q.sn, r < nrows);
        }
        cp_commit();
        q_due = true;
      }
      {
        TrSegInfo info;
        info.b = s.b;
        info.kvh = s.kvh;
        info.n = s.span.n;
        info.lo = s.span.lo;
        info.draft_tiles = s.span.draft_tiles;
        info.max_depth = 0;
        if (A.W > 0) {
#pragma unroll 1
          for (int t = lane; t < A.T; t += 32) info.max_depth = max(info.max_depth, draft_depth(A, s.b, t));
          info.max_depth = __reduce_max_sync(0xffffffffu, info.max_depth);
        }
        const bool whole = s.u0 == 0 && s.u1 == s.span.tiles;
        info.slot = whole ? -1 : rb * 2 * W.ranges + 2 * range + (s.u0 == 0 ? 1 : 0);
        info.pad = 0;
        if (lt == 0) {
          S.seg[segs % kTrRing] = info;
          if (s.u0 == 0 && rb == 0)
            W.table[s.b * A.Hk + s.kvh] = make_int2(range, (s.base + s.span.tiles - 1) / per - range + 1);
        }
        ++segs;
      }
      const int drafts_end = min(s.u1, s.span.draft_tiles);
      more = walk.next(A);
      for (int u = s.u0; u < drafts_end && ok; ++u)
        ok = gather(A.kn, A.vn, s, u, u + 1 == s.u1 ? last_flags : seg_flags, [&](int r, bool& live) {
          const int j = u * kTrKeys + r;
          live = j < A.T;
          return live ? j : 0;
        });
      if (!ok || s.u1 <= s.span.draft_tiles) continue;
      if constexpr (!SEL) {
        auto by_tma = [&](int u, uint32_t& p0, int& left, int& first) {  // a whole tile of neighbouring rows
          p0 = (uint32_t)s.span.lo + (uint32_t)(u - s.span.draft_tiles) * kTrKeys;
          left = s.span.n - (int)p0;  // committed rows from here on
          first = row_of(A, p0);
          return use_tma && left >= kTrKeys && A.N - first >= kTrKeys;
        };
        auto load = [&](const CUtensorMap* map, uint8_t* tile, uint64_t* full, int first) {
          mbar_expect_tx(full, kTrTile);
          tma_load_4d(tile, map, full, 0, first, s.kvh, s.b);
          tma_load_4d(tile + kTrHalf, map, full, 64, first, s.kvh, s.b);
        };
        bool ahead = false;  // this tile's K is already on its way
#pragma unroll 1
        for (int u = max(s.u0, s.span.draft_tiles); u < s.u1 && ok; ++u) {
          uint32_t p0;
          int left, first;
          const int st = it & 1;
          if (by_tma(u, p0, left, first)) {
            // the next tile's K before this one's V: scores are computed ahead of the products with V
#pragma unroll 1
            for (int i = ahead ? 1 : 0; i < 2 && ok; ++i) {
              uint32_t q0;
              int rest, at;
              if (u + i == s.u1 || !by_tma(u + i, q0, rest, at)) {
                ahead = false;
                break;
              }
              it += i;
              ok = stage_free(S.k_empty);
              it -= i;
              if (lt == 0 && ok) {
                S.meta[(it + i) % kTrRing] = make_int2(u + i, u + i + 1 == s.u1 ? last_flags : seg_flags);
                load(&kmap, S.k[st ^ i], &S.k_full[st ^ i], at);
                k_loads = it + i + 1;
              }
              ahead = i;
              if (q_due) {
                cp_wait<0>();
                landed(nullptr);
              }
            }
            if (!ok || !(ok = stage_free(S.v_empty))) break;
            if (lt == 0) load(&vmap, S.v[st], &S.v_full[st], first);
            ++it;
          } else {
            ok = gather(A.k, A.v, s, u, u + 1 == s.u1 ? last_flags : seg_flags, [&](int r, bool& live) {
              live = r < left;
              return live ? row_of(A, p0 + (uint32_t)r) : 0;
            });
          }
        }
      } else {
        const int rounds = s.span.tiles - s.span.draft_tiles;
        int head = 0, count = 0, turn = 0;
        auto wrap = [](int i) { return i >= kTrQueue ? i - kTrQueue : i; };
        // this lane's rows: their mask rows, and the first key position their window admits
        const uint32_t* words[2];
        int from[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = lane + 32 * i;
          words[i] = nullptr;
          from[i] = 0;
          if (r < nrows) {
            words[i] = A.sel + ((int64_t)(s.b * A.Hq + s.kvh * A.G) * A.T + row0 + r) * A.sel_words;
            if (A.W > 0) {
              const int age = oldest_age(A, draft_depth(A, s.b, (row0 + r) % A.T));
              from[i] = age < 0 ? s.span.n : s.span.n - 1 - age;
            }
          }
        }
        // a round's mask words, on their way while the round before is worked on; neighbouring ranges take rounds
        // from all over the context (a prime larger than their number), since selected keys come in clusters
        uint32_t ahead[2][4];
        int next_key = 0;
        auto fetch = [&](int u) {
          const int i0 = u - s.span.draft_tiles;
          const int round = (int)((uint64_t)i0 * 2654435761ull % (uint64_t)rounds);
          next_key = s.span.lo + round * kTrRound + lw * 128;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int wb = next_key + 32 * w, rem = s.span.n - wb;
#pragma unroll
            for (int i = 0; i < 2; ++i) ahead[i][w] = words[i] && rem > 0 ? __ldg(words[i] + (wb >> 5)) : 0u;
          }
        };
        fetch(max(s.u0, s.span.draft_tiles));
        auto emit = [&](int take, int flags) {
          // one key per loader thread: its row bits for the softmax
          uint2 bits = make_uint2(0u, 0u);
          if (lt < take) bits = S.qbits[wrap(head + lt)];
          S.kmask[it & 3][0][lt] = bits.x;
          S.kmask[it & 3][1][lt] = bits.y;
          const int at = head;
          ok = gather(A.k, A.v, s, s.span.draft_tiles, flags, [&](int r, bool& live) {
            live = r < take;
            return live ? S.qkey[wrap(at + r)] : 0;
          });
          head = wrap(head + take);
          count -= take;
        };
        for (int u = max(s.u0, s.span.draft_tiles); u < s.u1 && ok; ++u) {
          uint32_t x[2][4], uni[4];
          const int key0 = next_key;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            x[0][w] = ahead[0][w];
            x[1][w] = ahead[1][w];
          }
          if (u + 1 < s.u1) fetch(u + 1);
          int mine = 0;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int wb = key0 + 32 * w, rem = s.span.n - wb;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (rem < 32) x[i][w] &= rem > 0 ? (1u << rem) - 1u : 0u;
              const int cut = from[i] - wb;
              if (cut > 0) x[i][w] &= cut < 32 ? ~0u << cut : 0u;
            }
            uni[w] = __reduce_or_sync(0xffffffffu, x[0][w] | x[1][w]);
            mine += __popc(uni[w]);
          }
          if (lane == 0) S.cnt[turn & 1][lw] = mine;
          named_sync(kBarLoad, kTrLoad);
          int before = 0, all = 0;
#pragma unroll
          for (int w = 0; w < kTrLoadWarps; ++w) {
            const int c = S.cnt[turn & 1][w];
            before += w < lw ? c : 0;
            all += c;
          }
          ++turn;
          int at = wrap(head + count + before);  // (head, count <= 128 and before < 512: one wrap at most)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (!uni[w]) continue;
            const uint32_t b0 = transpose32(x[0][w], lane), b1 = transpose32(x[1][w], lane);
            if ((uni[w] >> lane) & 1u) {  // this lane's key
              const int to = wrap(at + __popc(uni[w] & ((1u << lane) - 1u)));
              S.qkey[to] = key0 + 32 * w + lane;
              S.qbits[to] = make_uint2(b0, b1);
            }
            at = wrap(at + __popc(uni[w]));
          }
          count += all;
          named_sync(kBarLoad, kTrLoad);
          while (count > kTrKeys && ok) emit(kTrKeys, seg_flags);
        }
        if (ok) emit(count, last_flags);
      }
    }
    cp_wait<0>();
    if (lt == 0)  // copies still in flight land before the CTA ends
      {
      for (uint32_t i = k_loads > 2 ? k_loads - 2 : 0; i < k_loads; ++i) mbar_drain(&S.k_full[i & 1], (i >> 1) & 1u, A.err);
      for (uint32_t i = it > 2 ? it - 2 : 0; i < it; ++i) mbar_drain(&S.v_full[i & 1], (i >> 1) & 1u, A.err);
      }
  } else if (warp >= 2 * kTrSoft / 32 + kTrLoadWarps) {
    // ---------------- MMA issuer (one elected lane) ----------------
    regs_dec<kTrMmaRegs>();
    if (warp == 2 * kTrSoft / 32 + kTrLoadWarps && lane == 0 && work) {
      constexpr uint32_t idesc_s = umma_idesc_bf16_f32(kTrKeys, kTrStream);
      constexpr uint32_t idesc_o = umma_idesc_bf16_f32(kHeadDim, 2 * kTrStream) | (1u << 15) | (1u << 16);  // MN-major
      auto ready = [&](uint64_t* bar, uint32_t parity) { return mbar_test(bar, parity & 1u); };
      // Op o: the scores, later the product with V, of stream o % 2 and its tile.  Each of these returns false,
      // having done nothing, while something it needs is missing.
      auto tile_of = [](uint32_t o) { return kSplitRows ? o >> 1 : o; };
      auto tile_done = [](uint32_t o) { return !kSplitRows || (o & 1u); };  // no later op of the other stream needs it
      bool seg_start = true, end = false;
      uint32_t segs = 0, epochs[2] = {0u, 0u};
      int end_seg = 0;
      auto issue_s = [&](uint32_t o) -> bool {
        const uint32_t tile = tile_of(o), st = tile & 1, x = o & 1;
        if (!ready(&S.s_free[x], (o >> 1) ^ 1u)) return false;
        if ((!kSplitRows || x == 0) && !ready(&S.k_full[st], tile >> 1)) return false;
        if (seg_start) {
          if (!ready(&S.q_full, segs)) return false;
          ++segs;
          seg_start = false;
        }
        tc_fence_after();
        const uint32_t ka = smem_addr(S.k[st]), qa = smem_addr(S.q) + (kSplitRows ? x * kTrStream * 128u : 0u);
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk) {
          const uint32_t h = (uint32_t)(kk >> 2), b = 32u * (uint32_t)(kk & 3);
          umma_f16(tmem + x * kTmemStream, umma_desc_sw128(ka + h * kTrHalf + b, 16),
                   umma_desc_sw128(qa + h * (NR * 128u) + b, 16), idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit(&S.s_full[x]);
        const int2 meta = S.meta[tile % kTrRing];
        S.cur[x] = make_int4((int)tile, meta.x, meta.y, 0);
        mbar_arrive(&S.s_full[x]);
        if (tile_done(o)) {
          umma_commit(&S.k_empty[st]);
          const int flags = meta.y;
          if (flags & 1) {
            umma_commit(&S.q_free);
            seg_start = true;
          }
          if (flags & 2) {
            end = true;
            end_seg = (flags >> 2) + 1;
          }
        }
        return true;
      };
      auto issue_pv = [&](uint32_t o) -> bool {
        const uint32_t tile = tile_of(o), st = tile & 1, x = o & 1;
        if (!ready(&S.p_full[x], o >> 1) || !ready(&S.v_full[st], tile >> 1)) return false;
        const bool fresh = S.new_epoch[x] != 0;
        uint32_t& ep = x ? epochs[1] : epochs[0];
        if (fresh) {
          if (ep > 0 && !ready(&S.o_free[x], ep - 1)) return false;
          ++ep;
        }
        tc_fence_after();
        const uint32_t va = smem_addr(S.v[st]), pa = smem_addr(S.p[x][0]);
#pragma unroll
        for (int kk = 0; kk < kTrKeys / 16; ++kk)
          umma_f16(tmem + x * kTmemStream + kTmemOe, umma_desc_sw128(va + (uint32_t)kk * 2048u, kTrHalf),
                   umma_desc_sw128(pa + (uint32_t)kk * 2048u, kTrHalf), idesc_o, fresh && kk == 0 ? 0u : 1u);
        if (tile_done(o)) umma_commit(&S.v_empty[st]);
        umma_commit(&S.p_free[x]);
        return true;
      };
      // After the last op one more for each stream, that tells it so: the other may be waiting for its sums.
      auto issue_end = [&](uint32_t o) -> bool {
        const uint32_t x = o & 1;
        if (!ready(&S.s_free[x], (o >> 1) ^ 1u)) return false;
        S.cur[x] = make_int4(-1, 0, 4 * end_seg, 0);
        mbar_arrive(&S.s_full[x]);
        mbar_arrive(&S.s_full[x]);
        return true;
      };
      // Whichever is ready, in each line's order (a stream's scores come after it has read the ones before).
      uint32_t so = 0, po = 0, ops = 0;  // (two more score ops than ops: the ends)
      long long since = clock64();
#pragma unroll 1
      while (!end || po < ops || so < ops + 2) {
        bool moved = false;
        if (!end) {
          if (issue_s(so)) {
            moved = true;
            if (end) ops = so + 1;
            ++so;
          }
        } else if (so < ops + 2 && issue_end(so)) {
          moved = true;
          ++so;
        }
        if (po < so && (!end || po < ops) && issue_pv(po)) {
          moved = true;
          ++po;
        }
        const long long now = clock64();
        if (moved) {
          since = now;
        } else if (now - since > A.budget) {
          atomicExch(A.err, kDevErrTimeout);
          break;
        }
      }
      umma_commit(&S.fin);  // every product issued is done before TMEM is freed
      mbar_drain(&S.fin, 0, A.err);
    }
  } else {
    // ---------------- softmax, output ----------------
    regs_inc<kTrSoftRegs>();
    const int x = tid / kTrSoft;                                 // stream
    const int quad = warp & 3, col0 = 32 * ((warp >> 2) & 1);    // this thread: key (then dim) 32 quad + lane, rows col0 ..
    const int key = 32 * quad + lane;
    const int row_base = row0 + (kSplitRows ? kTrStream * x : 0);
    const int srows = max(0, min(kTrStream, rows - row_base));   // rows of the stream
    const int act = max(0, min(2, (srows - col0 + 15) / 16));    // this thread's 16-row halves that hold rows
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t my_base = lane_base + (uint32_t)x * kTmemStream + (uint32_t)col0;
    const int t_first = (row_base + col0) % A.T;
    float* alpha = S.alpha[x];
    uint32_t* colmax = S.colmax[x];
    const int sc = tid % kTrSoft;                                // thread of the stream
    uint64_t scale2;
    asm("mov.b64 %0, {%1, %1};\n" : "=l"(scale2) : "f"(A.scale_log2));
    auto wait_warp = [&](uint64_t* b, uint32_t parity) {
      if (!__all_sync(0xffffffffu, wait_bar(b, parity & 1u, alive, A))) alive = false;
    };
    auto arrive_warp = [&](uint64_t* b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };

    // The stream's barrier (bounded, as every wait here).
    uint32_t syncs = 0;
    auto sync = [&]() {
      arrive_warp(&S.sync[x]);
      wait_warp(&S.sync[x], syncs++);
    };

    uint64_t l2[16];  // row sums over this thread's keys, in pairs
#pragma unroll
    for (int i = 0; i < 16; ++i) l2[i] = 0ull;
    uint32_t seen = 0u;                   // rows that attend any of them
    int seg = 0;                          // current segment
    int seg_b = 0, seg_n = 0, seg_lo = 0, seg_drafts = 0, seg_depth = 0;  // what its masks need
    int row_depth = 0;                    // (lane c: of row col0 + c)
    bool has = false, has_total = false;  // the stream has taken a tile of it; its epochs have a total
    int in_epoch = 0;
    uint32_t n = 0, checks = 0;           // ops of this stream so far; epochs whose sums were looked at
#pragma unroll 1
    while (work) {
      wait_warp(&S.s_full[x], n);
      if (!alive) break;
      const int4 cur = S.cur[x];
      const bool turn = n == 0 || seg < (cur.z >> 2);

      // ---- segments that ended before this tile: row sums over all keys, then O ----
#pragma unroll 1
      for (; seg < (cur.z >> 2); ++seg) {
        const TrSegInfo& info = S.seg[seg % kTrRing];
        if (has) {
          wait_warp(&S.p_free[x], n - 1);
          tc_fence_after();
        }
        seen = __reduce_or_sync(0xffffffffu, seen);
        if (lane == 0 && seen) atomicOr(&S.seen[x][col0 >> 5], seen);
        seen = 0u;
        // (the stream's P tile is free: 128 keys x 64 rows of partial sums, pairs of rows by key)
        float* scratch = reinterpret_cast<float*>(&S.p[x][0][0]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          reinterpret_cast<uint64_t*>(scratch)[(col0 / 2 + i) * kTrKeys + key] = l2[i];
          l2[i] = 0ull;
        }
        sync();
        const int row = sc >> 2;  // four threads a row, 32 keys each
        float sum = 0.f;
#pragma unroll 16
        for (int i = 0; i < 32; ++i)
          sum += scratch[((row >> 1) * kTrKeys + 32 * (sc & 3) + ((i + lane) & 31)) * 2 + (row & 1)];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const bool mine = (sc & 3) == 0, seen_row = (S.seen[x][row >> 5] >> (row & 31)) & 1u;
        // the row's scale: its reference plus the exponent of its sum (infinite if the sum has left its range or is a
        // NaN: all that it meets becomes a NaN)
        const bool fits = sum >= kTrLow && sum <= kTrTop;
        const float ref = -S.nref[x][row];
        const float lse = !seen_row ? kTrNone : fits ? ref + (float)((int)(__float_as_uint(sum) >> 23) - 127) : INFINITY;
        float m = lse, all = sum;  // the piece: 2^m all
        if constexpr (kSplitRows) {
          all = !seen_row ? 0.f : fits ? sum * ex2a(ref - m) : INFINITY;
          if (mine) alpha[row] = !seen_row ? 0.f : fits ? 1.f / sum : __int_as_float(0x7fffffff);
        } else {  // with the other stream's
          if (mine) {
            alpha[row] = lse;
            S.sum[x][row] = sum;
          }
          if (sc == 0) S.state[x] = (has ? 1 : 0) + (has_total ? 2 : 0);
          tc_fence_before();
          arrive_warp(&S.sum_full[x]);
          wait_warp(&S.sum_full[x], (uint32_t)seg);
          wait_warp(&S.sum_full[x ^ 1], (uint32_t)seg);
          tc_fence_after();
          if (mine) {
            const float a = S.alpha[0][row], b = S.alpha[1][row];
            m = fmaxf(a, b);
            const float fa = a <= kTrNone ? 0.f : ex2a(-S.nref[0][row] - m);
            const float fb = b <= kTrNone ? 0.f : ex2a(-S.nref[1][row] - m);
            all = S.sum[0][row] * fa + S.sum[1][row] * fb;
            const float inv = m <= kTrNone ? 0.f : 1.f / all;
            S.wt[x][0][row] = fa * inv;
            S.wt[x][1][row] = fb * inv;
          }
        }
        if (!alive) break;
        if (info.slot >= 0 && mine && row < srows && (kSplitRows || x == 0))
          W.ml[(int64_t)info.slot * NR + row_base - row0 + row] = make_float2(m, all);
        sync();
        // eight rows at a time: all 32 of this thread's, or 16 when the streams share them
        const int c_first = kSplitRows ? col0 : col0 + 16 * x;
#pragma unroll 1
        for (int c0 = c_first; c0 < c_first + (kSplitRows ? 32 : 16) && c0 < srows; c0 += 8) {
          float y[8], e[kSplitRows ? 1 : 2][3][8];  // of each stream: the epoch's O (hi, lo), the total
#pragma unroll
          for (int k = 0; k < (kSplitRows ? 1 : 2); ++k) {
            const int src = kSplitRows ? x : k, state = kSplitRows ? 1 + (has_total ? 2 : 0) : S.state[src];
            const uint32_t at = lane_base + (uint32_t)src * kTmemStream + (uint32_t)c0;
#pragma unroll
            for (int i = 0; i < 24; ++i) e[k][i / 8][i % 8] = 0.f;
            if (state & 1) {
              tmem_ld8(at + kTmemOe, e[k][0]);
              tmem_ld8(at + kTmemOe + kTrStream, e[k][1]);
            }
            if (state & 2) tmem_ld8(at + kTmemOt, e[k][2]);
          }
#pragma unroll
          for (int k = 0; k < (kSplitRows ? 1 : 2); ++k) {
            const float* wt = kSplitRows ? alpha : S.wt[kSplitRows ? 0 : x][k];
            tmem_wait(e[k][0]);
            tmem_wait(e[k][1]);
            tmem_wait(e[k][2]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float sum_e = e[k][0][i] + e[k][1][i] + e[k][2][i];
              y[i] = k == 0 ? sum_e * wt[c0 + i] : __fmaf_rn(sum_e, wt[c0 + i], y[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) scratch[(c0 + i) * kHeadDim + key] = y[i];
        }
        tc_fence_before();
        if constexpr (!kSplitRows) {  // both streams are done with each other's sums
          arrive_warp(&S.sum_free[x ^ 1]);
          wait_warp(&S.sum_free[x], (uint32_t)seg);
        }
        if (has) arrive_warp(&S.o_free[x]);
        sync();
        // a warp per row: out, or to where the pieces of the group meet
        const int64_t o_seg = info.b * A.o.sb + (int64_t)info.kvh * A.G * A.o.sh;
        float4* part = reinterpret_cast<float4*>(W.o) + ((int64_t)info.slot * NR + row_base - row0) * 32 + lane;
#pragma unroll 4
        for (int i = warp & 7; i < (kSplitRows ? 64 : 32); i += 8) {
          const int c = kSplitRows ? i : (i & 15) + 32 * (i >> 4) + 16 * x;  // (the rows whose columns were this stream's)
          if (c >= srows) continue;
          float4 y = reinterpret_cast<const float4*>(scratch)[c * 32 + lane];
          if (info.slot >= 0) {
            part[c * 32] = y;
          } else {
            const int at = S.row_at[row_base - row0 + c];
            if (__any_sync(0xffffffffu, !finite4(y))) scalar_row(A, info.b, info.kvh * A.G + (at & 7), at >> 3, y);
            store4(A, o_seg + (at & 7) * A.o.sh + (at >> 3) * A.o.sn + 4 * lane, y);
          }
        }
        if (srows < kTrStream) {  // P's columns past the last row are zeros again
          sync();
#pragma unroll 1
          for (int i = sc; i < kTrKeys * kTrStream / 4; i += kTrSoft)
            reinterpret_cast<uint4*>(scratch)[i] = make_uint4(0u, 0u, 0u, 0u);
          fence_async();
        }
        if (sc < 2) S.seen[x][sc] = 0u;
        has = has_total = false;
        sync();  // (from here on the stream's arrays are the next segment's)
      }
      if (cur.x < 0 || !alive) break;
      if (turn) {
        const TrSegInfo& info = S.seg[seg % kTrRing];
        seg_b = info.b;
        seg_n = info.n;
        seg_lo = info.lo;
        seg_drafts = info.draft_tiles;
        seg_depth = info.max_depth;
        row_depth = draft_depth(A, seg_b, (t_first + lane) % A.T);
      }

      // ---- which of this thread's rows attend its key, and whether it is one at all ----
      uint32_t mw = ~0u;
      bool is_key;
      if (cur.y < seg_drafts) {
        const int j = cur.y * kTrKeys + key;
        is_key = j < A.T;
        // lane c reads the tree word of row c; transposed, a lane has its key's bits over the rows
        const bool words = cur.y * kTrKeys + 32 * quad < A.T && col0 + lane < srows;
        mw = transpose32(words ? __ldg(A.tree + ((int64_t)seg_b * A.T + (t_first + lane) % A.T) * A.tree_words +
                                       4 * cur.y + quad)
                               : 0u,
                         lane);
        if (!is_key) mw = 0u;
        if (A.W > 0 && seg_depth >= A.W) {
          const int dj = is_key ? draft_depth(A, seg_b, j) : 0;
          uint32_t in = 0u;
#pragma unroll 4
          for (int c = 0; c < 32; ++c) in |= (uint32_t)(dj > __shfl_sync(0xffffffffu, row_depth, c) - A.W) << c;
          mw &= in;
        }
      } else if constexpr (SEL) {
        mw = S.kmask[cur.x & 3][col0 >> 5][key];
        is_key = mw != 0u;
      } else {
        const uint32_t p0 = (uint32_t)seg_lo + (uint32_t)(cur.y - seg_drafts) * kTrKeys;
        const int age = seg_n - 1 - (int)(p0 + (uint32_t)key);  // (below 0: past the end)
        is_key = age >= 0;
        if (!is_key) mw = 0u;
        if (A.W > 0 && seg_n - 1 - (int)p0 > oldest_age(A, seg_depth)) {
          uint32_t in = 0u;
#pragma unroll 4
          for (int c = 0; c < 32; ++c)
            in |= (uint32_t)(age <= oldest_age(A, __shfl_sync(0xffffffffu, row_depth, c))) << c;
          mw &= in;
        }
      }
      seen |= mw;

      const bool fresh = !has || in_epoch == kTrEpoch;
      bool raise = false;
      tc_fence_after();
      if (!has) {
        // the references: each row's logit of the tile's first key, as a whole number (so that no factor between
        // references rounds)
        if (quad == 0) {
#pragma unroll 1
          for (int hh = 0; hh < act; ++hh) {
            uint32_t v[16];
            tmem_ld16(my_base + 16u * hh, v);
            tmem_wait(v);
            if (lane == 0) {
#pragma unroll
              for (int c = 0; c < 16; c += 4) {
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  y[i] = -rintf(__uint_as_float(v[c + i]) * A.scale_log2);
                  y[i] = (fabsf(y[i]) < 1e30f) & is_key ? y[i] : 0.f;
                }
                *reinterpret_cast<float4*>(&S.nref[x][col0 + 16 * hh + c]) = make_float4(y[0], y[1], y[2], y[3]);
              }
            }
          }
        }
        sync();
      } else if (fresh) {
        // an epoch is over: raise the references of rows whose sums have grown large, by a power of two
        float l[32], top = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          unpack2(l2[i], l[2 * i], l[2 * i + 1]);
          top = max3f(top, l[2 * i], l[2 * i + 1]);
        }
        const uint32_t e = checks++ & 1u;
        if (__any_sync(0xffffffffu, top > kTrHigh)) {
          const float m = reduce_columns<16>(l, lane, [](float a, float b) { return fmaxf(a, b); });
          atomicMax(&colmax[col0 + lane], __float_as_uint(fmaxf(m, 0.f)));
          if (lane == 0) S.raise[x][e] = 1;
        }
        sync();
        raise = S.raise[x][e] != 0;
        if (sc == 0) S.raise[x][e ^ 1u] = 0;
        if (raise) {
          if (sc < kTrStream) {
            const float up = __uint_as_float(colmax[sc]);
            const float by = up > kTrHigh ? (float)ilogbf(up) : 0.f;
            S.nref[x][sc] -= by;
            alpha[sc] = up <= kTrTop ? ex2a(-by) : __int_as_float(0x7fffffff);  // (out of range: the scalar way)
          }
          sync();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            unpack2(l2[i], a, b);
            l2[i] = pack2(a * alpha[col0 + 2 * i], b * alpha[col0 + 2 * i + 1]);
          }
        }
        if (sc < kTrStream) colmax[sc] = 0u;  // (the next epoch's sums come after a wait of all)
      }

      // ---- P = 2^(logit - reference) as bf16 hi + lo, key-major rows of 64 query rows (128 bytes, swizzled) ----
      auto scores = [&](int hh, const uint32_t (&v)[16], float (&d)[16]) {
        const ulonglong2* nr = reinterpret_cast<const ulonglong2*>(S.nref[x] + col0 + 16 * hh);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ulonglong2 r = nr[i];
          fma2c(v[4 * i], v[4 * i + 1], scale2, r.x, d[4 * i], d[4 * i + 1]);
          fma2c(v[4 * i + 2], v[4 * i + 3], scale2, r.y, d[4 * i + 2], d[4 * i + 3]);
        }
        if (mw != ~0u) {
          const uint32_t w = mw >> (16 * hh);
#pragma unroll
          for (int c = 0; c < 16; ++c) d[c] = (w >> c) & 1u ? d[c] : -INFINITY;
        }
      };
      uint32_t hi_w[8], lo_w[8];
      auto exps = [&](int hh, const float (&d)[16]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t p = pack2(ex2a(d[2 * i]), ex2a(d[2 * i + 1]));
          l2[8 * hh + i] = add2u(l2[8 * hh + i], p);
          float p0, p1;
          unpack2(p, p0, p1);
          hi_w[i] = pack_bf16x2(p0, p1);
          unpack2(sub2u(p, pack2(bf16_lo(hi_w[i]), bf16_hi(hi_w[i]))), p0, p1);
          lo_w[i] = pack_bf16x2(p0, p1);
        }
      };
      auto put = [&](int hh) {
        const int c8 = (col0 + 16 * hh) >> 3;  // first 16-byte chunk of these rows
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t o = (uint32_t)key * 128u + (uint32_t)(((c8 + i) ^ (key & 7)) << 4);
          *reinterpret_cast<uint4*>(&S.p[x][0][o]) =
              make_uint4(hi_w[4 * i], hi_w[4 * i + 1], hi_w[4 * i + 2], hi_w[4 * i + 3]);
          *reinterpret_cast<uint4*>(&S.p[x][1][o]) =
              make_uint4(lo_w[4 * i], lo_w[4 * i + 1], lo_w[4 * i + 2], lo_w[4 * i + 3]);
        }
      };
      if (act > 0) {
        uint32_t v[16];
        float d[16];
        tmem_ld16(my_base, v);
        tmem_wait(v);
        scores(0, v, d);
        if (act > 1) tmem_ld16(my_base + 16u, v);
        exps(0, d);
        wait_warp(&S.p_free[x], n ^ 1u);
        put(0);
        if (act > 1) {
          tmem_wait(v);
          tc_fence_before();
          arrive_warp(&S.s_free[x]);
          scores(1, v, d);
          exps(1, d);
          put(1);
        }
      } else {
        wait_warp(&S.p_free[x], n ^ 1u);
      }
      if (act < 2) {
        tc_fence_before();
        arrive_warp(&S.s_free[x]);
      }
      fence_async();
      if (sc == 0) S.new_epoch[x] = fresh;
      arrive_warp(&S.p_full[x]);

      // ---- the epoch before this tile joins the total ----
      if (fresh && has) {
        tc_fence_after();  // (its last product is done: p_free above)
#pragma unroll 1
        for (int c0 = 0; c0 < 16 * act; c0 += 8) {
          float e[8], r[8];
          tmem_ld8(my_base + kTmemOe + c0, e);
          tmem_ld8(my_base + kTmemOe + kTrStream + c0, r);
          tmem_wait(e);
          tmem_wait(r);
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] += r[i];
          if (has_total) {
            tmem_ld8(my_base + kTmemOt + c0, r);
            tmem_wait(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] += r[i];
          }
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(raise ? e[i] * alpha[col0 + c0 + i] : e[i]);
          tmem_st8(my_base + kTmemOt + c0, o);
        }
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(&S.o_free[x]);
        has_total = true;
      }

      in_epoch = fresh ? 1 : in_epoch + 1;
      has = true;
      ++n;
      if (!alive) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_free(tmem, kTmemCols);
}

// Joins the pieces of groups that several CTAs worked on: WPR warps per query row, pieces in turn, four
// head dims per lane.
constexpr int kTrJoinThreads = 256;
template <int WPR>
__global__ void __launch_bounds__(kTrJoinThreads) tree_join_kernel(const __grid_constant__ TreeAttnArgs A,
                                                                   const __grid_constant__ TrParts W) {
  constexpr int kWarps = kTrJoinThreads / 32;
  __shared__ float4 so[kWarps][32];
  __shared__ float2 sml[kWarps];
  pdl_wait();
  pdl_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WPR;
  const int64_t rows = (int64_t)A.G * A.T, x = (int64_t)blockIdx.x * (kWarps / WPR) + warp / WPR;
  const bool have = x < rows * A.B * A.Hk;
  const int grp = have ? (int)(x / rows) : 0, r = have ? (int)(x % rows) : 0;
  const int2 pieces = have ? W.table[grp] : make_int2(0, 1);
  const bool join = pieces.y > 1;  // (one piece: its CTA has written the output)
  float m = kTrNone, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  // one more piece (or partial join): 2^s w to the sum, 2^s v y to the output (an infinite s makes both NaNs)
  auto take = [&](float s, float w, float v, const float4& y, float mn) {
    const float f = s <= kTrNone ? 0.f : ex2a(s - mn);
    if (f == 0.f && w == w) return;  // (what it holds may be anything)
    l += f * w;
    const float g = f * v;
    o = make_float4(o.x + g * y.x, o.y + g * y.y, o.z + g * y.z, o.w + g * y.w);
  };
  if (join) {
    const int c = r % W.nr;
    const int64_t slot0 = (int64_t)(r / W.nr) * 2 * W.ranges;
    auto at = [&](int i) { return (slot0 + 2 * (pieces.x + i) + (i == 0)) * W.nr + c; };
    constexpr int kUnroll = 4;
    for (int i = part; i < pieces.y; i += WPR * kUnroll) {
      float2 s[kUnroll];
      float4 y[kUnroll];
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        const int p = i + WPR * q;
        s[q] = make_float2(kTrNone, 0.f);
        y[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < pieces.y) {
          s[q] = W.ml[at(p)];
          y[q] = reinterpret_cast<const float4*>(W.o + at(p) * kHeadDim)[lane];
        }
      }
      float mn = m;
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) mn = fmaxf(mn, s[q].x);
      const float al = ex2a(m - mn);
      m = mn;
      l *= al;
      o = make_float4(o.x * al, o.y * al, o.z * al, o.w * al);
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) take(s[q].x, s[q].y, s[q].y, y[q], mn);
    }
  }
  if (WPR > 1) {
    so[warp][lane] = o;
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (part != 0) return;
    float M = kTrNone;
#pragma unroll
    for (int w = 0; w < WPR; ++w) M = fmaxf(M, sml[warp + w].x);
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WPR; ++w) take(sml[warp + w].x, sml[warp + w].y, 1.f, so[warp + w][lane], M);
  }
  if (!join) return;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  const int b = grp / A.Hk, h = grp % A.Hk * A.G + r / A.T, t = r % A.T;
  if (__any_sync(0xffffffffu, !finite4(o))) scalar_row(A, b, h, t, o);
  store4(A, b * A.o.sb + h * A.o.sh + t * A.o.sn + 4 * lane, o);
}

template <int NR, bool SEL>
cudaError_t launch_tiles(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeAttnArgs& a, const TrParts& w,
                         int use_tma, cudaStream_t stream) {
  const size_t smem = sizeof(TrSmem<NR>);
  static_assert(sizeof(TrSmem<NR>) <= 232448, "shared memory of one CTA");
  cudaError_t e =
      cudaFuncSetAttribute(tree_attn_kernel<NR, SEL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_attn_kernel<NR, SEL>, dim3((unsigned)(w.rbs * w.ranges)), dim3(kTrThreads), smem, stream, 1,
                    kmap, vmap, a, w, use_tma);
}

template <int WPR>
cudaError_t launch_join(const TreeAttnArgs& a, const TrParts& w, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.B * a.Hq * a.T, per = kTrJoinThreads / 32 / WPR;
  return launch_pdl(tree_join_kernel<WPR>, dim3((unsigned)((rows + per - 1) / per)), dim3(kTrJoinThreads), 0, stream, 1,
                    a, w);
}

}  // namespace

size_t tree_attn_workspace_bytes(int64_t B, int64_t Hq, int64_t T, int64_t Hk, int64_t N) {
  (void)N;
  const size_t plain = tree_layout(B, Hq, T, Hk, false).bytes(), sel = tree_layout(B, Hq, T, Hk, true).bytes();
  return plain > sel ? plain : sel;
}

cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t stream) {
  if ((int64_t)a.B * a.Hq * a.T == 0) return cudaSuccess;
  const TrLayout L = tree_layout(a.B, a.Hq, a.T, a.Hk, a.sel != nullptr);
  TrParts w;
  char* ws = static_cast<char*>(a.ws);
  w.table = reinterpret_cast<int2*>(ws);
  w.o = reinterpret_cast<float*>(ws + L.table);
  w.ml = reinterpret_cast<float2*>(ws + L.table + L.o);
  w.nr = L.nr;
  w.rbs = L.rbs;
  w.ranges = L.ranges;
  // strides that the tensor map's encoder refuses (0 in a dim of several rows): every tile by cp.async
  CUtensorMap kmap{}, vmap{};
  const int use_tma = !a.sel && a.N >= kTrKeys && make_row_map(&kmap, a.k, a.B, a.Hk, a.N, kTrKeys) &&
                      make_row_map(&vmap, a.v, a.B, a.Hk, a.N, kTrKeys);
  const cudaError_t e = a.sel          ? launch_tiles<64, true>(kmap, vmap, a, w, 0, stream)
                        : L.nr == 64 ? launch_tiles<64, false>(kmap, vmap, a, w, use_tma, stream)
                                     : launch_tiles<128, false>(kmap, vmap, a, w, use_tma, stream);
  if (e != cudaSuccess) return e;
  // about this many pieces in a group: one warp per row takes four at a time
  const int64_t pieces = L.ranges / ((int64_t)a.B * a.Hk) + 1;
  if (pieces <= 4) return launch_join<1>(a, w, stream);
  if (pieces <= 16) return launch_join<4>(a, w, stream);
  return launch_join<8>(a, w, stream);
}

}  // namespace rtp
