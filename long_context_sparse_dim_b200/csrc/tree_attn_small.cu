// rtp_tree_attn over few keys: the latency form.
//
// A call over a thousand keys is a few microseconds of work, and the persistent
// forms (tree_attn.cu, tree_attn_wide.cu) spend ten on their warp roles, their
// search for a CTA's share of the work and their cold code.  Here a CTA is one
// block of 64 query rows of a KV head and one tile of 64 of its keys, found by
// block index alone: gather, one product, a softmax, the other product, out.
//
// Four warps of mma.sync m16n8k16: with R rows in the block, warps take 16 rows
// each and, when R is below 64, share out the 64 keys, too (RG row groups x 4 /
// RG key groups, met in shared memory at the end).  K and V rows come by 16-byte
// cp.async with zeros in the rows that hold no token.  P as a bf16 hi + lo pair
// in registers (three terms, all 24 bits, for fp32 outputs: nothing here waits on
// the tensor core); fp32 sums.  The tiles of a group are joined by the kernel that
// joins the other forms' pieces.
//
// Bound by latency: 1000 keys x 8 drafts of 8 KV heads (4 MB) take 11.1 us,
// launches back to back, of which 7.5 are this kernel's and the rest the join's;
// the persistent form takes 19.0.  (One tile to a CTA: with several the CTAs are
// fewer and larger, 11.8 us, and three of them fit on an SM, not two.)
#include "tree_attn.cuh"

namespace rtp {

namespace {

constexpr int kSmThreads = 128;
constexpr int kSmRows = 64;       // query rows of a block
constexpr int kSmKeys = 64;       // keys of a tile
constexpr int kSmTile = kSmKeys * 256;

struct SmSmem {
  alignas(128) uint8_t q[kSmRows * 256];
  alignas(128) uint8_t k[kSmTile];
  alignas(128) uint8_t v[kSmTile];  // (k and v: at the end the rows' O)
  float2 ml[4][16];                    // per warp: its rows' maxima and sums
  float2 row_ml[kSmRows];
};

// Offset of 16-byte chunk c of row r (rows of 256 bytes, chunk index XOR row % 8).
RTP_DEVICE uint32_t swz(int r, int c) { return (uint32_t)(r * 256 + ((c ^ (r & 7)) << 4)); }
RTP_DEVICE void ldsm(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
RTP_DEVICE void ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
RTP_DEVICE void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// RG: groups of 16 query rows among the four warps (1, 2 or 4).
template <int RG>
__global__ void __launch_bounds__(kSmThreads)
tree_attn_small_kernel(const __grid_constant__ TreeAttnArgs A, const __grid_constant__ TrParts W) {
  constexpr int KG = 4 / RG, KW = kSmKeys / KG;  // key groups; keys of a tile per warp
  extern __shared__ __align__(128) unsigned char smem_raw[];
  SmSmem& S = *reinterpret_cast<SmSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rb = blockIdx.y % W.rbs, grp = blockIdx.y / W.rbs;
  const int b = grp / A.Hk, kvh = grp - b * A.Hk;
  const int row0 = rb * kSmRows, rows = A.G * A.T, nrows = min(kSmRows, rows - row0);
  pdl_wait();
  pdl_release();
  const int n = committed(A, b);
  const int lo = A.W > 0 ? max(0, n - (A.W - 1)) : 0, lo_al = A.sel ? lo / kSmKeys * kSmKeys : lo;
  const int draft_tiles = (A.T + kSmKeys - 1) / kSmKeys;
  const int tiles = draft_tiles + (int)(((uint32_t)(n - lo_al) + kSmKeys - 1) / kSmKeys);
  const int u = blockIdx.x;
  if (u >= tiles) return;
  if (u == 0 && rb == 0 && tid == 0) W.table[grp] = make_int2(0, tiles);
  const bool draft = u < draft_tiles;
  const int key0 = draft ? u * kSmKeys : lo_al + (u - draft_tiles) * kSmKeys, keys_left = (draft ? A.T : n) - key0;

  // ---- loads: this thread's 16-byte column of rows tid / 16 + 8 i ----
  const int col = tid & 15, r_first = tid >> 4;
  const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(A.q.data) + b * A.q.sb + (int64_t)kvh * A.G * A.q.sh;
#pragma unroll
  for (int i = 0; i < RG * 2; ++i) {
    const int r = r_first + 8 * i, rr = min(row0 + r, rows - 1), g = rr / A.T, t = rr - g * A.T;
    cp16(smem_addr(S.q) + swz(r, col), qb + g * A.q.sh + t * A.q.sn + col * 8, r < nrows);
  }
  // keys of the tile that some row of the block selected (all, without a selection)
  const uint32_t* sel_rows =
      A.sel ? A.sel + ((int64_t)(b * A.Hq + kvh * A.G) * A.T + row0) * A.sel_words : nullptr;
  uint64_t keys = ~0ull;
  if (A.sel && !draft) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll 1
      for (int r = lane; r < nrows; r += 32)
        if (32 * i < keys_left) w[i] |= __ldg(sel_rows + (int64_t)r * A.sel_words + (key0 >> 5) + i);
    keys = (uint64_t)__reduce_or_sync(0xffffffffu, w[1]) << 32 | __reduce_or_sync(0xffffffffu, w[0]);
  }
  int64_t row[8];  // (-1: no token)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r_first + 8 * i;
    const bool ok = r < keys_left && ((keys >> r) & 1ull);
    row[i] = !ok ? -1 : draft ? key0 + r : row_of(A, (uint32_t)(key0 + r));
  }
  auto load = [&](const View4& x, uint8_t* to) {
    const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(x.data) + b * x.sb + kvh * x.sh + col * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      cp16(smem_addr(to) + swz(r_first + 8 * i, col), row[i] >= 0 ? (const void*)(from + row[i] * x.sn) : A.q.data,
           row[i] >= 0);
    cp_commit();
  };
  load(draft ? A.kn : A.k, S.k);
  load(draft ? A.vn : A.v, S.v);

  // ---- this thread's two rows of the products: 16 rg + g8 and 8 further ----
  const int rg = warp % RG, kg = warp / RG, g8 = lane >> 2, c2 = 2 * (lane & 3);
  int t_row[2], old_row[2];
  bool live[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 16 * rg + g8 + 8 * i, rr = min(row0 + r, rows - 1);
    live[i] = r < nrows;
    t_row[i] = rr % A.T;
    old_row[i] = A.W > 0 ? oldest_age(A, draft_depth(A, b, t_row[i])) : 0;
  }

  float m[2], l[2] = {0.f, 0.f};
  float o[16][4];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  cp_wait<1>();
  __syncthreads();

  // S = Q K^T: 16 rows x KW keys
  float s[KW / 8][4];
#pragma unroll
  for (int i = 0; i < KW / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
  const uint32_t ka = smem_addr(S.k), va = smem_addr(S.v), qa = smem_addr(S.q);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    uint32_t a[4];
    ldsm(qa + swz(16 * rg + (lane & 15), 2 * kk + (lane >> 4)), a);
#pragma unroll
    for (int i = 0; i < KW / 16; ++i) {
      uint32_t bb[4];
      ldsm(ka + swz(KW * kg + 16 * i + (lane & 7) + 8 * (lane >> 4), 2 * kk + ((lane >> 3) & 1)), bb);
      mma16(s[2 * i], a, bb[0], bb[1]);
      mma16(s[2 * i + 1], a, bb[2], bb[3]);
    }
  }
  // which of them each row attends (bit j of `in`: key KW kg + j of the tile)
  const int p0 = key0 + KW * kg, left = keys_left - KW * kg;
  float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint64_t in = left >= 64 ? ~0ull : left > 0 ? (1ull << left) - 1ull : 0ull;
    if (draft) {
      const uint32_t* words = A.tree + ((int64_t)b * A.T + t_row[h]) * A.tree_words;
      const int j0 = p0 & ~31, sh = p0 & 31;  // (KW = 16: a half word)
      uint64_t bits = j0 < A.T ? __ldg(words + (j0 >> 5)) : 0u;
      if (KW == 64 && j0 + 32 < A.T) bits |= (uint64_t)__ldg(words + (j0 >> 5) + 1) << 32;
      in &= bits >> sh;
      const int depth = A.W > 0 ? draft_depth(A, b, t_row[h]) : 0;
      if (A.W > 0 && depth >= A.W) {  // (below it the window holds every draft)
#pragma unroll 1
        for (int j = 0; j < KW && j < left; ++j)
          if (draft_depth(A, b, p0 + j) <= depth - A.W) in &= ~(1ull << j);
      }
    } else {
      if (A.sel) {
        const uint32_t* words = sel_rows + (int64_t)min(16 * rg + g8 + 8 * h, nrows - 1) * A.sel_words;
        const int j0 = p0 & ~31, sh = p0 & 31;
        uint64_t bits = j0 < n ? __ldg(words + (j0 >> 5)) : 0u;
        if (KW == 64 && j0 + 32 < n) bits |= (uint64_t)__ldg(words + (j0 >> 5) + 1) << 32;
        in &= bits >> sh;
      }
      if (A.W > 0) {  // key j is left - 1 - j tokens older than the newest
        const int cut = old_row[h] < 0 ? 64 : max(left - 1 - old_row[h], 0);
        in &= cut < 64 ? ~0ull << cut : 0ull;
      }
    }
    if (!live[h]) in = 0ull;
    in >>= c2;  // bit 8 i + e
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float y = s[i][2 * h + e] * A.scale_log2;
        s[i][2 * h + e] = ((i < 4 ? (uint32_t)in : (uint32_t)(in >> 32)) >> (8 * (i & 3) + e)) & 1u ? y : -INFINITY;
        top[h] = fmaxf(top[h], s[i][2 * h + e]);
      }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], d));
    m[h] = top[h];
    const float ref = top[h] == -INFINITY ? 0.f : top[h];
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float p = ex2a(s[i][2 * h + e] - ref);
        s[i][2 * h + e] = p;
        l[h] += p;
      }
  }
  // O = P V
  cp_wait<0>();
  __syncthreads();
#pragma unroll
  for (int ks = 0; ks < KW / 16; ++ks) {
    uint32_t hi[4], lw[4], ll[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p0v = s[2 * ks + (i >> 1)][2 * (i & 1)], p1v = s[2 * ks + (i >> 1)][2 * (i & 1) + 1];
      hi[i] = pack_bf16x2(p0v, p1v);
      const float r0 = p0v - bf16_lo(hi[i]), r1 = p1v - bf16_hi(hi[i]);
      lw[i] = pack_bf16x2(r0, r1);
      ll[i] = pack_bf16x2(r0 - bf16_lo(lw[i]), r1 - bf16_hi(lw[i]));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t bb[4];
      ldsm_t(va + swz(KW * kg + 16 * ks + (lane & 15), 2 * i + (lane >> 4)), bb);
      mma16(o[2 * i], hi, bb[0], bb[1]);
      mma16(o[2 * i + 1], hi, bb[2], bb[3]);
      mma16(o[2 * i], lw, bb[0], bb[1]);
      mma16(o[2 * i + 1], lw, bb[2], bb[3]);
      if (!A.o_bf16) {
        mma16(o[2 * i], ll, bb[0], bb[1]);
        mma16(o[2 * i + 1], ll, bb[2], bb[3]);
      }
    }
  }
  __syncthreads();  // (O goes over K and V)
  // ---- the warps' rows together: O in shared memory, key groups in turn ----
  float* acc = reinterpret_cast<float*>(S.k);  // [rows][128]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], d);
    if ((lane & 3) == 0) S.ml[warp][g8 + 8 * h] = make_float2(m[h], l[h]);
  }
  __syncthreads();
  float f[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float M = -INFINITY, all = 0.f;
#pragma unroll
    for (int k = 0; k < KG; ++k) M = fmaxf(M, S.ml[rg + RG * k][g8 + 8 * h].x);
#pragma unroll
    for (int k = 0; k < KG; ++k) {
      const float2 x = S.ml[rg + RG * k][g8 + 8 * h];
      all += x.x == -INFINITY ? x.y : x.y * ex2a(x.x - M);
    }
    const float inv = all != 0.f ? 1.f / all : 0.f;
    f[h] = m[h] == -INFINITY ? inv : ex2a(m[h] - M) * inv;
    if (kg == 0 && (lane & 3) == 0)
      // (a maximum near the one that stands for no key at all: poisoned, for the join to compute the row anew)
      S.row_ml[16 * rg + g8 + 8 * h] =
          make_float2(M == -INFINITY && all == 0.f ? kTrNone : M < 0.5f * kTrNone ? INFINITY : M, all);
  }
#pragma unroll
  for (int k = 0; k < KG; ++k) {
    if (kg == k) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2* p = reinterpret_cast<float2*>(acc + (16 * rg + g8 + 8 * h) * kHeadDim + 8 * i + c2);
          float2 y = make_float2(o[i][2 * h] * f[h], o[i][2 * h + 1] * f[h]);
          if (k > 0) y = make_float2(p->x + y.x, p->y + y.y);
          *p = y;
        }
    }
    __syncthreads();
  }
  const int64_t slot = ((int64_t)blockIdx.y * gridDim.x + u) * kSmRows;
#pragma unroll 2
  for (int r = warp; r < nrows; r += 4) {
    const float4 y = reinterpret_cast<const float4*>(acc)[r * 32 + lane];
    if (tiles > 1) {
      reinterpret_cast<float4*>(W.o)[(slot + r) * 32 + lane] = y;
      if (lane == 0) W.ml[slot + r] = S.row_ml[r];
    } else {
      const int g = (row0 + r) / A.T, t = row0 + r - g * A.T, h = kvh * A.G + g;
      store4(A, b * A.o.sb + h * A.o.sh + t * A.o.sn + 4 * lane, y);
    }
  }
}

template <int RG>
cudaError_t launch(const TreeAttnArgs& a, const TrParts& w, int tiles, cudaStream_t stream) {
  const size_t smem = sizeof(SmSmem);
  cudaError_t e =
      cudaFuncSetAttribute(tree_attn_small_kernel<RG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_attn_small_kernel<RG>, dim3((unsigned)tiles, (unsigned)(a.B * a.Hk * w.rbs)),
                    dim3(kSmThreads), smem, stream, 1, a, w);
}

}  // namespace

cudaError_t launch_tree_attn_small(const TreeAttnArgs& a, const TrParts& w, int tiles, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.G * a.T;
  if (rows <= 16) return launch<1>(a, w, tiles, stream);
  if (rows <= 32) return launch<2>(a, w, tiles, stream);
  return launch<4>(a, w, tiles, stream);
}

}  // namespace rtp
