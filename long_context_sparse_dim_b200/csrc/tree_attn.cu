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
#include <math.h>

#include "common.cuh"
#include "launch.h"

namespace rtp {

namespace {

constexpr int kTrThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

// Committed tokens of sequence b, and how many cache rows hold one of them.
RTP_DEVICE int committed(const TreeAttnArgs& A, int b) {
  const int n = A.lens ? max(A.lens[b], 0) : A.N;
  return A.ring ? n : min(n, A.N);
}

// Tokens between cache row j and the newest committed one (0: the newest).
RTP_DEVICE int row_age(const TreeAttnArgs& A, int n, int j) {
  if (!A.ring || n <= A.N) return n - 1 - j;
  const int newest = (n - 1) % A.N;
  return newest >= j ? newest - j : newest - j + A.N;
}

RTP_DEVICE float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// One CTA per (sequence, query head, draft); its warps take keys in turn.
__global__ void __launch_bounds__(kTrThreads) tree_attn_kernel(TreeAttnArgs A) {
  __shared__ float wm[4], wl[4];
  __shared__ __align__(16) float wo[4][kHeadDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, bh = blockIdx.y;
  const int b = bh / A.Hq, h = bh % A.Hq, kvh = h / A.G;
  const int n = committed(A, b), used = min(n, A.N);
  const int depth = A.W > 0 ? max(A.depth[(int64_t)b * A.T + t], 0) : 0;
  auto row = [&](const View4& x, int head, int64_t r) {
    return static_cast<const __nv_bfloat16*>(x.data) + b * x.sb + head * x.sh + r * x.sn + 4 * lane;
  };
  auto load = [](const __nv_bfloat16* p) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  };
  const float4 q = load(row(A.q, h, t));
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto take = [&](const __nv_bfloat16* kp, const __nv_bfloat16* vp) {
    const float4 k = load(kp), v = load(vp);
    const float s = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w) * A.scale_log2;
    const float mn = fmaxf(m, s);
    const float al = mn == -INFINITY ? 1.f : ex2(m - mn), p = mn == -INFINITY ? 0.f : ex2(s - mn);
    m = mn;
    l = l * al + p;
    o = make_float4(o.x * al + p * v.x, o.y * al + p * v.y, o.z * al + p * v.z, o.w * al + p * v.w);
  };
  const uint32_t* sel = A.sel ? A.sel + ((int64_t)bh * A.T + t) * A.sel_words : nullptr;
  const int oldest = A.W > 0 ? A.W - 2 - depth : n;  // age of the oldest committed key the token attends
  const int first = A.ring ? 0 : oldest < 0 ? used : max(0, n - 1 - oldest);
  for (int j = first + warp; j < used; j += 4) {
    if (row_age(A, n, j) > oldest) continue;
    if (sel && !((__ldg(sel + (j >> 5)) >> (j & 31)) & 1u)) continue;
    take(row(A.k, kvh, j), row(A.v, kvh, j));
  }
  const uint32_t* tree = A.tree + ((int64_t)b * A.T + t) * A.tree_words;
  for (int j = warp; j < A.T; j += 4) {
    if (!((__ldg(tree + (j >> 5)) >> (j & 31)) & 1u)) continue;
    if (A.W > 0 && max(A.depth[(int64_t)b * A.T + j], 0) <= depth - A.W) continue;
    take(row(A.kn, kvh, j), row(A.vn, kvh, j));
  }
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
  reinterpret_cast<float4*>(wo[warp])[lane] = o;
  __syncthreads();
  const int d = threadIdx.x;
  float M = -INFINITY, L = 0.f, x = 0.f;
  for (int w = 0; w < 4; ++w) M = fmaxf(M, wm[w]);
  for (int w = 0; w < 4; ++w) {
    const float f = wm[w] == -INFINITY ? 0.f : ex2(wm[w] - M);
    L += f * wl[w];
    x += f * wo[w][d];
  }
  const float y = L != 0.f ? x / L : 0.f;  // (a NaN stays one)
  const int64_t off = b * A.o.sb + h * A.o.sh + t * A.o.sn + d;
  if (A.o_bf16)
    static_cast<__nv_bfloat16*>(A.o.data)[off] = __float2bfloat16_rn(y);
  else
    static_cast<float*>(A.o.data)[off] = y;
}

}  // namespace

size_t tree_attn_workspace_bytes(int64_t B, int64_t Hq, int64_t T, int64_t Hk, int64_t N) {
  (void)B; (void)Hq; (void)T; (void)Hk; (void)N;
  return 0;
}

cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t stream) {
  if ((int64_t)a.B * a.Hq * a.T == 0) return cudaSuccess;
  tree_attn_kernel<<<dim3((unsigned)a.T, (unsigned)(a.B * a.Hq)), kTrThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace rtp
