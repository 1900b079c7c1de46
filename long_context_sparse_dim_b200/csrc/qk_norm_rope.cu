// Per-head norm of queries and keys with the position rotation, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w           (skipped for a tensor without w)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)   over 64 pairs (a, b),
//   pair i turned by the angle position * inv_freq[i].
//
// This makes the post-rotary queries and keys that every other call takes
// ("RTPurbo: Turning Dense LLMs into Sparse Attention Models ...", "Three Key
// Insights" 2 speaks of rotary coordinates; the pages leave the rotation to the
// model).
//
// Bound: HBM (each row is read once and written once, about 10 operations per
// element).  Eight lanes hold a row, 8 pairs each, so that every access is a
// 16-byte vector, the sum of squares takes three shuffles, and the rotation
// needs no exchange at all: a lane holds both members of its pairs.  A lane
// group stays on one token and walks over heads, so the cosines and sines of
// the token (8 pairs per lane) are computed once and kept in registers.
//
// The angle is formed in fp64 as a fraction of a turn (position * inv_freq /
// 2 pi, less its nearest integer): in fp32 the product alone is off by 0.03
// radians a million tokens into a context.  Norm and rotation stay in fp32, one
// rounding at the end.
#include "common.cuh"
#include "launch.h"

namespace rtp {

namespace {

constexpr int kNrThreads = 256;
constexpr int kNrLanes = 8;   // lanes per row
constexpr int kNrPairs = 8;   // pairs per lane
constexpr int kNrUnroll = 2;  // heads in flight per lane group

// A lane's 16 elements of a row as raw 16-byte vectors: a = first members of its pairs, b = second (half
// pairing: dims 8l .. and 64 + 8l ..), or all in one run (adjacent pairing: dims 16l ..).
template <typename T, bool kHalf>
struct LaneRow {
  static constexpr int kVec = sizeof(T) == 2 ? 1 : 2;  // 16-byte vectors per 8 elements
  uint4 v[2][kVec];
  RTP_DEVICE static int64_t offset(int part, int lane) { return kHalf ? part * 64 + 8 * lane : 16 * lane + 8 * part; }
  // (plain loads: the output may be the input)
  RTP_DEVICE void load(const T* row, int lane) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[p][i] = reinterpret_cast<const uint4*>(row + offset(p, lane))[i];
  }
  RTP_DEVICE void to_float(float (&a)[kNrPairs], float (&b)[kNrPairs]) const {
    float x[2][8];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if constexpr (sizeof(T) == 2) {
        const uint32_t w[4] = {v[p][0].x, v[p][0].y, v[p][0].z, v[p][0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[p][2 * i] = bf16_lo(w[i]);
          x[p][2 * i + 1] = bf16_hi(w[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          x[p][4 * i] = __uint_as_float(v[p][i].x);
          x[p][4 * i + 1] = __uint_as_float(v[p][i].y);
          x[p][4 * i + 2] = __uint_as_float(v[p][i].z);
          x[p][4 * i + 3] = __uint_as_float(v[p][i].w);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kNrPairs; ++i) {
      a[i] = kHalf ? x[0][i] : x[i >> 2][2 * (i & 3)];
      b[i] = kHalf ? x[1][i] : x[i >> 2][2 * (i & 3) + 1];
    }
  }
};

template <typename T, bool kHalf>
RTP_DEVICE void store_row(T* row, int lane, const float (&a)[kNrPairs], const float (&b)[kNrPairs]) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = kHalf ? (p ? b[2 * i] : a[2 * i]) : a[4 * p + i];
      x[2 * i + 1] = kHalf ? (p ? b[2 * i + 1] : a[2 * i + 1]) : b[4 * p + i];
    }
    T* dst = row + (kHalf ? p * 64 + 8 * lane : 16 * lane + 8 * p);
    if constexpr (sizeof(T) == 2) {
      uint4 w;
      w.x = pack_bf16x2(x[0], x[1]);
      w.y = pack_bf16x2(x[2], x[3]);
      w.z = pack_bf16x2(x[4], x[5]);
      w.w = pack_bf16x2(x[6], x[7]);
      *reinterpret_cast<uint4*>(dst) = w;
    } else {
      reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

template <bool kHalf>
RTP_DEVICE void load_weight(const void* w, int64_t row_off, bool bf16, int lane, float (&a)[kNrPairs],
                            float (&b)[kNrPairs]) {
  if (bf16) {
    LaneRow<__nv_bfloat16, kHalf> r;
    r.load(static_cast<const __nv_bfloat16*>(w) + row_off, lane);
    r.to_float(a, b);
  } else {
    LaneRow<float, kHalf> r;
    r.load(static_cast<const float*>(w) + row_off, lane);
    r.to_float(a, b);
  }
}

RTP_DEVICE float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < kNrLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// x <- x * rsqrt(mean(x^2) + eps) * w.  Rows whose sum of squares leaves the range of fp32 (elements past
// about 1e15, or all tiny with an eps as tiny) are summed in fp64.
RTP_DEVICE void norm_row(float (&a)[kNrPairs], float (&b)[kNrPairs], const float (&wa)[kNrPairs],
                         const float (&wb)[kNrPairs], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kNrPairs; ++i) ss = __fmaf_rn(a[i], a[i], __fmaf_rn(b[i], b[i], ss));
  ss = group_sum(ss);
  const bool wide = !(ss < 1e30f) || ss + 128.f * eps < 1e-30f;
  if (!__any_sync(0xffffffffu, wide)) {
    const float r = __frsqrt_rn(__fmaf_rn(ss, 1.f / kHeadDim, eps));
#pragma unroll
    for (int i = 0; i < kNrPairs; ++i) {
      a[i] = a[i] * r * wa[i];
      b[i] = b[i] * r * wb[i];
    }
    return;
  }
  double sd = 0.0;
#pragma unroll
  for (int i = 0; i < kNrPairs; ++i) sd += (double)a[i] * a[i] + (double)b[i] * b[i];
#pragma unroll
  for (int o = 1; o < kNrLanes; o <<= 1) sd += __shfl_xor_sync(0xffffffffu, sd, o);
  const double r = 1.0 / sqrt(sd / kHeadDim + (double)eps);
#pragma unroll
  for (int i = 0; i < kNrPairs; ++i) {
    a[i] = (float)(a[i] * r) * wa[i];
    b[i] = (float)(b[i] * r) * wb[i];
  }
}

// Thread block: kNrThreads / 8 tokens x A.heads_per_group heads (of the Hq query then Hk key heads).
template <typename Tin, typename Tout, bool kHalf>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_kernel(NormRopeArgs A) {
  const int lane = threadIdx.x & (kNrLanes - 1);
  const int64_t tok = (int64_t)blockIdx.x * (blockDim.x / kNrLanes) + threadIdx.x / kNrLanes;
  const bool live = tok < (int64_t)A.B * A.T;  // (the shuffles below take whole warps)
  const int b = live ? (int)(tok / A.T) : 0, t = live ? (int)(tok % A.T) : 0;

  float cs[kNrPairs], sn[kNrPairs];
  {
    const double p = live ? (double)((int64_t)A.pos[b] + (A.offs ? A.offs[(int64_t)b * A.T + t] : t)) : 0.0;
    const double* f = A.inv_freq + kNrPairs * lane;
#pragma unroll
    for (int i = 0; i < kNrPairs; ++i) {
      const double turns = p * __ldg(f + i) * 0.15915494309189533577;  // 1 / (2 pi)
      sincospif((float)(2.0 * (turns - rint(turns))), &sn[i], &cs[i]);
    }
  }
  const int H = A.Hq + A.Hk;
  const int h0 = blockIdx.y * A.heads_per_group, h1 = min(h0 + A.heads_per_group, H);
  float wa[kNrPairs], wb[kNrPairs];
  bool have_w = false;
  for (int h = h0; h < h1; h += kNrUnroll) {
    LaneRow<Tin, kHalf> x[kNrUnroll];
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      const int hh = h + u;
      if (hh >= h1 || !live) continue;
      const View4& src = hh < A.Hq ? A.q : A.k;
      x[u].load(static_cast<const Tin*>(src.data) + b * src.sb + (hh < A.Hq ? hh : hh - A.Hq) * src.sh + t * src.sn,
                lane);
    }
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      const int hh = h + u;
      if (hh >= h1) continue;  // uniform over the block
      const bool is_q = hh < A.Hq;
      const int hk = is_q ? hh : hh - A.Hq;
      const void* w = is_q ? A.qw : A.kw;
      float a[kNrPairs], c[kNrPairs];
      if (live) {
        x[u].to_float(a, c);
      } else {
#pragma unroll
        for (int i = 0; i < kNrPairs; ++i) a[i] = c[i] = 0.f;
      }
      if (w) {
        const int64_t ws = is_q ? A.qw_stride : A.kw_stride;  // 0: one weight row for all heads
        if (!have_w || ws || hh == A.Hq) {
          load_weight<kHalf>(w, ws * hk, is_q ? A.qw_bf16 : A.kw_bf16, lane, wa, wb);
          have_w = true;
        }
        norm_row(a, c, wa, wb, A.eps);
      }
      if (!live) continue;
      float ya[kNrPairs], yb[kNrPairs];
#pragma unroll
      for (int i = 0; i < kNrPairs; ++i) {
        ya[i] = __fmaf_rn(a[i], cs[i], -(c[i] * sn[i]));
        yb[i] = __fmaf_rn(c[i], cs[i], a[i] * sn[i]);
      }
      const MutView4& dst = is_q ? A.q_out : A.k_out;
      store_row<Tout, kHalf>(static_cast<Tout*>(dst.data) + b * dst.sb + hk * dst.sh + t * dst.sn, lane, ya, yb);
    }
  }
}

template <typename Tin, typename Tout>
cudaError_t launch(const NormRopeArgs& a, bool half, dim3 grid, int threads, cudaStream_t stream) {
  if (half)
    qk_norm_rope_kernel<Tin, Tout, true><<<grid, threads, 0, stream>>>(a);
  else
    qk_norm_rope_kernel<Tin, Tout, false><<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(NormRopeArgs a, bool in_bf16, bool out_bf16, bool half, cudaStream_t stream) {
  const int64_t toks = (int64_t)a.B * a.T;
  const int H = a.Hq + a.Hk;
  if (toks == 0 || H == 0) return cudaSuccess;
  const int threads = kNrThreads;
  const int64_t blocks = (toks * kNrLanes + threads - 1) / threads;
  a.heads_per_group = 8;
  const dim3 grid((unsigned)blocks, (unsigned)((H + a.heads_per_group - 1) / a.heads_per_group));
  if (in_bf16)
    return out_bf16 ? launch<__nv_bfloat16, __nv_bfloat16>(a, half, grid, threads, stream)
                    : launch<__nv_bfloat16, float>(a, half, grid, threads, stream);
  return out_bf16 ? launch<float, __nv_bfloat16>(a, half, grid, threads, stream)
                  : launch<float, float>(a, half, grid, threads, stream);
}

}  // namespace rtp
