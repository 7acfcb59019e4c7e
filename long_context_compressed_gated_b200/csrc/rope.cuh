// rope.cuh - per-head RMS norm and position rotation of query / key rows, shared
// by the prefill kernels (rope.cu) and the paged append (paged.cu).
//
// One row = the d channels of one (token, head).  The norm multiplies by
//   r = 1 / sqrt(mean_c x_c^2 + eps)   and by a weight w_c;
// the rotation turns channel pairs (a, b) of [start, start + rot) by the angle
// theta_p = pos * f_p of their pair p:
//   y_a = x_a cos theta - x_b sin theta,   y_b = x_b cos theta + x_a sin theta,
// with (a, b) = start + (p, p + rot/2) for CSA_ROPE_HALVES and
// start + (2p, 2p + 1) for CSA_ROPE_PAIRS.  Norm weight and rotation act on a
// row as one pair of coefficients per channel,
//   y_c = r (x_c A_c + x_c' B_c),  A_c = w_c cos theta,  B_c = -+ w_c' sin theta
// (c' the partner channel), which depend on the token and not on the head: they
// are built once per token and used for all its heads.
//
// Angles of far positions: a 32-bit product pos * f is off by 0.06 rad at
// position 2^20.  Here f is held as a 64-bit binary fraction of a turn,
// F = round(f / 2pi * 2^64), and pos * F wraps modulo 2^64 exactly as the angle
// wraps modulo a turn, so the product is exact for every 64-bit position
// (negative ones too) and only the rounding of F remains: |pos| * 2^-65 turns.
//
// Thread layout: a group of d/8 lanes owns a row, lane l channels 8l .. 8l+7 (16
// bytes of bf16), so a row is one coalesced access and its norm log2(d/8)
// shuffles.  Every lane evaluates four pairs' sine and cosine: its own four
// pairs (PAIRS), or one half of the eight that it shares with its partner lane,
// which evaluates the other half (HALVES).
#pragma once
#include "common.cuh"

namespace csa {

constexpr int kRopeMaxPairs = 64;  // rot <= d <= 128

// What the host hands to a kernel about the norm and the rotation.
struct RopeParams {
  uint64_t turn[kRopeMaxPairs];  // F_p, 2^-64 turns per position
  const int64_t* pos;            // [T] device, or null: position t0 + t
  int64_t t0;
  int start, rot, style;
  float eps;
};

// Host: F_p from radians per position; false when one is not finite.
bool rope_params(const double* inv_freq, int rot, RopeParams& p);

// Heads of one token that a lane group takes: `most`, halved while the groups would leave
// an SM under 384 threads (a decode step of 16 tokens x 64 heads: 2 heads, 3.6 us; with 16
// heads 6.8).  The coefficients are built once per group, so long calls keep `most` (32768
// tokens of 65 heads, bf16: 173 us with 16, 192 with 8).
int rope_head_chunk(int64_t T, int heads, int d, int most);

__device__ __forceinline__ float4 ld_f4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// Eight consecutive channels as fp32.
struct Raw8b { uint4 v; };
struct Raw8f { float4 a, b; };
__device__ __forceinline__ void load8(const __nv_bfloat16* p, Raw8b& r) { r.v = *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void load8(const float* p, Raw8f& r) { r.a = ld_f4(p), r.b = ld_f4(p + 4); }
__device__ __forceinline__ void unpack8(const Raw8b& r, float* x) {
  x[0] = bf16_lo(r.v.x), x[1] = bf16_hi(r.v.x), x[2] = bf16_lo(r.v.y), x[3] = bf16_hi(r.v.y);
  x[4] = bf16_lo(r.v.z), x[5] = bf16_hi(r.v.z), x[6] = bf16_lo(r.v.w), x[7] = bf16_hi(r.v.w);
}
__device__ __forceinline__ void unpack8(const Raw8f& r, float* x) {
  x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w, x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
}
__device__ __forceinline__ Raw8b shfl8(uint32_t mask, const Raw8b& r, int src) {
  return Raw8b{make_uint4(__shfl_sync(mask, r.v.x, src), __shfl_sync(mask, r.v.y, src),
                          __shfl_sync(mask, r.v.z, src), __shfl_sync(mask, r.v.w, src))};
}
__device__ __forceinline__ Raw8f shfl8(uint32_t mask, const Raw8f& r, int src) {
  return Raw8f{make_float4(__shfl_sync(mask, r.a.x, src), __shfl_sync(mask, r.a.y, src),
                           __shfl_sync(mask, r.a.z, src), __shfl_sync(mask, r.a.w, src)),
               make_float4(__shfl_sync(mask, r.b.x, src), __shfl_sync(mask, r.b.y, src),
                           __shfl_sync(mask, r.b.z, src), __shfl_sync(mask, r.b.w, src))};
}
// The outputs are rounded once, here (round to nearest even for bf16).
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* y) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                            pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}
__device__ __forceinline__ void store8(float* p, const float* y) {
  *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(y[4], y[5], y[6], y[7]);
}
template <typename T> struct RawOf;
template <> struct RawOf<__nv_bfloat16> { using type = Raw8b; };
template <> struct RawOf<float> { using type = Raw8f; };

// cos and sin of a phase in 2^-64 turns: the nearest quarter turn is taken off
// exactly, the rest |angle| <= pi/4 goes through the Taylor series of sine and
// cosine (remainders (pi/4)^11/11! < 2e-9 and (pi/4)^12/12! < 2e-10).
__device__ __forceinline__ void phase_cos_sin(uint64_t phase, float& c, float& s) {
  const uint64_t quad = (phase + (1ull << 61)) >> 62;    // 0 .. 3 (the sum wraps like the angle)
  const int64_t rest = (int64_t)(phase - (quad << 62));  // in [-2^61, 2^61)
  // in units of 2^-34 turns, 2 pi / 2^34 radians each
  const float a = (float)(int32_t)(rest >> 30) * 3.65729520e-10f;
  const float a2 = a * a;
  float sn = fmaf(a2, 2.75573192e-6f, -1.98412698e-4f);
  sn = fmaf(a2, sn, 8.33333333e-3f);
  sn = fmaf(a2, sn, -1.66666667e-1f);
  sn = fmaf(a * a2, sn, a);
  float cs = fmaf(a2, -2.75573192e-7f, 2.48015873e-5f);
  cs = fmaf(a2, cs, -1.38888889e-3f);
  cs = fmaf(a2, cs, 4.16666667e-2f);
  cs = fmaf(a2, cs, -0.5f);
  cs = fmaf(a2, cs, 1.0f);
  const float cc = (quad & 1) ? sn : cs, ss = (quad & 1) ? cs : sn;
  c = (quad == 1 || quad == 2) ? -cc : cc;
  s = (quad & 2) ? -ss : ss;
}

// A lane's place in its row and in the rotation.
struct RopeLane {
  int l;         // lane in the group: channels 8l .. 8l+7
  int partner;   // warp lane that holds the partner channels (HALVES; itself when not turned)
  bool turned;   // channels inside [start, start + rot)
  bool high;     // HALVES: second half of the pairs
  int pair0;     // first of its pairs
};

template <int D, int STYLE>
__device__ __forceinline__ RopeLane rope_lane(const RopeParams& p) {
  constexpr int LPR = D / 8;
  RopeLane r;
  const int lane = threadIdx.x & 31;
  r.l = lane % LPR;
  const int rel = r.l - p.start / 8;
  r.turned = rel >= 0 && rel < p.rot / 8;
  r.partner = lane;
  r.high = false;
  r.pair0 = 0;
  if (r.turned) {
    if (STYLE == CSA_ROPE_HALVES) {
      const int hw = p.rot / 16;
      r.high = rel >= hw;
      r.pair0 = 8 * (r.high ? rel - hw : rel);
      r.partner = r.high ? lane - hw : lane + hw;
    } else {
      r.pair0 = 4 * rel;
    }
  }
  return r;
}

// cos / sin for a token at position `pos`: PAIRS c[0..3] / s[0..3] of the lane's
// four pairs; HALVES c[0..7] / s[0..7] of its eight channels' pairs.  Every lane
// of the group calls this (mask: the group's lanes).  A lane that is not turned
// gets cos 1, sin 0.  turn: the F_p in shared memory.
template <int STYLE>
__device__ __forceinline__ void rope_angles(const RopeLane& r, const uint64_t* turn, int64_t pos, uint32_t mask,
                                            float* c, float* s) {
  float c4[4], s4[4];
  const int p0 = r.pair0 + (STYLE == CSA_ROPE_HALVES && r.high ? 4 : 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    c4[j] = 1.f, s4[j] = 0.f;
    if (r.turned) phase_cos_sin((uint64_t)pos * turn[p0 + j], c4[j], s4[j]);
  }
  if (STYLE == CSA_ROPE_HALVES) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float co = __shfl_sync(mask, c4[j], r.partner), so = __shfl_sync(mask, s4[j], r.partner);
      c[j] = r.high ? co : c4[j];
      c[j + 4] = r.high ? c4[j] : co;
      s[j] = r.high ? so : s4[j];
      s[j + 4] = r.high ? s4[j] : so;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = c4[j], s[j] = s4[j];
  }
}

// The coefficients A, B of a lane's eight channels: y = r (x A + x' B).
// w: the lane's weights (8), wp: its partner channels' (HALVES).
template <int STYLE>
__device__ __forceinline__ void rope_coef(const RopeLane& r, const float* c, const float* s, const float* w,
                                          const float* wp, float* A, float* B) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (STYLE == CSA_ROPE_HALVES) {
      A[j] = w[j] * c[j];
      B[j] = r.high ? wp[j] * s[j] : -(wp[j] * s[j]);
    } else {
      A[j] = w[j] * c[j >> 1];
      B[j] = (j & 1) ? w[j ^ 1] * s[j >> 1] : -(w[j ^ 1] * s[j >> 1]);
    }
  }
}

// r = 1 / sqrt(mean x^2 + eps) of the group's row (fp32 sums).
template <int D>
__device__ __forceinline__ float row_rms(const float* x, float eps, uint32_t mask) {
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) a = fmaf(x[j], x[j], a), b = fmaf(x[j + 1], x[j + 1], b);
  a += b;
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) a += __shfl_xor_sync(mask, a, o);
  return rsqrtf(a * (1.0f / D) + eps);
}

// y = r (x A + x' B) for the lane's eight channels of one row.  Channels that are not turned
// have no partner (B is 0 there, but 0 times an infinite x' would be NaN).
template <int STYLE, typename Raw>
__device__ __forceinline__ void rope_row(const Raw& raw, const float* x, float r, const float* A, const float* B,
                                         const RopeLane& rl, uint32_t mask, float* y) {
  float xp[8];
  if (STYLE == CSA_ROPE_HALVES) unpack8(shfl8(mask, raw, rl.partner), xp);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float xa = x[j] * A[j], xb = STYLE == CSA_ROPE_HALVES ? xp[j] : x[j ^ 1];
    y[j] = r * (rl.turned ? fmaf(xb, B[j], xa) : xa);
  }
}

template <int D>
__device__ __forceinline__ uint32_t group_mask() {
  constexpr int LPR = D / 8;
  return (uint32_t)((1ull << LPR) - 1) << ((threadIdx.x & 31) / LPR * LPR);
}

__device__ __forceinline__ void load_weights(const float* w, int l, float* o) {
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = 1.f;
    return;
  }
  const float4 a = ld_f4(w + 8 * l), b = ld_f4(w + 8 * l + 4);
  o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
}

// The F_p of the kernel's argument block into shared memory (a divergent index
// into the argument block would be one access per lane).
__device__ __forceinline__ void stage_turns(const RopeParams& p, uint64_t* s_turn) {
  for (int i = threadIdx.x; i < p.rot / 2; i += blockDim.x) s_turn[i] = p.turn[i];
  __syncthreads();
}

}  // namespace csa
