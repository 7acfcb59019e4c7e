// rope.cu - per-head RMS norm of queries and keys with the position rotation, and
// its backward pass (formulas and thread layout in rope.cuh).
//
// Forward, per row:  y_c = r (x_c A_c + x_c' B_c).
// Backward, from dy: the rotation's transpose first, g = R^T dy, then with
// xh = x r:  dx = r (g w - xh mean_c(g w xh)),  dw_c = sum over rows of g_c xh_c;
// without a norm (no weight) dx = g.  r is recomputed from x, which is read
// anyway, so the forward saves nothing.
//
// Bound: HBM.  Forward reads x and writes y once; backward reads x and dy and
// writes dx.  A group of d/8 lanes takes one token's chunk of heads, so the
// rotation's coefficients are built once per chunk; to keep enough bytes in flight
// the forward loads kAhead rows before it uses one (32768 tokens of 65 heads of 128,
// bf16, 1.09 GB: 170-175 us, 6.2-6.4 TB/s), the backward has rows on their way in shared memory
// (half the tokens, 0.82 GB: 127 us, 6.4 TB/s, then the sum of dw).
#include <cmath>

#include "checks.cuh"
#include "rope.cuh"
#include "sm100.cuh"

namespace csa {

bool rope_params(const double* inv_freq, int rot, RopeParams& p) {
  constexpr long double kTurns = 0.15915494309189533576888376337251436L;  // 1 / 2 pi
  constexpr long double k64 = 18446744073709551616.0L;                    // 2^64
  for (int i = 0; i < rot / 2; ++i) {
    if (!std::isfinite(inv_freq[i])) return false;
    long double t = (long double)inv_freq[i] * kTurns;
    if (!(t < 0.5L && t > -0.5L)) t -= std::floor(t + 0.5L);  // whole turns a position change nothing
    // now in [-1/2, 1/2): a signed 64-bit fraction, whose wrapped value is the phase
    const long double f = t * k64;
    p.turn[i] = f >= 9223372036854775808.0L ? 1ull << 63 : (uint64_t)std::llrint(f);
  }
  return true;
}

int rope_head_chunk(int64_t T, int heads, int d, int most) {
  const int64_t groups = (int64_t)sm_count() * (384 / (d / 8));
  int c = most;
  while (c > 2 && T * ceil_div(heads, c) < groups) c /= 2;
  return c < heads ? c : heads;
}

namespace {

constexpr int kThreads = 256;      // forward
constexpr int kAhead = 4;          // rows of a group loaded before the first is used
// Forward blocks per SM, by the input's element size.  600 MB of 65 heads of 128: fp32 three 99 and
// 105 us (halves, pairs; two, as it comes without a bound, 117 and 121); bf16 four.
constexpr int fwd_blocks_per_sm(int bytes_x) { return bytes_x == 4 ? 3 : 4; }
// Backward: blocks per SM and rows of a group on their way, by element sizes.  600 MB of 65
// heads of 128 with the sum of dw (the bytes alone take 92 us): bf16 five and three 101 us (two
// 106, four 102; six and three 117); fp32 four and four 96 (three 105, five blocks 124; 121 in
// pairs); fp32 gradients of bf16 four and four 93 (five blocks 106); bf16 gradients of fp32 five
// and five 106 (four ahead 115, four blocks 114).
constexpr int kBwdThreads = 128;
constexpr int bwd_blocks_per_sm(int bytes_y) { return bytes_y == 4 ? 4 : 5; }
constexpr int bwd_ahead(int bytes_x, int bytes_y) { return bytes_y == 4 ? 4 : bytes_x == 4 ? 5 : 3; }
constexpr bool bwd_wide(int bytes_x, int bytes_y) { return bytes_x + bytes_y > 4; }
// Most heads of one token that share a set of coefficients: fewer sets with 16, shorter pieces
// of memory with 8.  Forward: bf16 outputs 173 us with 16, 192 with 8 (1.09 GB), fp32 outputs 99
// and 97 (of bf16, 600 MB), 118 and 107 (of fp32, pairs); backward, 600 MB: bf16 101 and 106
// (all channels in halves 109 and 120), fp32 126 and 121 (pairs), bf16 gradients of fp32 113 and 111.
constexpr int head_chunk_most(bool wide) { return wide ? 8 : 16; }
// What a unit costs beside its rows (its token's coefficients, the first loads), in rows.
constexpr int kUnitRows = 2;

// Queries or keys of one call.
struct RopeSide {
  const void *x, *dy;   // x [T, heads, d], token rows x_stride elements apart; dy dense
  void *y, *dx;         // y dense; dx token rows dx_stride apart
  const float* w;       // [d], or null: no norm
  int64_t x_stride, dx_stride;
  int heads, chunk, chunks;  // heads per unit, units per token
  int64_t blocks;       // thread blocks of this side
};

struct RopeArgs {
  RopeParams p;
  RopeSide side[2];  // queries, keys
  int64_t T;
  float* dw_part;  // backward: [blocks of both sides][d] partial weight gradients
};

// A lane's piece of a row on its way into shared memory.  L1: through the first-level cache
// (two pieces of 16 bytes share each 32-byte sector of an fp32 row: 97 us against 158).
template <bool L1>
__device__ __forceinline__ void copy16(uint4* to, const uint4* from) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  if (L1) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
}
// The lane's piece of a row in shared memory, as load8 gives it.
__device__ __forceinline__ void take(Raw8b& r, const uint4* p) { r.v = p[0]; }
__device__ __forceinline__ void take(Raw8f& r, const uint4* p) {
  r.a = *reinterpret_cast<const float4*>(p), r.b = *reinterpret_cast<const float4*>(p + kBwdThreads);
}

template <int D, typename TX, typename TY, int STYLE>
__global__ void __launch_bounds__(kThreads, fwd_blocks_per_sm(sizeof(TX))) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPR = D / 8, GROUPS = kThreads / LPR;
  __shared__ uint64_t s_turn[kRopeMaxPairs];
  stage_turns(a.p, s_turn);
  const bool keys = (int64_t)blockIdx.x >= a.side[0].blocks;
  const RopeSide& sd = a.side[keys];
  const int64_t unit = ((int64_t)blockIdx.x - (keys ? a.side[0].blocks : 0)) * GROUPS + threadIdx.x / LPR;
  const int64_t t = unit / sd.chunks;
  if (t >= a.T) return;
  const int h0 = (int)(unit % sd.chunks) * sd.chunk;
  const int n = sd.heads - h0 < sd.chunk ? sd.heads - h0 : sd.chunk;
  const uint32_t mask = group_mask<D>();
  const RopeLane rl = rope_lane<D, STYLE>(a.p);
  using Raw = typename RawOf<TX>::type;
  const TX* x = static_cast<const TX*>(sd.x) + t * sd.x_stride + (int64_t)h0 * D + 8 * rl.l;
  TY* y = static_cast<TY*>(sd.y) + (t * sd.heads + h0) * D + 8 * rl.l;
  Raw raw[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (u < n) load8(x + u * D, raw[u]);
  float A[8], B[8];
  {
    float w[8], wp[8], c[8], s[8];
    load_weights(sd.w, rl.l, w);
    load_weights(sd.w, rl.partner % LPR, wp);
    rope_angles<STYLE>(rl, s_turn, a.p.pos ? a.p.pos[t] : a.p.t0 + t, mask, c, s);
    rope_coef<STYLE>(rl, c, s, w, wp, A, B);
  }
  const bool norm = sd.w != nullptr;
  for (int h = 0; h < n; h += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (h + u >= n) break;
      const Raw cur = raw[u];
      float f[8], o[8];
      unpack8(cur, f);
      const float r = norm ? row_rms<D>(f, a.p.eps, mask) : 1.f;
      rope_row<STYLE>(cur, f, r, A, B, rl, mask, o);
      if (h + u + kAhead < n) load8(x + (int64_t)(h + u + kAhead) * D, raw[u]);
      store8(y + (int64_t)(h + u) * D, o);
    }
  }
}

// Backward.  A block's groups take its side's units in turn (block i of the side
// the units i * GROUPS .., i * GROUPS + blocks * GROUPS .., ...), keep their share
// of dw in registers, and the block adds its groups' shares in order: one partial
// row per block, summed in order by norm_rope_dw_kernel (no atomics).  Rows wait in
// shared memory, not in registers: the bytes in flight are what bounds it (rows in
// registers: 117 us where this takes 101, 16384 tokens of 65 heads 149 and 141).
template <int D, typename TX, typename TY, int STYLE>
__global__ void __launch_bounds__(kBwdThreads, bwd_blocks_per_sm(sizeof(TY)))
    norm_rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPR = D / 8, GROUPS = kBwdThreads / LPR;
  constexpr int kAheadRows = bwd_ahead(sizeof(TX), sizeof(TY));
  constexpr int PX = sizeof(TX) / 2, PY = sizeof(TY) / 2;   // 16-byte pieces of a lane's eight channels
  __shared__ uint64_t s_turn[kRopeMaxPairs];
  __shared__ float s_dw[GROUPS * D];
  __shared__ uint4 s_row[kAheadRows + 1][PX + PY][kBwdThreads];
  griddep_launch_dependents();  // the sum of dw is set up while the last blocks run
  stage_turns(a.p, s_turn);
  const bool keys = (int64_t)blockIdx.x >= a.side[0].blocks;
  const RopeSide& sd = a.side[keys];
  const int64_t block = (int64_t)blockIdx.x - (keys ? a.side[0].blocks : 0);
  const uint32_t mask = group_mask<D>();
  const RopeLane rl = rope_lane<D, STYLE>(a.p);
  float w[8], dw[8], one[8];
  load_weights(sd.w, rl.l, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = 0.f, one[j] = 1.f;
  const bool norm = sd.w != nullptr;
  const int64_t step = sd.blocks * GROUPS, first = block * GROUPS + threadIdx.x / LPR;
  const int64_t step_t = step / sd.chunks;
  const int step_c = (int)(step - step_t * sd.chunks);
  // a place in the group's units: token, chunk of heads
  struct Place {
    int64_t t;
    int c;
  };
  auto next = [&](Place& p) {
    p.t += step_t, p.c += step_c;
    if (p.c >= sd.chunks) p.c -= sd.chunks, ++p.t;
  };
  auto size = [&](const Place& p) {
    const int left = sd.heads - p.c * sd.chunk;
    return left < sd.chunk ? left : sd.chunk;
  };
  Place at;
  at.t = first / sd.chunks, at.c = (int)(first - at.t * sd.chunks);
  // The copies run kAheadRows rows ahead, across units: every lane copies, and later reads, its
  // own pieces, so nobody waits for another.
  Place ahead = at;
  int ah = 0, an = 0;
  const TX* ax = nullptr;
  const TY* ay = nullptr;
  auto open = [&]() {
    if (ahead.t < a.T) {
      const int h0 = ahead.c * sd.chunk;
      ax = static_cast<const TX*>(sd.x) + ahead.t * sd.x_stride + (int64_t)h0 * D + 8 * rl.l;
      ay = static_cast<const TY*>(sd.dy) + (ahead.t * sd.heads + h0) * D + 8 * rl.l;
      an = size(ahead);
    }
    ah = 0;
  };
  open();
  auto fetch = [&](int slot) {
    if (ahead.t < a.T) {
#pragma unroll
      for (int i = 0; i < PX; ++i) copy16<(PX > 1)>(&s_row[slot][i][threadIdx.x], reinterpret_cast<const uint4*>(ax) + i);
#pragma unroll
      for (int i = 0; i < PY; ++i) copy16<(PY > 1)>(&s_row[slot][PX + i][threadIdx.x], reinterpret_cast<const uint4*>(ay) + i);
      ax += D, ay += D;
      if (++ah == an) next(ahead), open();
    }
    sm100::cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kAheadRows; ++i) fetch(i);
  int slot = 0;
  auto position = [&](const Place& p) { return a.p.pos ? (p.t < a.T ? a.p.pos[p.t] : 0) : a.p.t0 + p.t; };
  int64_t pos = position(at);
#pragma unroll 1
  while (at.t < a.T) {
    const int n = size(at), h0 = at.c * sd.chunk;
    TX* dx = static_cast<TX*>(sd.dx) + at.t * sd.dx_stride + (int64_t)h0 * D + 8 * rl.l;
    float A[8], B[8];
    {
      float c[8], s[8];
      rope_angles<STYLE>(rl, s_turn, pos, mask, c, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = -s[j];  // the transpose turns back
      rope_coef<STYLE>(rl, c, s, one, one, A, B);
    }
    next(at);
    pos = position(at);
#pragma unroll 1
    for (int h = 0; h < n; ++h) {
      sm100::cp_async_wait<kAheadRows - 1>();
      typename RawOf<TX>::type cx;
      typename RawOf<TY>::type cy;
      take(cx, &s_row[slot][0][threadIdx.x]);
      take(cy, &s_row[slot][PX][threadIdx.x]);
      float f[8], e[8], g[8];
      unpack8(cx, f);
      unpack8(cy, e);
      fetch(slot == 0 ? kAheadRows : slot - 1);  // the place of the row before
      slot = slot == kAheadRows ? 0 : slot + 1;
      rope_row<STYLE>(cy, e, 1.f, A, B, rl, mask, g);
      if (norm) {
        float q = 0.f, v = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) q = fmaf(f[j], f[j], q), v = fmaf(g[j] * w[j], f[j], v);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) {
          q += __shfl_xor_sync(mask, q, o);
          v += __shfl_xor_sync(mask, v, o);
        }
        const float r = rsqrtf(q * (1.0f / D) + a.p.eps);
        const float k = v * (1.0f / D) * r * r;  // x k = xh mean(g w xh)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[j] = fmaf(g[j], f[j] * r, dw[j]);
          g[j] = r * fmaf(-f[j], k, g[j] * w[j]);
        }
      }
      store8(dx + (int64_t)h * D, g);
    }
  }
  if (!norm) return;
  const int grp = threadIdx.x / LPR;
#pragma unroll
  for (int j = 0; j < 8; ++j) s_dw[grp * D + 8 * rl.l + j] = dw[j];
  __syncthreads();
  if ((int)threadIdx.x < D) {
    float sum = 0.f;
    for (int i = 0; i < GROUPS; ++i) sum += s_dw[i * D + threadIdx.x];
    a.dw_part[(int64_t)blockIdx.x * D + threadIdx.x] = sum;
  }
}

// dw = sum of a side's partial rows (blockIdx.y 0 the queries', 1 the keys'), 32 channels a
// block: its warps take every 32nd row each, then their sums are added in order.  (Two blocks,
// eight rows at a time, took 3 us more of a call with 740 rows a side.)
constexpr int kDwWarps = 32;

template <int D>
__global__ void __launch_bounds__(32 * kDwWarps) norm_rope_dw_kernel(const float* part, int64_t qblocks,
                                                                     int64_t kblocks, float* dwq, float* dwk) {
  griddep_wait();
  float* dw = blockIdx.y ? dwk : dwq;
  if (dw == nullptr) return;
  const int64_t n = blockIdx.y ? kblocks : qblocks;
  const float* p = part + (blockIdx.y ? qblocks * D : 0);
  __shared__ float s[kDwWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float sum = 0.f;
#pragma unroll 12
  for (int64_t i = warp; i < n; i += kDwWarps) sum += p[i * D + c];
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 1; i < kDwWarps; ++i) sum += s[i][lane];
    dw[c] = sum;
  }
}

int64_t side_units(int64_t T, int heads, int d, bool wide) {
  return T * ceil_div(heads, rope_head_chunk(T, heads, d, head_chunk_most(wide)));
}

// Blocks of the queries and of the keys in the backward pass: all at once on the GPU, each
// with its share of the work; each leaves one partial row of dw.
void bwd_split(int64_t T, int H, int Hk, int d, int bytes_x, int bytes_y, int64_t* blocks) {
  const int heads[2] = {H, Hk};
  int64_t need[2] = {0, 0}, work[2] = {0, 0};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] <= 0) continue;
    const int64_t units = side_units(T, heads[i], d, bwd_wide(bytes_x, bytes_y));
    need[i] = ceil_div(units, kBwdThreads / (d / 8));
    work[i] = T * heads[i] + units * kUnitRows;
  }
  const int64_t most = (int64_t)bwd_blocks_per_sm(bytes_y) * sm_count();
  blocks[0] = need[0], blocks[1] = need[1];
  if (need[0] + need[1] <= most) return;
  int64_t k = (int64_t)((double)most * work[1] / (work[0] + work[1]) + 0.5);
  if (k < 1) k = 1;
  if (k > most - 1 && H > 0) k = most - 1;
  if (k > need[1]) k = need[1];
  blocks[0] = need[0] < most - k ? need[0] : most - k;
  blocks[1] = need[1] < most - blocks[0] ? need[1] : most - blocks[0];
}

void fill_side(RopeSide& s, int64_t T, int heads, int d, bool wide) {
  s.heads = heads;
  s.chunk = heads > 0 ? rope_head_chunk(T, heads, d, head_chunk_most(wide)) : 1;
  s.chunks = heads > 0 ? (int)ceil_div(heads, s.chunk) : 1;
}

template <int D, typename TX, typename TY, int STYLE>
cudaError_t launch_one(const RopeArgs& a, bool bwd, cudaStream_t stream) {
  const int64_t grid = a.side[0].blocks + a.side[1].blocks;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_kernel(bwd ? norm_rope_bwd_kernel<D, TX, TY, STYLE> : norm_rope_kernel<D, TX, TY, STYLE>,
                       dim3((unsigned)grid), dim3(bwd ? kBwdThreads : kThreads), 0, stream, false, a);
}

template <int D>
cudaError_t launch_types(const RopeArgs& a, int xt, int yt, bool bwd, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  const bool halves = a.p.style == CSA_ROPE_HALVES;
#define CSA_GO(TX, TY)                                                                   \
  (halves ? launch_one<D, TX, TY, CSA_ROPE_HALVES>(a, bwd, stream)                       \
          : launch_one<D, TX, TY, CSA_ROPE_PAIRS>(a, bwd, stream))
  if (xt == CSA_BF16) return yt == CSA_BF16 ? CSA_GO(bf, bf) : CSA_GO(bf, float);
  return yt == CSA_BF16 ? CSA_GO(float, bf) : CSA_GO(float, float);
#undef CSA_GO
}

// Arguments that forward and backward share.
int check_rope(int64_t T, int H, int Hk, int d, int x_dtype, int y_dtype, const void* q, int64_t q_stride,
               const void* k, int64_t k_stride, const float* wq, const float* wk, float eps,
               const double* inv_freq, int rot_start, int rot_dim, int rot_style, bool wide, RopeArgs& a) {
  if (T < 0 || H < 0 || Hk < 0 || H > 4096 || Hk > 4096 || !valid_odtype(x_dtype) || !valid_odtype(y_dtype))
    return CSA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return CSA_ERR_UNSUPPORTED_SHAPE;
  const int unit = x_dtype == CSA_BF16 ? 8 : 4;  // elements of 16 bytes
  if (H > 0 && (q_stride < (int64_t)H * d || q_stride % unit != 0)) return CSA_ERR_INVALID_ARG;
  if (Hk > 0 && (k_stride < (int64_t)Hk * d || k_stride % unit != 0)) return CSA_ERR_INVALID_ARG;
  int rc = check_rotation(d, inv_freq, rot_start, rot_dim, rot_style, eps);
  if (rc) return rc;
  if (T > 0 && H > 0 && (rc = check_ptrs(q))) return rc;
  if (T > 0 && Hk > 0 && (rc = check_ptrs(k))) return rc;
  if ((rc = check_opt(wq)) || (rc = check_opt(wk))) return rc;
  if (!rope_params(inv_freq, rot_dim, a.p)) return CSA_ERR_INVALID_ARG;
  a.p.start = rot_start;
  a.p.rot = rot_dim;
  a.p.style = rot_style;
  a.p.eps = eps;
  a.T = T;
  fill_side(a.side[0], T, H, d, wide);
  fill_side(a.side[1], T, Hk, d, wide);
  a.side[0].x = q, a.side[0].x_stride = q_stride, a.side[0].w = wq;
  a.side[1].x = k, a.side[1].x_stride = k_stride, a.side[1].w = wk;
  return CSA_OK;
}

}  // namespace

int check_rotation(int d, const double* inv_freq, int rot_start, int rot_dim, int rot_style, float eps) {
  if ((rot_style != CSA_ROPE_HALVES && rot_style != CSA_ROPE_PAIRS) || !(std::isfinite(eps) && eps >= 0.f))
    return CSA_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim % 16 != 0 || rot_start < 0 || rot_start % 8 != 0 || rot_start + rot_dim > d)
    return CSA_ERR_UNSUPPORTED_SHAPE;
  return rot_dim > 0 && inv_freq == nullptr ? CSA_ERR_INVALID_ARG : CSA_OK;
}

}  // namespace csa

using namespace csa;

extern "C" {

int csa_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* wq,
                     const float* wk, float eps, const int64_t* pos, int64_t t0, const double* inv_freq,
                     int rot_start, int rot_dim, int rot_style, int64_t T, int H, int Hk, int d, int x_dtype,
                     void* yq, void* yk, int y_dtype, csa_stream_t stream) {
  RopeArgs a{};
  const bool wide = y_dtype == CSA_F32;
  int rc = check_rope(T, H, Hk, d, x_dtype, y_dtype, q, q_stride, k, k_stride, wq, wk, eps, inv_freq, rot_start,
                      rot_dim, rot_style, wide, a);
  if (rc) return rc;
  if ((rc = check_opt(pos))) return rc;
  if (T == 0 || (H == 0 && Hk == 0)) return CSA_OK;
  if (H > 0 && (rc = check_ptrs(yq))) return rc;
  if (Hk > 0 && (rc = check_ptrs(yk))) return rc;
  // in place is fine (a row's lanes read it before they write it); any other overlap is not
  const int heads[2] = {H, Hk};
  void* out[2] = {yq, yk};
  for (int i = 0; i < 2; ++i) {
    const size_t on = span(T, (int64_t)heads[i] * d, heads[i], d, y_dtype);
    for (int j = 0; j < 2; ++j) {
      const RopeSide& s = a.side[j];
      const bool in_place = i == j && out[i] == s.x && x_dtype == y_dtype && s.x_stride == (int64_t)s.heads * d;
      if (!in_place && overlap(out[i], on, s.x, span(T, s.x_stride, s.heads, d, x_dtype))) return CSA_ERR_INVALID_ARG;
    }
    a.side[i].y = out[i];
    a.side[i].blocks = heads[i] > 0 ? ceil_div(side_units(T, heads[i], d, wide), kThreads / (d / 8)) : 0;
  }
  const Bytes outs[2] = {{yq, span(T, (int64_t)H * d, H, d, y_dtype)}, {yk, span(T, (int64_t)Hk * d, Hk, d, y_dtype)}};
  const size_t wn = (size_t)d * 4, pn = (size_t)T * 8;
  if (overlap_any(outs[0], {outs[1], {wq, wn}, {wk, wn}, {pos, pn}}) ||
      overlap_any(outs[1], {{wq, wn}, {wk, wn}, {pos, pn}}))
    return CSA_ERR_INVALID_ARG;
  a.p.pos = pos;
  a.p.t0 = t0;
  cudaError_t e = d == 128 ? launch_types<128>(a, x_dtype, y_dtype, false, (cudaStream_t)stream)
                           : launch_types<64>(a, x_dtype, y_dtype, false, (cudaStream_t)stream);
  return e == cudaSuccess ? CSA_OK : cuda_fail(e);
}

size_t csa_qk_norm_rope_backward_workspace_bytes(int64_t T, int H, int Hk, int d) {
  if (T <= 0 || (d != 64 && d != 128)) return kWorkspaceHeader;  // no rows, or a head dim that is refused
  int64_t most = 0, blocks[2];
  for (int types = 0; types < 4; ++types) {  // whatever they are
    bwd_split(T, H, Hk, d, types & 1 ? 4 : 2, types & 2 ? 4 : 2, blocks);
    if (blocks[0] + blocks[1] > most) most = blocks[0] + blocks[1];
  }
  return kWorkspaceHeader + align256((size_t)most * d * 4);
}

int csa_qk_norm_rope_backward(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* wq,
                              const float* wk, float eps, const int64_t* pos, int64_t t0, const double* inv_freq,
                              int rot_start, int rot_dim, int rot_style, const void* dyq, const void* dyk, int64_t T,
                              int H, int Hk, int d, int x_dtype, int y_dtype, void* dq, int64_t dq_stride, void* dk,
                              int64_t dk_stride, float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                              csa_stream_t stream) {
  RopeArgs a{};
  const int bytes_x = x_dtype == CSA_BF16 ? 2 : 4, bytes_y = y_dtype == CSA_BF16 ? 2 : 4;
  int rc = check_rope(T, H, Hk, d, x_dtype, y_dtype, q, q_stride, k, k_stride, wq, wk, eps, inv_freq, rot_start,
                      rot_dim, rot_style, bwd_wide(bytes_x, bytes_y), a);
  if (rc) return rc;
  if ((rc = check_opt(pos))) return rc;
  if ((H > 0 && wq != nullptr) != (dwq != nullptr) || (Hk > 0 && wk != nullptr) != (dwk != nullptr))
    return CSA_ERR_INVALID_ARG;
  if ((rc = check_opt(dwq)) || (rc = check_opt(dwk))) return rc;
  const int heads[2] = {H, Hk};
  const void* dy[2] = {dyq, dyk};
  void* dx[2] = {dq, dk};
  const int64_t dxs[2] = {dq_stride, dk_stride};
  const int unit = x_dtype == CSA_BF16 ? 8 : 4;
  for (int i = 0; i < 2; ++i)
    if (heads[i] > 0 && (dxs[i] < (int64_t)heads[i] * d || dxs[i] % unit != 0)) return CSA_ERR_INVALID_ARG;
  rc = check_ws(workspace, workspace_bytes, csa_qk_norm_rope_backward_workspace_bytes(T, H, Hk, d));
  if (rc) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {  // no rows: the weight gradients are empty sums
    cudaError_t e = cudaSuccess;
    for (float* dw : {dwq, dwk})
      if (dw != nullptr && e == cudaSuccess) e = cudaMemsetAsync(dw, 0, (size_t)d * 4, s);
    return e == cudaSuccess ? CSA_OK : cuda_fail(e);
  }
  if (H == 0 && Hk == 0) return CSA_OK;
  // (dq and dk may lie between each other's rows, in one packed gradient)
  const size_t wn = (size_t)d * 4;
  if (overlap_any({dwq, wn}, {{dwk, wn}})) return CSA_ERR_INVALID_ARG;
  int64_t blocks[2];
  bwd_split(T, H, Hk, d, bytes_x, bytes_y, blocks);
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    if ((rc = check_ptrs(dy[i], dx[i]))) return rc;
    const size_t dn = span(T, dxs[i], heads[i], d, x_dtype);
    if (overlap_any({dx[i], dn}, {{wq, wn}, {wk, wn}, {pos, (size_t)T * 8}, {dwq, wn}, {dwk, wn}}))
      return CSA_ERR_INVALID_ARG;
    for (int j = 0; j < 2; ++j) {
      if (overlap(dx[i], dn, a.side[j].x, span(T, a.side[j].x_stride, heads[j], d, x_dtype)) ||
          overlap(dx[i], dn, dy[j], span(T, (int64_t)heads[j] * d, heads[j], d, y_dtype)))
        return CSA_ERR_INVALID_ARG;
    }
    a.side[i].dy = dy[i];
    a.side[i].dx = dx[i];
    a.side[i].dx_stride = dxs[i];
    a.side[i].blocks = blocks[i];
  }
  a.p.pos = pos;
  a.p.t0 = t0;
  a.dw_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWorkspaceHeader);
  cudaError_t e = d == 128 ? launch_types<128>(a, x_dtype, y_dtype, true, s)
                           : launch_types<64>(a, x_dtype, y_dtype, true, s);
  if (e == cudaSuccess && (dwq || dwk))
    e = launch_kernel(d == 128 ? norm_rope_dw_kernel<128> : norm_rope_dw_kernel<64>, dim3(d / 32, 2),
                      dim3(32 * kDwWarps), 0, s, true, (const float*)a.dw_part, a.side[0].blocks, a.side[1].blocks, dwq, dwk);
  return e == cudaSuccess ? CSA_OK : cuda_fail(e);
}

}  // extern "C"
