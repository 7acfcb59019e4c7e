// tree.cu - attention of drafted tokens over a paged raw K/V cache.
//
// Node i of sequence b (row r of the call) sees the committed rows s < L_b of its
// sequence (with a window: s > pos_r - W) and those drafted rows L_b + j whose
// bit j its mask holds; one softmax over both:
//   O = sum_s p_s v_s,  p_s = exp(scale q.k_s - lse),  lse = log sum_s exp(scale q.k_s).
// One token per sequence with mask 1 is ordinary decode over the cache.
#include <cmath>

#include "checks.cuh"

namespace csa {

namespace {

struct TreeArgs {
  const __nv_bfloat16 *q, *Kp, *Vp;
  const int32_t *table, *lens, *q_start;
  const uint64_t* mask;
  const int64_t* pos;
  int64_t R, n_pages;
  int B, H, Hk, max_pages, page_shift, W;
  float scale_log2;
  void* O;
  int o_f32;
  float* lse;
  int* status;
};

// One warp per (row, head): lanes own d/32 channels, the running maximum and sum
// of the softmax in fp32.
template <int D>
__global__ void __launch_bounds__(128) tree_attn_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t r = w / a.H;
  const int h = (int)(w % a.H);
  if (r >= a.R) return;
  int b = -1;
  for (int i = 0; i < a.B; ++i) {
    const int64_t r0 = a.q_start[i], r1 = a.q_start[i + 1];
    if (r0 < 0 || r1 < r0 || r1 > a.R) report(a.status, CSA_ERR_INDEX);
    else if (r0 <= r && r < r1) b = i;
  }
  if (b < 0) return;  // behind the last sequence
  const int64_t L = a.lens[b];
  const int n = a.q_start[b + 1] - a.q_start[b];
  if (L < 0 || n > 64 || L + n > ((int64_t)a.max_pages << a.page_shift)) {
    report(a.status, CSA_ERR_INDEX);
    return;
  }
  const uint64_t mask = a.mask[r];
  const int hk = h / (a.H / a.Hk);
  float q[C], o[C];
  for (int c = 0; c < C; ++c) q[c] = __bfloat162float(a.q[(r * a.H + h) * D + lane * C + c]), o[c] = 0.f;
  int64_t lo = 0;
  if (a.W >= 0) {
    lo = a.pos[r] - a.W + 1;
    lo = lo < 0 ? 0 : lo > L ? L : lo;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t s = lo; s < L + n; ++s) {
    if (s >= L && !(mask >> (s - L) & 1)) continue;
    const int64_t page = a.table[(int64_t)b * a.max_pages + (s >> a.page_shift)];
    if (page < 0 || page >= a.n_pages) {
      report(a.status, CSA_ERR_INDEX);
      continue;
    }
    const int64_t at = (((page * a.Hk + hk) << a.page_shift) + (s & ((1 << a.page_shift) - 1))) * D + lane * C;
    float z = 0.f;
    for (int c = 0; c < C; ++c) z = fmaf(q[c], __bfloat162float(a.Kp[at + c]), z);
    for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    z *= a.scale_log2;
    const float mn = fmaxf(m, z), f = exp2f(m - mn), p = exp2f(z - mn);
    l = l * f + p;
    for (int c = 0; c < C; ++c) o[c] = o[c] * f + p * __bfloat162float(a.Vp[at + c]);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int c = 0; c < C; ++c) {
    const int64_t at = (r * a.H + h) * D + lane * C + c;
    if (a.o_f32) static_cast<float*>(a.O)[at] = o[c] * inv;
    else static_cast<__nv_bfloat16*>(a.O)[at] = __float2bfloat16(o[c] * inv);
  }
  if (a.lse && lane == 0) a.lse[r * a.H + h] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" {

size_t csa_tree_attn_workspace_bytes(int, int64_t, int, int, int, int, int) { return kWorkspaceHeader; }

int csa_tree_attn(const void* q, const void* Kpages, const void* Vpages, const int32_t* block_table,
                  const int32_t* seq_lens, const int32_t* q_start, const uint64_t* mask, const int64_t* pos, int64_t R,
                  int B, int H, int Hk, int d, int page, int64_t n_pages, int max_pages, int W, float scale, void* O,
                  int o_dtype, float* lse, void* workspace, size_t workspace_bytes, csa_stream_t stream) {
  if (R < 0 || R > 0x7FFFFFFF || B < 0 || H < 1 || Hk < 1 || n_pages < 0 || max_pages < 0 || W < -1 ||
      !(std::isfinite(scale) && scale > 0.f) || !valid_odtype(o_dtype))
    return CSA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || !valid_page(page) || H > 1024 || H % Hk != 0) return CSA_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)max_pages * page > 0x7FFFFFFF) return CSA_ERR_UNSUPPORTED_SHAPE;
  int rc = check_ws(workspace, workspace_bytes, csa_tree_attn_workspace_bytes(B, R, H, Hk, d, page, max_pages));
  if (rc) return rc;
  if (R == 0 || B == 0) return CSA_OK;
  if ((rc = check_ptrs(q, seq_lens, q_start, mask, O))) return rc;
  if (W >= 0 && (rc = check_ptrs(pos))) return rc;
  if (max_pages > 0 && (rc = check_ptrs(block_table))) return rc;
  if (n_pages > 0 && (rc = check_ptrs(Kpages, Vpages))) return rc;
  if ((rc = check_opt(lse))) return rc;
  TreeArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.Kp = static_cast<const __nv_bfloat16*>(Kpages);
  a.Vp = static_cast<const __nv_bfloat16*>(Vpages);
  a.table = block_table;
  a.lens = seq_lens;
  a.q_start = q_start;
  a.mask = mask;
  a.pos = pos;
  a.R = R;
  a.n_pages = n_pages;
  a.B = B;
  a.H = H;
  a.Hk = Hk;
  a.max_pages = max_pages;
  while ((1 << a.page_shift) < page) ++a.page_shift;
  a.W = W;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.O = O;
  a.o_f32 = o_dtype == CSA_F32;
  a.lse = lse;
  a.status = status_word(workspace);
  const int64_t grid = ceil_div(R * H, 4);
  if (grid > 0x7FFFFFFF) return CSA_ERR_UNSUPPORTED_SHAPE;
  cudaError_t e = launch_kernel(d == 128 ? tree_attn_kernel<128> : tree_attn_kernel<64>, dim3((unsigned)grid), dim3(128),
                                0, (cudaStream_t)stream, false, a);
  return e == cudaSuccess ? CSA_OK : cuda_fail(e);
}

}  // extern "C"
