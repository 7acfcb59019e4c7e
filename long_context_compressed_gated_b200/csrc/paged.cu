// paged.cu - new keys and values into a paged raw cache, the keys normed and
// rotated on the way (formulas and thread layout in rope.cuh).
//
// Cache: Kpages / Vpages [n_pages, Hk, page, d] bf16; row `slot` of sequence b
// is row slot % page of page block_table[b, slot / page].  One (page, key head)
// is page x d contiguous elements, the block that the attention over this cache
// fetches with one tile copy.
//
// Bound: HBM for long chunks (K and V read once and written once), launch and
// the chain seq, slot -> table -> store for single tokens.  A group of d/8 lanes
// takes one token's chunk of key heads: the page number and the rotation are
// found once per chunk, and K and V rows are loaded before either is needed.  28.9 k
// tokens of 8 key heads of 128 (237 MB): 44 us, 5.3 TB/s; with 4 heads a group 49 us, with
// 2 heads 61; four rows ahead instead of two 55.  Four blocks an SM leave 64 registers a thread,
// of which the rotation in halves spills 36 bytes, in pairs 12.  200 k tokens of one key head
// (205 MB): 70 us, 2.9 TB/s: a token's angles then serve one row and the instructions bound it.
#include "checks.cuh"
#include "rope.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;      // head rows (K and V each) loaded before the first is used
constexpr int kHeadChunk = 8;  // most key heads of one token that a group takes

struct AppendArgs {
  RopeParams p;
  const __nv_bfloat16 *k, *v;
  int64_t k_stride, v_stride;
  const float* wk;
  const int64_t* slot;  // or null: pos
  const int32_t *seq, *table;
  __nv_bfloat16 *Kp, *Vp;
  int64_t T, n_pages;
  int B, max_pages, page_shift, Hk, chunk, chunks;
  int* status;
};

template <int D, int STYLE>
__global__ void __launch_bounds__(kThreads, 4) paged_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int LPR = D / 8, GROUPS = kThreads / LPR;
  __shared__ uint64_t s_turn[kRopeMaxPairs];
  const int64_t unit = (int64_t)blockIdx.x * GROUPS + threadIdx.x / LPR;
  const int64_t t = unit / a.chunks;
  const bool live = t < a.T;
  const int h0 = (int)(unit % a.chunks) * a.chunk;
  const int n = a.Hk - h0 < a.chunk ? a.Hk - h0 : a.chunk;
  const RopeLane rl = rope_lane<D, STYLE>(a.p);
  const int64_t pos = live ? a.p.pos[t] : 0;
  const int64_t slot = live ? (a.slot ? a.slot[t] : pos) : -1;
  const int b = live ? a.seq[t] : 0;
  const __nv_bfloat16* k = a.k + t * a.k_stride + (int64_t)h0 * D + 8 * rl.l;
  const __nv_bfloat16* v = a.v + t * a.v_stride + (int64_t)h0 * D + 8 * rl.l;
  Raw8b rk[kAhead], rv[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (live && u < n) load8(k + u * D, rk[u]), load8(v + u * D, rv[u]);
  stage_turns(a.p, s_turn);
  if (!live || slot < 0) return;  // a padding row
  const int64_t pg = slot >> a.page_shift;
  int64_t page = -1;
  if (b >= 0 && b < a.B && pg < a.max_pages) page = a.table[(int64_t)b * a.max_pages + pg];
  if (page < 0 || page >= a.n_pages) {
    report(a.status, CSA_ERR_INDEX);
    return;
  }
  const uint32_t mask = group_mask<D>();
  float A[8], B[8];
  {
    float w[8], wp[8], c[8], s[8];
    load_weights(a.wk, rl.l, w);
    load_weights(a.wk, rl.partner % LPR, wp);
    rope_angles<STYLE>(rl, s_turn, pos, mask, c, s);
    rope_coef<STYLE>(rl, c, s, w, wp, A, B);
  }
  const bool norm = a.wk != nullptr;
  const int64_t row0 = ((page * a.Hk + h0) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
  for (int h = 0; h < n; h += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (h + u >= n) break;
      const Raw8b ck = rk[u], cv = rv[u];
      if (h + u + kAhead < n) {
        load8(k + (int64_t)(h + u + kAhead) * D, rk[u]);
        load8(v + (int64_t)(h + u + kAhead) * D, rv[u]);
      }
      const int64_t at = (row0 + ((int64_t)(h + u) << a.page_shift)) * D + 8 * rl.l;
      float f[8], o[8];
      unpack8(ck, f);
      const float r = norm ? row_rms<D>(f, a.p.eps, mask) : 1.f;
      rope_row<STYLE>(ck, f, r, A, B, rl, mask, o);
      store8(a.Kp + at, o);
      *reinterpret_cast<uint4*>(a.Vp + at) = cv.v;
    }
  }
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" int csa_paged_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* wk,
                                float eps, const int64_t* pos, const int64_t* slot, const int32_t* seq,
                                const double* inv_freq, int rot_start, int rot_dim, int rot_style,
                                const int32_t* block_table, int64_t T, int Hk, int d, int B, int max_pages,
                                int64_t n_pages, int page, void* Kpages, void* Vpages, void* workspace,
                                size_t workspace_bytes, csa_stream_t stream) {
  if (T < 0 || Hk < 1 || Hk > 4096 || B < 0 || max_pages < 0 || n_pages < 0) return CSA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return CSA_ERR_UNSUPPORTED_SHAPE;
  if (!valid_page(page)) return CSA_ERR_UNSUPPORTED_SHAPE;
  if (k_stride < (int64_t)Hk * d || v_stride < (int64_t)Hk * d || k_stride % 8 != 0 || v_stride % 8 != 0)
    return CSA_ERR_INVALID_ARG;
  int rc = check_rotation(d, inv_freq, rot_start, rot_dim, rot_style, eps);
  if (rc) return rc;
  if ((rc = check_ws(workspace, workspace_bytes, kWorkspaceHeader))) return rc;
  if (T == 0) return CSA_OK;
  if ((rc = check_ptrs(k, v, pos, seq))) return rc;
  if ((rc = check_opt(wk)) || (rc = check_opt(slot))) return rc;
  if (B > 0 && max_pages > 0 && (rc = check_ptrs(block_table))) return rc;
  if (n_pages > 0 && (rc = check_ptrs(Kpages, Vpages))) return rc;
  const size_t cache = (size_t)n_pages * Hk * page * d * 2;
  for (const void* c : {Kpages, Vpages})
    if (overlap_any({c, cache}, {{k, span(T, k_stride, Hk, d, CSA_BF16)},
                                 {v, span(T, v_stride, Hk, d, CSA_BF16)},
                                 {wk, (size_t)d * 4},
                                 {pos, (size_t)T * 8},
                                 {slot, (size_t)T * 8},
                                 {seq, (size_t)T * 4},
                                 {block_table, (size_t)B * max_pages * 4}}))
      return CSA_ERR_INVALID_ARG;
  if (overlap(Kpages, cache, Vpages, cache)) return CSA_ERR_INVALID_ARG;
  AppendArgs a{};
  if (!rope_params(inv_freq, rot_dim, a.p)) return CSA_ERR_INVALID_ARG;
  a.p.pos = pos;
  a.p.start = rot_start;
  a.p.rot = rot_dim;
  a.p.style = rot_style;
  a.p.eps = eps;
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.wk = wk;
  a.slot = slot;
  a.seq = seq;
  a.table = block_table;
  a.Kp = static_cast<__nv_bfloat16*>(Kpages);
  a.Vp = static_cast<__nv_bfloat16*>(Vpages);
  a.T = T;
  a.n_pages = n_pages;
  a.B = max_pages > 0 ? B : 0;
  a.max_pages = max_pages;
  while ((1 << a.page_shift) < page) ++a.page_shift;
  a.Hk = Hk;
  a.chunk = rope_head_chunk(T, Hk, d, kHeadChunk);
  a.chunks = (int)ceil_div(Hk, a.chunk);
  a.status = status_word(workspace);
  const int64_t grid = ceil_div(T * a.chunks, kThreads / (d / 8));
  if (grid > 0x7FFFFFFF) return CSA_ERR_UNSUPPORTED_SHAPE;
  const bool halves = rot_style == CSA_ROPE_HALVES;
  auto kern = d == 128 ? (halves ? paged_append_kernel<128, CSA_ROPE_HALVES> : paged_append_kernel<128, CSA_ROPE_PAIRS>)
                       : (halves ? paged_append_kernel<64, CSA_ROPE_HALVES> : paged_append_kernel<64, CSA_ROPE_PAIRS>);
  cudaError_t e = launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), 0, (cudaStream_t)stream, false, a);
  return e == cudaSuccess ? CSA_OK : cuda_fail(e);
}
