// Attention over the paged 8-bit cache: decode, causal chunks, cross attention.
// logit = scale <q, k>, p = softmax over the visible tokens, out = sum p v, k and v the
// values the codes stand for.
#include <cuda_fp8.h>

#include "paged.cuh"

namespace tq {
namespace {

// A workspace begins with this word (tq_paged_workspace_init), so that one that was never made
// ready is reported instead of used.
constexpr uint32_t kWsMagic = 0x70384b56u;
constexpr size_t kWsHeader = 4096;

__global__ void k_paged_ws_init(uint32_t* ws) {
  pdl_wait();
  for (int i = threadIdx.x; i < (int)(kWsHeader / 4); i += blockDim.x) ws[i] = i == 0 ? kWsMagic : 0u;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float byte_value(uint32_t u, int code) {
  if (code == TQ_CODE_INT8) return (float)((int)u - 128);
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)u, __NV_E4M3)));
}

// One warp per (query token, head), a token at a time: the form every other is held against.
template <int D>
__global__ void __launch_bounds__(128) k_paged_attn_plain(PGeom g, PagedAttn a) {
  pdl_wait();
  if (*static_cast<const uint32_t*>(a.ws) != kWsMagic) {
    if (threadIdx.x == 0) atomicOr(&g.state->status, kPagedBadWorkspace);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= a.total_q * a.Hq) return;
  const int64_t tok = w / a.Hq;
  const int hq = (int)(w % a.Hq), h = hq / (a.Hq / g.Hkv);
  if (tok >= a.cu[a.n] || tok < a.cu[0]) return;      // rows behind the last sequence stay
  int i = 0;
  for (int lo = 0, hi = a.n; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= tok) lo = mid; else hi = mid;
    i = lo;
  }
  const int slot = a.slots[i], len = paged_len(g, slot);
  const int nq = a.cu[i + 1] - a.cu[i], qi = (int)(tok - a.cu[i]);
  if (nq > a.max_q && lane == 0) atomicOr(&g.state->status, kPagedBadOffsets);
  const int vis = a.causal ? max(0, min(len, len - nq + qi + 1)) : len;
  constexpr int N = D / 32;
  float q[N], o[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    q[k] = load_f(a.Q, tok * a.q_stride + (int64_t)hq * D + 32 * k + lane, g.dtype);
    o[k] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < vis; ++t) {
    const int pid = g.table[(int64_t)slot * g.max_pages + t / g.page];
    if ((unsigned)pid >= (unsigned)g.pages) continue;
    const int si = t % g.page / g.sub, tb = t % g.page % g.sub;
    const uint8_t* kb = paged_block(g, a.layer, pid, 0, h, si);
    const uint8_t* vb = paged_block(g, a.layer, pid, 1, h, si);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) s = fmaf(q[k], byte_value(kb[paged_k_off(D, tb, 32 * k + lane)], g.code), s);
    s = warp_sum(s) * *reinterpret_cast<const float*>(kb + g.sub * D) * a.scale;
    const float mn = fmaxf(m, s), al = exp2f((m - mn) * kLog2e), p = exp2f((s - mn) * kLog2e);
    const float sv = *reinterpret_cast<const float*>(vb + g.sub * D) * p;
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = fmaf(sv, byte_value(vb[(32 * k + lane) * g.sub + tb], g.code), o[k] * al);
    l = l * al + p;
    m = mn;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) store_f(a.out, w * D + 32 * k + lane, g.dtype, l > 0.f ? o[k] / l : 0.f);
  if (a.lse && lane == 0) a.lse[w] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t paged_attn_ws_bytes(int d) { return kWsHeader; }
cudaError_t paged_launch_ws_init(void* ws, cudaStream_t s) {
  return launch_pdl(k_paged_ws_init, dim3(1), dim3(256), 0, s, static_cast<uint32_t*>(ws));
}

cudaError_t paged_launch_attention(const PGeom& g, const PagedAttn& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.total_q * a.Hq + 3) / 4));
  if (g.d == 64) return launch_pdl(k_paged_attn_plain<64>, grid, dim3(128), 0, s, g, a);
  if (g.d == 128) return launch_pdl(k_paged_attn_plain<128>, grid, dim3(128), 0, s, g, a);
  return launch_pdl(k_paged_attn_plain<256>, grid, dim3(128), 0, s, g, a);
}

TQ_BOUNDS_READER(bounds_flag_paged_attn)

}  // namespace tq
