// Attention of many query rows over the paged 8-bit cache (chunks, prompts, cross attention
// of bf16 / f16 models) on the fifth-generation tensor cores.
//
// A CTA works on R = 128 MT query rows of one KV head (row r: query r / G, head r mod G, so that
// grouped heads share every tile) and walks its share of their tiles of T tokens:
//   S_w = Q_w K^T       A = Q_w (128 x D, shared memory), B = K (T x D), fp32 in tensor memory
//   P_w = 2^(f S_w + log2 s_v - M)      a thread per row, f16 back into tensor memory over S_w
//   O_w += P_w V        A = P_w (tensor memory), B = V (D x T, shared memory)
// Four kinds of warps: one warpgroup per row block w (softmax), three converter warps that read
// the next tile's codes into registers while they expand the last one's into the f16 operands,
// and one warp whose first thread issues the products.  The products of one row block run while
// the other's softmax does; with MT = 1 two S buffers take their place.
//
// The scales enter exactly and at no cost per element: a page's key scale multiplies the row's
// factor f (one per 16 tokens), its value scale is added to the exponent, so that O sums code
// products only.  M is a running reference of f S + log2 s_v, raised only when a tile passes it by
// more than 2^4 (O is rescaled then); p is at most 2^15, and p <= 2^11 when M is fresh.  The
// weights' sum, taken in fp32 before p is rounded to f16, divides s_v out again, against the
// first tile's scale so that it stays in range.  Rounding p to f16 (2^-11 relative, as fine as the
// output's own rounding) is the one loss beside q's, which is held to 2^-11 of a f16 entry's own
// bits or exactly (bf16, f16 entries have at most 11 bits; q is scaled by a power of two per row).
#include "paged_split.cuh"
#include "tc_common.cuh"

namespace tq {
namespace {
using namespace paged;

constexpr int kChunkCtas = 148;
constexpr int kConv = 3;                   // converter warps; the products' warp completes their warpgroup
constexpr float kNone = -1e30f;            // reference of a row that has seen no token
constexpr float kBias = 11.f;              // p is held times 2^11
constexpr float kSlack = 4.f;

template <int D>
__host__ __device__ constexpr int chunk_tokens() { return D == 256 ? 64 : 128; }
template <int D>
__host__ __device__ constexpr int chunk_max_mt() { return D == 256 ? 1 : 2; }
template <int D, int MT>
__host__ __device__ constexpr size_t chunk_smem() {
  return (size_t)MT * 128 * D * 2 + 4 * (size_t)chunk_tokens<D>() * D * 2;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, f16 operands, issued by one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct ChunkWs {
  int* count;          // [CTAs]
  float* lse;          // [2 x CTAs][R] log2 of a part's weight sum (-inf: none)
  float* o;            // [2 x CTAs][R][D] a part's output
};
template <int D, int MT>
__device__ __forceinline__ ChunkWs chunk_ws(void* ws) {
  ChunkWs w;
  unsigned char* p = static_cast<unsigned char*>(ws);
  w.count = reinterpret_cast<int*>(p + 256);
  w.lse = reinterpret_cast<float*>(p + kWsHeader);
  w.o = w.lse + (size_t)2 * kChunkCtas * 128 * MT;
  return w;
}

template <int D, int MT>
struct ChunkShared {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_ready[2], pv_done[2];
  uint64_t scales[4];
  int64_t sum[4 * MT + 4];
  float sk[4][8], lv[4][8];                // a tile's scales per 16 tokens: of the keys, log2 of the values'
  Cursor cur;
  uint32_t tmem;
  int abort, last;
};

template <int D, int CODE, int MT>
__global__ void __launch_bounds__(128 * MT + 128, 1) k_paged_chunk(PGeom g, PagedAttn a) {
  constexpr int T = chunk_tokens<D>(), R = 128 * MT, NTH = R + 128;
  constexpr int NG = T / 16;                          // 16-token groups of a tile
  constexpr int NB = T * D / 512;                     // 8-row x 64-byte pieces of a tile's keys (values)
  constexpr int NK = (NB + kConv - 1) / kConv;        // of them per converter warp
  constexpr uint32_t kTb = T * D * 2;                 // bytes of an f16 operand tile
  constexpr uint32_t cO = 0, cS = MT * D;             // tensor memory columns
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ ChunkShared<D, MT> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wg = warp >> 2;                           // < MT: softmax of row block wg
  const bool is_soft = wg < MT, is_mma = warp == 4 * MT + kConv, is_conv = !is_soft && !is_mma;
  const uint32_t sQ = smem_u32(smem), sK = sQ + R * D * 2, sV = sK + 2 * kTb;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(&sh.scales[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], kConv);
      mbar_init(&sh.k_free[i], 1);
      mbar_init(&sh.v_full[i], kConv);
      mbar_init(&sh.v_free[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_ready[i], 4);
      mbar_init(&sh.pv_done[i], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sh.abort = 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  const int G = a.Hq / g.Hkv;
  if (*static_cast<const volatile uint32_t*>(a.ws) != kWsMagic) {
    if (tid == 0) atomicOr(&g.state->status, kPagedBadWorkspace);
    return;
  }
  if (cta_first_checks(g, a)) atomicOr(&g.state->status, kPagedBadOffsets);
  const int64_t W = count_tiles<R, T, NTH>(g, a, G, sh.sum);
  if (W == 0) return;
  const int64_t C = share_ctas(W, gridDim.x, 2);
  const int cta = blockIdx.x;
  if (cta >= C) return;
  const int64_t x0 = share_begin(W, C, cta), x1 = share_begin(W, C, cta + 1);
  if (warp == 0) {
    const Cursor f = find_unit<R, T>(g, a, G, x0);
    if (lane == 0) sh.cur = f;
  }
  if (is_mma) {
    tc::tmem_alloc(smem_u32(&sh.tmem), 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;
  Cursor cur = sh.cur;
  const ChunkWs ws = chunk_ws<D, MT>(a.ws);
  auto wait = [&](uint64_t* bar, int index) {         // completion `index` (0, 1, ...) of a barrier
    if (*static_cast<volatile int*>(&sh.abort)) return;
    if (!mbar_wait_timed(bar, (uint32_t)(index & 1))) {
      sh.abort = 1;
      atomicOr(&g.state->status, kPagedWait);
    }
  };

  int n0 = 0;                                         // tiles of this CTA before the segment
  int64_t x = x0;
  while (x < x1) {
    const int64_t ue = cur.u0 + cur.nt, xe = min(x1, ue);
    const int uvis = group_visible<R>(cur.s, G, cur.rg, a.causal);
    const int nt = uvis > 0 ? (int)(xe - x) : 0;      // tiles of the segment
    const int tok0 = (int)(x - cur.u0) * T;           // its first token
    const int rows = (int)min((int64_t)R, (int64_t)cur.s.nq * G - (int64_t)cur.rg * R);
    float fr = 0.f, M = kNone, l = 0.f, lvr = 0.f;
    int vis = 0;
    __syncthreads();                                  // the last segment's operands are free

    if (is_soft) {
      // ---- this thread's query row into the A operand
      const int r = tid, row = cur.rg * R + r;
      const int64_t tok = (int64_t)cur.s.q0 + row / G;
      const bool ok = r < rows && tok >= 0 && tok < a.total_q;
      if (ok) vis = visible(cur.s, row / G, a.causal);
      uint4 q[D / 8];
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.Q) + tok * a.q_stride +
                                                        (int64_t)(cur.h * G + row % G) * D);
#pragma unroll
      for (int k = 0; k < D / 8; ++k) q[k] = ok ? src[k] : make_uint4(0, 0, 0, 0);
      auto both = [&](uint32_t u) {
        return g.dtype == TQ_F16 ? __half22float2(*reinterpret_cast<const __half2*>(&u))
                                 : make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
      };
      float mx = 0.f;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = both(w[i]);
          const float t0 = fabsf(v.x), t1 = fabsf(v.y);
          mx = fmaxf(mx, t0 <= 3.402823466e38f ? t0 : 0.f);
          mx = fmaxf(mx, t1 <= 3.402823466e38f ? t1 : 0.f);
        }
      }
      // the largest entry of the row into [2^14, 2^15); a negative scale turns the row's sign
      int e = mx > 0.f ? 141 - (int)(__float_as_uint(mx) >> 23) : 0;
      e = min(e, 120);
      const float up = copysignf(__int_as_float((127 + e) << 23), a.scale);
      fr = ok ? fabsf(a.scale) * kLog2e * __int_as_float((127 - e) << 23) : 0.f;
      unsigned char* Q = smem + (size_t)(r >> 7) * 128 * D * 2;
      const int rr = r & 127;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = both(w[i]);
          o[i] = pack_half(v.x * up, v.y * up);
        }
        *reinterpret_cast<uint4*>(Q + ((rr >> 3) * (D / 8) + k) * 128 + (rr & 7) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      tc::fence_async_shared();
    }
    __syncthreads();

    if (is_conv) {
      // ================================================= converters
      const int cw = warp & 3;
      const int lsub = 31 - __clz(g.sub);
      const int64_t vofs = (int64_t)g.Hkv * g.hb;
      const int last = cur.s.len - 1;
      uint4 kr[NK], vr[NK];
      const uint8_t* ptr = nullptr;                   // lane k: key sub-block k of the tile in hand
      float sk = 0.f, sv = 0.f;
      int pid = 0, psub = 0;
      auto look = [&](int t) {                        // lane k: page of sub-block k of tile t
        const int tk = min(tok0 + t * T + (lane << lsub), last);     // past the end: the last one, masked
        pid = lane < (T >> lsub) ? g.table[(int64_t)cur.s.slot * g.max_pages + tk / g.page] : 0;
        psub = (tk % g.page) >> lsub;
      };
      auto aim = [&]() {
        if ((unsigned)pid >= (unsigned)g.pages) {
          atomicOr(&g.state->status, kPagedBadPage);
          pid = 0;
        }
        ptr = paged_block(g, a.layer, pid, 0, cur.h, psub);
      };
      auto sub_ptr = [&](int i) {                     // sub-block i's pointer, from lane i
        return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(ptr), i));
      };
      auto load_k = [&]() {
#pragma unroll
        for (int it = 0; it < NK; ++it) {
          const int b = it * kConv + cw, row = (b / (D / 64)) * 8 + (lane & 7), ch = (b % (D / 64)) * 4 + (lane >> 3);
          if (b >= NB) break;
          const uint8_t* p = sub_ptr(row >> lsub) + paged_k_off(D, row & (g.sub - 1), 16 * ch);
          kr[it] = TQ_CHECKED(p, 16, g.base, g.total, 421) ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
        }
        const uint8_t* p = sub_ptr((16 * (lane & (NG - 1))) >> lsub);
        sk = *reinterpret_cast<const float*>(p + g.sub * D);
        sv = *reinterpret_cast<const float*>(p + vofs + g.sub * D);
      };
      auto load_v = [&]() {
#pragma unroll
        for (int it = 0; it < NK; ++it) {
          const int b = it * kConv + cw, ch = (b / (T / 64)) * 8 + (lane & 7), q = (b % (T / 64)) * 4 + (lane >> 3);
          if (b >= NB) break;
          const uint8_t* p = sub_ptr((16 * q) >> lsub) + vofs + ((int64_t)ch << lsub) + ((16 * q) & (g.sub - 1));
          vr[it] = TQ_CHECKED(p, 16, g.base, g.total, 422) ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
        }
      };
      auto put = [&](unsigned char* to, const uint4& v) {        // 16 codes -> two 16-byte pieces of a row
        uint32_t o[8];
        expand4<CODE>(v.x, o[0], o[1]);
        expand4<CODE>(v.y, o[2], o[3]);
        expand4<CODE>(v.z, o[4], o[5]);
        expand4<CODE>(v.w, o[6], o[7]);
        *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(to + 128) = make_uint4(o[4], o[5], o[6], o[7]);
      };
      if (nt > 0) {
        look(0);
        aim();
        load_k();
        load_v();
        if (nt > 1) look(1);
      }
      for (int t = 0; t < nt; ++t) {
        const int n = n0 + t, b2 = n & 1;
        unsigned char* K = smem + R * D * 2 + b2 * kTb;
        unsigned char* V = K + 2 * kTb;
        if (n >= 2) wait(&sh.k_free[b2], (n >> 1) - 1);
        // four sets of scales: the products of tile n - 2 are done, so the softmax of tile n - 4 is
        if (cw == 0 && lane < NG) {
          sh.sk[n & 3][lane] = sk;
          sh.lv[n & 3][lane] = sv > 0.f ? __log2f(sv) : 0.f;     // a block of zeros: any scale will do
        }
        __syncwarp();
        if (cw == 0 && lane == 0) mbar_arrive(&sh.scales[n & 3]);
#pragma unroll
        for (int it = 0; it < NK; ++it) {
          const int b = it * kConv + cw, rg = b / (D / 64), ch = (b % (D / 64)) * 4 + (lane >> 3);
          if (b < NB) put(K + (rg * (D / 8) + 2 * ch) * 128 + (lane & 7) * 16, kr[it]);
        }
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.k_full[b2]);
        // the next tile's pages were looked up a tile ago; its keys travel while the values expand
        if (t + 1 < nt) {
          aim();
          load_k();
          if (t + 2 < nt) look(t + 2);
        }
        if (n >= 2) wait(&sh.v_free[b2], (n >> 1) - 1);
#pragma unroll
        for (int it = 0; it < NK; ++it) {
          const int b = it * kConv + cw, rg = b / (T / 64), q = (b % (T / 64)) * 4 + (lane >> 3);
          if (b < NB) put(V + (rg * (T / 8) + 2 * q) * 128 + (lane & 7) * 16, vr[it]);
        }
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.v_full[b2]);
        if (t + 1 < nt) load_v();
      }
    } else if (is_mma) {
      // ================================================= products
      if (lane == 0 && nt > 0) {
        constexpr uint32_t iS = tc::idesc_f16(128, T), iO = tc::idesc_f16(128, D);
        auto qk = [&](int w, int sb, int b2) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma_f16(tmem + cS + sb * T, tc::smem_desc_sbo(sQ + w * 128 * D * 2 + 256 * k, 16 * D),
                        tc::smem_desc_sbo(sK + b2 * kTb + 256 * k, 16 * D), iS, k > 0);
        };
        auto pv = [&](int w, int sb, int b2, bool first) {
#pragma unroll
          for (int k = 0; k < T / 16; ++k)
            mma_f16_ts(tmem + cO + w * D, tmem + cS + sb * T + 8 * k,
                       tc::smem_desc_sbo(sV + b2 * kTb + 256 * k, 16 * T), iO, !(first && k == 0));
        };
        if constexpr (MT == 2) {
          wait(&sh.k_full[n0 & 1], n0 >> 1);
          tc::fence_after_sync();
          qk(0, 0, n0 & 1);
          tc::mma_commit(smem_u32(&sh.s_full[0]));
          qk(1, 1, n0 & 1);
          tc::mma_commit(smem_u32(&sh.s_full[1]));
          tc::mma_commit(smem_u32(&sh.k_free[n0 & 1]));
          for (int t = 0; t < nt; ++t) {
            const int n = n0 + t, b2 = n & 1, m = n + 1;
            wait(&sh.v_full[b2], n >> 1);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              wait(&sh.p_ready[w], n);
              tc::fence_after_sync();
              pv(w, w, b2, t == 0);
              tc::mma_commit(smem_u32(&sh.pv_done[w]));
              if (w == 1) tc::mma_commit(smem_u32(&sh.v_free[b2]));
              if (t + 1 < nt) {
                if (w == 0) wait(&sh.k_full[m & 1], m >> 1);
                wait(&sh.pv_done[w], n);              // P_w lies over S_w
                tc::fence_after_sync();
                qk(w, w, m & 1);
                tc::mma_commit(smem_u32(&sh.s_full[w]));
                if (w == 1) tc::mma_commit(smem_u32(&sh.k_free[m & 1]));
              }
            }
          }
        } else {
          for (int t = -1; t < nt; ++t) {
            const int n = n0 + t, m = n + 1;
            if (t + 1 < nt) {
              wait(&sh.k_full[m & 1], m >> 1);
              if (t >= 1) wait(&sh.pv_done[m & 1], (n - 1) >> 1);      // its P lies over this S buffer
              tc::fence_after_sync();
              qk(0, m & 1, m & 1);
              tc::mma_commit(smem_u32(&sh.s_full[m & 1]));
              tc::mma_commit(smem_u32(&sh.k_free[m & 1]));
            }
            if (t >= 0) {
              wait(&sh.v_full[n & 1], n >> 1);
              wait(&sh.p_ready[n & 1], n >> 1);
              tc::fence_after_sync();
              pv(0, n & 1, n & 1, t == 0);
              tc::mma_commit(smem_u32(&sh.pv_done[n & 1]));
              tc::mma_commit(smem_u32(&sh.v_free[n & 1]));
            }
          }
        }
      }
      __syncwarp();
    } else {
      // ================================================= softmax
      const uint32_t lrow = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t tO = tmem + lrow + cO + wg * D;
      // A parity tells a completion only from its neighbours, so every waiter has to be within one
      // of it.  MT = 2: S_w of tile n came after the products P V of n - 1.  MT = 1: after those of
      // n - 2 only, hence a barrier per buffer.
      auto pv_wait = [&](int n) {
        if (MT == 2) wait(&sh.pv_done[wg], n); else wait(&sh.pv_done[n & 1], n >> 1);
      };
      // rows of the warp see at least wmin tokens (those in use)
      const int wmin = __reduce_min_sync(0xffffffffu, vis);
      for (int t = 0; t < nt; ++t) {
        const int n = n0 + t, sc = n & 3;
        const uint32_t tS = tmem + lrow + cS + (MT == 2 ? wg : n & 1) * T;
        const int base = tok0 + t * T;                 // the tile's first token
        wait(&sh.scales[sc], n >> 2);
        if (MT == 2) wait(&sh.s_full[wg], n); else wait(&sh.s_full[n & 1], n >> 1);
        tc::fence_after_sync();
        if (t == 0) lvr = sh.lv[sc][0];
        const bool masked = base + T > wmin;           // uniform in the warp
        uint32_t pk[T / 2];
        float zmax, ladd;
        // exponents f S + c of the tile against M; their largest, and (EXP) p and its sum
        auto pass = [&](auto EXP, auto MASK) {
          zmax = -INFINITY;
          ladd = 0.f;
#pragma unroll
          for (int c = 0; c < T / 32; ++c) {
            uint32_t v[32];
            tc::tmem_ld32(tS + 32 * c, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float f = fr * sh.sk[sc][2 * c + h];
              const float lv = sh.lv[sc][2 * c + h];
              const float cst = decltype(EXP)::value ? lv - M + kBias : lv;
              const float2 f2 = make_float2(f, f), c2 = make_float2(cst, cst);
              float2 ls = make_float2(0.f, 0.f);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int col = 32 * c + 16 * h + 2 * i;
                float2 z = fma2(make_float2(__uint_as_float(v[16 * h + 2 * i]), __uint_as_float(v[16 * h + 2 * i + 1])), f2, c2);
                if (decltype(MASK)::value) {
                  z.x = base + col < vis ? z.x : -INFINITY;
                  z.y = base + col + 1 < vis ? z.y : -INFINITY;
                }
                zmax = fmaxf(zmax, fmaxf(z.x, z.y));
                if (decltype(EXP)::value) {
                  const float2 p = make_float2(ex2(z.x), ex2(z.y));
                  ls = add2(ls, p);
                  pk[16 * c + 8 * h + i] = pack_half(p.x, p.y);
                }
              }
              if (decltype(EXP)::value) ladd = fmaf(ls.x + ls.y, ex2(lvr - lv), ladd);
            }
          }
        };
        bool fresh = __any_sync(0xffffffffu, M == kNone && vis > base);
        for (;;) {
          if (fresh) {
            if (masked) pass(std::false_type(), std::true_type()); else pass(std::false_type(), std::false_type());
            const float Mn = M == kNone ? (zmax == -INFINITY ? kNone : zmax) : fmaxf(M, zmax);
            const float alpha = M == kNone ? 0.f : ex2(M - Mn);
            M = Mn;
            l *= alpha;
            if (t > 0) {
              pv_wait(n - 1);
              tc::fence_after_sync();
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tc::tmem_ld32(tO + 32 * c, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                tc::tmem_st32(tO + 32 * c, v);
              }
            }
          }
          if (masked) pass(std::true_type(), std::true_type()); else pass(std::true_type(), std::false_type());
          if (fresh) break;
          fresh = __any_sync(0xffffffffu, zmax > kBias + kSlack);
          if (!fresh) break;
        }
        l += ladd;
#pragma unroll
        for (int c = 0; c < T / 64; ++c) {
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = pk[32 * c + i];
          tc::tmem_st32(tS + 32 * c, v);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        // (a warp may finish tile n + 1 before another has finished n, but not n + 2)
        if (lane == 0) mbar_arrive(&sh.p_ready[MT == 2 ? wg : n & 1]);
      }
      // ---- the row's output, or its part
      const bool whole = x == cur.u0 && xe == ue;
      const int r = tid, row = cur.rg * R + r;
      const int64_t tok = (int64_t)cur.s.q0 + row / G;
      const int hq = cur.h * G + row % G;
      const bool ok = r < rows && tok >= 0 && tok < a.total_q;
      const float inv = l > 0.f ? ex2(lvr) / l : 0.f;
      const float lse2 = l > 0.f ? log2f(l) + (M - lvr - kBias) : -INFINITY;
      const int slot = 2 * cta + (x == cur.u0 ? 1 : 0);
      if (nt > 0) {
        pv_wait(n0 + nt - 1);
        tc::fence_after_sync();
      }
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        if (nt > 0) {
          tc::tmem_ld32(tO + 32 * c, v);
          tc::tmem_wait_ld();
        }
        float o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = l > 0.f ? __uint_as_float(v[i]) * inv : 0.f;
        if (!whole) {
          float4* po = reinterpret_cast<float4*>(ws.o + ((int64_t)slot * R + r) * D + 32 * c);
          if (r < rows)
#pragma unroll
            for (int i = 0; i < 8; ++i) po[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else if (ok) {
          uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (tok * a.Hq + hq) * D + 32 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (g.dtype == TQ_F16) {
                w[k] = pack_half(o[8 * i + 2 * k], o[8 * i + 2 * k + 1]);
              } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(o[8 * i + 2 * k], o[8 * i + 2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t*>(&b);
              }
            }
            to[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (whole) {
        if (ok && a.lse) a.lse[tok * a.Hq + hq] = lse2 * (1.f / kLog2e);
      } else {
        if (r < rows) ws.lse[slot * R + r] = lse2;
        __threadfence();
      }
      tc::fence_before_sync();
    }

    if (!(x == cur.u0 && xe == ue)) {
      // the CTA that finishes its part of the unit last joins the parts, in their order
      const int c0 = share_owner(W, C, cur.u0), c1 = share_owner(W, C, ue - 1);
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        sh.last = atomicInc(reinterpret_cast<unsigned*>(&ws.count[c0]), (unsigned)(c1 - c0)) == (unsigned)(c1 - c0);
        __threadfence();
      }
      __syncthreads();
      if (sh.last) {
        auto slot_of = [&](int p) { return p == c0 ? 2 * p + 1 : 2 * p; };
        constexpr int Q4 = D / 4;
        for (int i = tid; i < rows * Q4; i += NTH) {
          const int r = i / Q4, k = i % Q4;
          float m = -INFINITY, L = 0.f;
          for (int p = c0; p <= c1; ++p) m = fmaxf(m, __ldcg(&ws.lse[slot_of(p) * R + r]));
          const float mu = m == -INFINITY ? 0.f : m;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p = c0; p <= c1; ++p) {
            const float w = ex2(__ldcg(&ws.lse[slot_of(p) * R + r]) - mu);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(ws.o + ((int64_t)slot_of(p) * R + r) * D) + k);
            L += w;
            o.x = fmaf(v.x, w, o.x);
            o.y = fmaf(v.y, w, o.y);
            o.z = fmaf(v.z, w, o.z);
            o.w = fmaf(v.w, w, o.w);
          }
          const float inv = L > 0.f ? 1.f / L : 0.f;
          const int row = cur.rg * R + r;
          const int64_t tok = (int64_t)cur.s.q0 + row / G;
          const int hq = cur.h * G + row % G;
          if (tok >= 0 && tok < a.total_q) {
            const int64_t at = (tok * a.Hq + hq) * D + 4 * k;
            if (g.dtype == TQ_F16) {
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                  make_uint2(pack_half(o.x * inv, o.y * inv), pack_half(o.z * inv, o.w * inv));
            } else {
              const __nv_bfloat162 b0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), b1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
            }
            if (a.lse && k == 0) a.lse[tok * a.Hq + hq] = L > 0.f ? (m + log2f(L)) * (1.f / kLog2e) : -INFINITY;
          }
        }
      }
    }
    n0 += nt;
    x = xe;
    if (x < x1) next_unit<R, T>(g, a, G, cur);
  }
  __syncthreads();
  if (is_mma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int D, int CODE, int MT>
cudaError_t chunk_t(const PGeom& g, const PagedAttn& a, cudaStream_t s) {
  constexpr size_t smem = chunk_smem<D, MT>();
  cudaError_t e = cudaFuncSetAttribute(k_paged_chunk<D, CODE, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_chunk<D, CODE, MT>, dim3(kChunkCtas), dim3(128 * MT + 128), smem, s, g, a);
}

template <int D>
cudaError_t chunk_d(const PGeom& g, const PagedAttn& a, cudaStream_t s) {
  const bool i8 = g.code == TQ_CODE_INT8;
  if constexpr (chunk_max_mt<D>() == 2) {
    // one row block where no sequence has more rows than it holds
    if ((int64_t)a.max_q * (a.Hq / g.Hkv) > 128)
      return i8 ? chunk_t<D, TQ_CODE_INT8, 2>(g, a, s) : chunk_t<D, TQ_CODE_E4M3, 2>(g, a, s);
  }
  return i8 ? chunk_t<D, TQ_CODE_INT8, 1>(g, a, s) : chunk_t<D, TQ_CODE_E4M3, 1>(g, a, s);
}

}  // namespace

size_t paged_chunk_ws_bytes(int d) {
  const size_t R = d == 256 ? 128 : 256;
  return kWsHeader + 2 * (size_t)kChunkCtas * R * (4 + 4 * (size_t)d);
}

cudaError_t paged_launch_chunk(const PGeom& g, const PagedAttn& a, cudaStream_t s) {
  if (g.d == 64) return chunk_d<64>(g, a, s);
  if (g.d == 128) return chunk_d<128>(g, a, s);
  return chunk_d<256>(g, a, s);
}

TQ_BOUNDS_READER(bounds_flag_paged_chunk)

}  // namespace tq
