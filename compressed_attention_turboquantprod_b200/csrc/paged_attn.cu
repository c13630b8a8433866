// Attention over the paged 8-bit cache: decode, causal chunks, cross attention.
// logit = scale <q, k>, p = softmax over the visible tokens, out = sum p v, k and v the
// values the codes stand for.
#include "paged_split.cuh"

namespace tq {
namespace {
using namespace paged;

// In the bounds-checked build tq_debug_paged_lose_copies makes the decode's copies fail their check, so
// that its waits run out, after a short time then.
#ifdef TQ_DEBUG_BOUNDS
__device__ int g_lose_copies;
#define TQ_LOSE_COPIES (*static_cast<volatile int*>(&g_lose_copies) != 0)
#else
#define TQ_LOSE_COPIES false
#endif

__global__ void k_paged_ws_init(uint32_t* ws) {
  pdl_wait();
  for (int i = threadIdx.x; i < (int)(kWsHeader / 4); i += blockDim.x) ws[i] = i == 0 ? kWsMagic : 0u;
}

constexpr int kTile = 64;

// ---------------------------------------------------------------- decode
// Up to 8 query rows of a KV head over its tokens, bound by reading the codes once.
//
// Both products run on warp-level m16n8k16 f16 MMA: 8 rows fill half an MMA, the other half
// carries what rounding the first to 11 bits left over (q in rows 0-7, q - f16(q) in rows
// 8-15, and p likewise), so that with exact f16 codes the products have 22 bits at no cost.
// q is scaled by a power of two per row so that its largest entry is in [2^14, 2^15).
//
// A warp owns whole tiles of 64 tokens: `cp.async.bulk` brings a tile's key sub-blocks, then
// its value sub-blocks, into the warp's own ring of stages; nothing in the loop waits for
// another warp.  No operand is shuffled: MMA k indices may be permuted alike in A and B, so
// lane (g, c) = (lane / 4, lane mod 4) reads 16 key bytes (channels 64 j + 16 c ...) of token
// 16 (g / 2) + 2 i + (g mod 2) for column g of n-tile i; its scores are then those of tokens
// 16 c + 2 i + {0, 1}: the 16 tokens whose value bytes are its one 16-byte read per channel.
// Each tile's P V starts from zero and is added to the fp32 output in round-to-nearest (the
// tensor core's own long sums truncate: 2^-25 a step, one way).
//
// Measured (one B200, copy peak 6466 GB/s): 8 sequences of 32768 tokens, 32 / 8 heads, d = 128, int8:
// 97-102 us on different cards for 537 MB, 0.82-0.86 of the peak, DRAM traffic 1.02 of that; d = 256, e4m3, 223 k tokens of 4 heads:
// 90 us, 0.79.  One sequence of 517 tokens: 15 us, a chain of about ten dependent loads and the first
// fetch of the code.  What bounds the long ones is latency within a warp: 8 warps an SM (4 at d = 256) at
// 44 % issue, as many as 240 registers allow; three CTAs at d = 64 (143 registers) gained nothing.
constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecRows = 8;

template <int D>
struct DecCfg {
  static constexpr int kCtas = D == 256 ? 1 : 2;              // resident CTAs per SM
  static constexpr int kStages = D == 64 ? 5 : 3;             // half tiles (keys or values) in flight per warp
};
// A sub-block's place in a stage: padded so that the four lanes c of a value read, which are in
// 64 / SUB sub-blocks, fall into different banks.
template <int D, int SUB>
__host__ __device__ constexpr int dec_sub_stride() { return SUB * D + 2 * SUB; }
template <int D, int SUB>
__host__ __device__ constexpr int dec_stage() { return kTile / SUB * dec_sub_stride<D, SUB>(); }
template <int D, int SUB>
__host__ __device__ constexpr size_t dec_smem() {
  return (size_t)kDecWarps * DecCfg<D>::kStages * dec_stage<D, SUB>() + (D / 16) * 32 * 16 +
         (kDecWarps / 2) * kDecRows * D * 4;
}

// Partials: [2 x CTAs][8] (m, l) and [2 x CTAs][8][D] o, after the workspace header.  CTA c
// writes slot 2 c for a unit that began before it, 2 c + 1 for one that goes on after it.
struct DecWs {
  int* count;          // [CTAs] finished parts of the unit that goes on after CTA c
  float2* ml;
  float* o;
};
constexpr int kMaxCtas = 2 * 148;

__host__ __device__ __forceinline__ DecWs dec_ws(void* ws) {
  DecWs w;
  unsigned char* p = static_cast<unsigned char*>(ws);
  w.count = reinterpret_cast<int*>(p + 256);
  w.ml = reinterpret_cast<float2*>(p + kWsHeader);
  w.o = reinterpret_cast<float*>(p + kWsHeader + (size_t)2 * kMaxCtas * kDecRows * 8);
  return w;
}

template <int D, int SUB, int CODE>
__global__ void __launch_bounds__(kDecThreads, DecCfg<D>::kCtas) k_paged_decode(PGeom g, PagedAttn a) {
  constexpr int NST = DecCfg<D>::kStages, SS = dec_sub_stride<D, SUB>(), STB = dec_stage<D, SUB>();
  constexpr int NSUB = kTile / SUB, KS = D / 16, NT = D / 8;
  constexpr uint32_t kBytes = NSUB * (SUB * D + kPagedTrailer);
  constexpr float kUp = 32768.f;           // p is held times 2^15: its halves reach 2^-40
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t s_full[kDecWarps][NST];
  __shared__ SplitPlan s_plan;
  __shared__ Cursor s_cur;
  __shared__ float s_fr[kDecRows];
  __shared__ int s_vis[kDecRows];
  __shared__ float2 s_ml[kDecWarps][kDecRows];
  __shared__ int s_abort, s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gi = lane >> 2, c = lane & 3;
  unsigned char* ring = smem + warp * (NST * STB);
  uint4* s_q = reinterpret_cast<uint4*>(smem + kDecWarps * NST * STB);          // [KS][32] A fragments
  float* s_o = reinterpret_cast<float*>(s_q + KS * 32);                         // [2 warps][8][D]
  if (tid == 0) {
    for (int w = 0; w < kDecWarps; ++w)
      for (int s = 0; s < NST; ++s) mbar_init(&s_full[w][s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_abort = 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  const int G = a.Hq / g.Hkv;
  const DivG by_g(G);
  const uint32_t magic = *static_cast<const volatile uint32_t*>(a.ws);
  const int cta = blockIdx.x;
  Cursor cur;
  int64_t W, C = 0, x0 = 0, x1 = 0;
  auto share = [&](int64_t w) {
    C = share_ctas(w, gridDim.x, kDecWarps);
    x0 = share_begin(w, C, cta);
    x1 = share_begin(w, C, cta + 1);
    return cta < C ? x0 : (int64_t)-1;
  };
  const bool few = a.n <= 32;
  if (few) {
    W = plan_in_warp<kDecRows, kTile, 0>(g, a, G, cur, share);
  } else {
    W = count_places<kDecRows, kTile, 0, kDecThreads>(g, a, G, s_plan);
    if (W > 0) share(W);
  }
  if (magic != kWsMagic) {
    if (tid == 0) atomicOr(&g.state->status, kPagedBadWorkspace);
    return;
  }
  if (cta_first_checks(g, a)) atomicOr(&g.state->status, kPagedBadOffsets);
  if (W == 0 || cta >= C) return;
  if (!few && warp == 0) {
    const Cursor f = find_unit<kDecRows, kTile, 0>(g, a, G, x0, s_plan);
    if (lane == 0) s_cur = f;
  }
  __syncthreads();                          // the barriers are initialised, the cursor is there
  if (!few) cur = s_cur;
  Cursor nxt = cur;                         // the unit of the tile to request next
  const DecWs ws = dec_ws(a.ws);

  // ---- requests: tile x belongs to warp x mod 4.  The pages of the warp's next tiles of a unit come 32
  // at a time: lane k holds that of sub-block k mod NSUB of the (k / NSUB)-th of them.
  constexpr int kBatch = 32 / NSUB;
  const int lpage = 31 - __clz(g.page);
  int64_t xi = x0 + ((warp - x0) & (kDecWarps - 1)), xb = xi;      // the next tile, the batch's first
  int nvis = 0, pids = 0;
  auto batch = [&]() {
    xb = xi;
    const int64_t t = (xi - nxt.u0 + (int64_t)(lane / NSUB) * kDecWarps) * kTile + (lane % NSUB) * SUB;
    // sub-blocks past the end repeat the last one: masked, but finite
    const int tk = (int)min(t, (int64_t)nxt.s.len - 1);
    pids = g.table[(int64_t)nxt.s.slot * g.max_pages + (tk >> lpage)];
  };
  // Find the tile at xi; tiles of a unit that sees nothing have nothing to load.
  auto look = [&]() {
    for (; xi < x1; xi += kDecWarps) {
      if (xi >= nxt.u0 + nxt.nt || nvis == 0) {
        while (xi >= nxt.u0 + nxt.nt) next_unit<kDecRows, kTile, 0>(g, a, G, nxt);
        nvis = group_visible<kDecRows>(nxt.s, G, nxt.rg, a.causal);
        if (nvis == 0) continue;
        batch();
      } else if (xi >= xb + kBatch * kDecWarps) {
        batch();
      }
      return;
    }
  };
  int ist = 0;                              // stage of the next request
  auto request = [&](int kv) {
    uint64_t* bar = &s_full[warp][ist];
    if (lane == 0) mbar_expect_tx(bar, kBytes);
    int pid = __shfl_sync(0xffffffffu, pids, (int)((xi - xb) / kDecWarps) * NSUB + (lane & (NSUB - 1)));
    if (lane < NSUB) {
      if ((unsigned)pid >= (unsigned)g.pages) {
        atomicOr(&g.state->status, kPagedBadPage);
        pid = 0;
      }
      const int tk = min((int)(xi - nxt.u0) * kTile + lane * SUB, nxt.s.len - 1);
      if (!TQ_LOSE_COPIES)
        cache_bulk_load(ring + ist * STB + lane * SS,
                        paged_block(g, a.layer, pid, kv, nxt.h, (tk & (g.page - 1)) / SUB), SUB * D + kPagedTrailer, bar,
                        g.base, g.total, 401);
    }
    ist = ist + 1 == NST ? 0 : ist + 1;
  };
  int half = 0;                             // 0: the keys of tile xi are next, 1: its values
  auto refill = [&]() {
    if (xi >= x1) return;
    request(half);
    half ^= 1;
    if (half == 0) {
      xi += kDecWarps;
      look();
    }
  };
  int cst = 0;
  uint32_t cph = 0;
  bool lost = false;
  int uvis = 0;                             // tokens that the unit's last row sees
  auto wait_stage = [&]() {
    const bool ok = mbar_wait_timed(&s_full[warp][cst], cph, &s_abort, TQ_LOSE_COPIES ? 1ll << 26 : kWaitCycles);
    // A wait that gave up ends the warp's requests (a stage still in flight must not be asked for again)
    // and its tiles: the call runs out on what there is, and the status says so.
    if (!__all_sync(0xffffffffu, ok)) {
      atomicOr(&g.state->status, kPagedWait);
      lost = true;
      xi = x1;
      uvis = 0;
    }
  };
  auto next_stage = [&]() {
    if (++cst == NST) {
      cst = 0;
      cph ^= 1;
    }
  };

  // ---- queries: warp w brings rows 2 w and 2 w + 1 of a unit, a unit ahead
  constexpr int NQ = D / 32;                // lane l holds channels NQ l .. NQ l + NQ - 1
  const bool f32 = g.dtype == TQ_F32, f16 = g.dtype == TQ_F16;
  uint32_t qn[2][NQ];                       // fp32, or two 16-bit entries a word in the first half of them
  auto bring = [&](const Cursor& u) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = u.rg * kDecRows + 2 * warp + j;
      const int q = by_g(row);
      const int64_t tok = (int64_t)u.s.q0 + q;
      const bool ok = row < u.s.nq * G && tok >= 0 && tok < a.total_q;
      const int64_t at = tok * a.q_stride + (u.h * G + row - q * G) * D + NQ * lane;
#pragma unroll
      for (int k = 0; k < NQ; ++k) qn[j][k] = 0;
      if (ok) {
        const uint32_t* p = static_cast<const uint32_t*>(a.Q) + (f32 ? at : at >> 1);
#pragma unroll
        for (int k = 0; k < NQ / 2; ++k) qn[j][k] = p[k];
        if (f32)
#pragma unroll
          for (int k = NQ / 2; k < NQ; ++k) qn[j][k] = p[k];
      }
    }
  };
  bring(cur);                               // (their latency passes behind the first requests')
  look();
#pragma unroll
  for (int st = 0; st < NST; ++st) refill();

  int64_t x = x0;
  while (x < x1) {
    const int64_t ue = cur.u0 + cur.nt, xe = min(x1, ue);
    // ---- the unit's queries as A fragments, two rows per warp
    __syncthreads();
    const int rows = (int)min((int64_t)kDecRows, (int64_t)cur.s.nq * G - (int64_t)cur.rg * kDecRows);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 2 * warp + j, row = cur.rg * kDecRows + r;
      const int64_t tok = (int64_t)cur.s.q0 + by_g(row);
      const bool ok = r < rows && tok >= 0 && tok < a.total_q;
      float qf[NQ], mx = 0.f;
#pragma unroll
      for (int k = 0; k < NQ; k += 2) {
        const float2 v = f32 ? make_float2(__uint_as_float(qn[j][k]), __uint_as_float(qn[j][k + 1])) : unpack2(qn[j][k / 2], f16);
        qf[k] = v.x;
        qf[k + 1] = v.y;
      }
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
        const float t = fabsf(qf[k]);
        mx = fmaxf(mx, t <= 3.402823466e38f ? t : 0.f);
      }
      mx = warp_max(mx);
      int e = mx > 0.f ? 141 - (int)(__float_as_uint(mx) >> 23) : 0;       // 2^e mx in [2^14, 2^15)
      e = min(e, 120);
      const float up = __int_as_float((127 + e) << 23);
      __half* A = reinterpret_cast<__half*>(s_q);
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
        const float v = qf[k] * up;
        const __half hi = __float2half_rn(v), lo = __float2half_rn(v - __half2float(hi));
        // channel 64 j + 16 c' + 4 w + b is k-step 4 j + w, lane (r, c'), register 2 (b / 2), half b mod 2
        const int ch = NQ * lane + k;
        const int ks = 4 * (ch >> 6) + ((ch >> 2) & 3), cc = (ch >> 4) & 3, b = ch & 3;
        __half* f = A + ((ks * 32 + 4 * r + cc) * 4 + 2 * (b >> 1)) * 2 + (b & 1);
        f[0] = hi;
        f[2] = lo;                                                       // the next register: row r + 8
      }
      if (lane == 0) {
        s_fr[r] = ok ? a.scale * kLog2e * __int_as_float((127 - e) << 23) : 0.f;
        s_vis[r] = ok ? visible(cur.s, by_g(row), a.causal) : 0;
      }
    }
    if (xe < x1) {
      Cursor after = cur;
      next_unit<kDecRows, kTile, 0>(g, a, G, after);
      bring(after);
    }
    __syncthreads();
    const float fr = s_fr[gi];
    const int vis = s_vis[gi];
    uvis = lost ? 0 : group_visible<kDecRows>(cur.s, G, cur.rg, a.causal);
    float m = -INFINITY, l = 0.f;
    float o[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = 0.f;

    for (int64_t xt = x + ((warp - x) & (kDecWarps - 1)); xt < xe && uvis > 0; xt += kDecWarps) {
      // ---- scores
      wait_stage();
      const unsigned char* kb = ring + cst * STB + (16 * (gi >> 1)) / SUB * SS + ((16 * (gi >> 1)) % SUB + (gi & 1)) * D + 16 * c;
      float sc[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll(D == 256 ? 4 : 1)            // (rolled where it costs nothing: every launch fetches the code anew)
      for (int j = 0; j < D / 64; ++j) {
        uint4 A[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) A[w] = s_q[(4 * j + w) * 32 + lane];
        const int jo = D == 64 ? 0 : (j ^ (gi & 1)) * 64;
        // four columns' products in turn: each waits for its own last one only
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += 4) {
          uint4 kw[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) kw[i] = *reinterpret_cast<const uint4*>(kb + 2 * (i0 + i) * D + jo);
          auto step = [&](auto word, const uint4& q) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t b0, b1;
              expand4<CODE>(word(kw[i]), b0, b1);
              hmma16816(sc[i0 + i], q.x, q.y, q.z, q.w, b0, b1);
            }
          };
          step([](const uint4& v) { return v.x; }, A[0]);
          step([](const uint4& v) { return v.y; }, A[1]);
          step([](const uint4& v) { return v.z; }, A[2]);
          step([](const uint4& v) { return v.w; }, A[3]);
        }
      }
      const float f = fr * *reinterpret_cast<const float*>(ring + cst * STB + 16 * c / SUB * SS + SUB * D);
      __syncwarp();
      next_stage();
      refill();
      // ---- softmax over this lane's tokens 16 c + 2 i + {0, 1} of row gi
      const int t0 = (int)(xt - cur.u0) * kTile + 16 * c;
      float p[8][2], mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float s = (sc[i][e] + sc[i][e + 2]) * f;
          p[i][e] = t0 + 2 * i + e < vis ? s : -INFINITY;
          mx = fmaxf(mx, p[i][e]);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
      const float alpha = ex2(m - mu);                 // m = -inf: 0
      m = mn;
      float ls = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          p[i][e] = ex2(p[i][e] - mu);
          ls += p[i][e];
        }
      l = l * alpha + ls;
      // ---- P V: p times its page's scale against the largest of those the row sees, split into two halves
      wait_stage();
      float sv = *reinterpret_cast<const float*>(ring + cst * STB + 16 * c / SUB * SS + SUB * D);
      if (NSUB > 1 && t0 >= vis) sv = 0.f;
      float st = sv;
      if constexpr (NSUB > 1) {
        st = fmaxf(st, __shfl_xor_sync(0xffffffffu, st, 1));
        st = fmaxf(st, __shfl_xor_sync(0xffffffffu, st, 2));
      }
      const float up = NSUB > 1 ? (st > 0.f ? __fdividef(sv, st) * kUp : 0.f) : kUp;
      uint32_t ph[8], pl[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v0 = p[i][0] * up, v1 = p[i][1] * up;
        const __half2 hi = __floats2half2_rn(v0, v1);
        const float2 back = __half22float2(hi);
        ph[i] = *reinterpret_cast<const uint32_t*>(&hi);
        pl[i] = pack_half(v0 - back.x, v1 - back.y);
      }
      const float so = st * (1.f / kUp);
      const unsigned char* vb = ring + cst * STB + 16 * c / SUB * SS + 16 * c % SUB + gi * SUB;
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += 4) {
        uint4 vw[4];
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vw[i] = *reinterpret_cast<const uint4*>(vb + (n0 + i) * 8 * SUB);
          acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        }
        auto step = [&](auto word, int j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            expand4<CODE>(word(vw[i]), b0, b1);
            hmma16816(acc[i], ph[j], pl[j], ph[j + 1], pl[j + 1], b0, b1);
          }
        };
        step([](const uint4& v) { return v.x; }, 0);
        step([](const uint4& v) { return v.y; }, 2);
        step([](const uint4& v) { return v.z; }, 4);
        step([](const uint4& v) { return v.w; }, 6);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[n0 + i][0] = fmaf(so, acc[i][0] + acc[i][2], o[n0 + i][0] * alpha);
          o[n0 + i][1] = fmaf(so, acc[i][1] + acc[i][3], o[n0 + i][1] * alpha);
        }
      }
      __syncwarp();
      next_stage();
      refill();
    }

    // ---- the warps' (m, l, o) into warp 0, in two rounds
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (c == 0) s_ml[warp][gi] = make_float2(m, l);
    __syncthreads();
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, s_ml[w][gi].x);
    const float Mu = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) L += s_ml[w][gi].y * ex2(s_ml[w][gi].x - Mu);
    const float mine = ex2(m - Mu);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      o[i][0] *= mine;
      o[i][1] *= mine;
    }
    // a lane's pairs, lane after lane: no bank conflicts
    float2* so2 = reinterpret_cast<float2*>(s_o);
    if (warp >= 2)
#pragma unroll
      for (int i = 0; i < NT; ++i) so2[((warp - 2) * NT + i) * 32 + lane] = make_float2(o[i][0], o[i][1]);
    __syncthreads();
    if (warp < 2)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float2 v = so2[(warp * NT + i) * 32 + lane];
        o[i][0] += v.x;
        o[i][1] += v.y;
      }
    __syncthreads();
    if (warp == 1)
#pragma unroll
      for (int i = 0; i < NT; ++i) so2[i * 32 + lane] = make_float2(o[i][0], o[i][1]);
    __syncthreads();
    const bool whole = x == cur.u0 && xe == ue;
    const int oq = by_g(cur.rg * kDecRows + gi);
    const int64_t otok = (int64_t)cur.s.q0 + oq;
    const int ohq = cur.h * G + cur.rg * kDecRows + gi - oq * G;
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float2 v = so2[i * 32 + lane];
        o[i][0] += v.x;
        o[i][1] += v.y;
      }
      if (whole) {
        if (gi < rows && otok >= 0 && otok < a.total_q &&
            TQ_CHECKED(static_cast<char*>(a.out) + (otok * a.Hq + ohq) * D * paged_esize(g.dtype), D * paged_esize(g.dtype), a.out,
                       a.total_q * a.Hq * D * paged_esize(g.dtype), 402)) {
          // only a row that sees nothing gives 0: a NaN in L, from a query that is not finite, is passed on
          const bool none = vis == 0;
          const float inv = 1.f / L;
          const int64_t at = (otok * a.Hq + ohq) * D;
          if (f32) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
              *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + 8 * i + 2 * c) =
                  none ? make_float2(0.f, 0.f) : make_float2(o[i][0] * inv, o[i][1] * inv);
          } else {
#pragma unroll
            for (int i = 0; i < NT; ++i)
              *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at + 8 * i + 2 * c) =
                  none ? 0u : pack2(o[i][0] * inv, o[i][1] * inv, f16);
          }
          if (a.lse && c == 0) a.lse[otok * a.Hq + ohq] = none ? -INFINITY : (M + log2f(L)) * (1.f / kLog2e);
        }
      } else {
        const int slot = 2 * cta + (x == cur.u0 ? 1 : 0);
        float* po = ws.o + ((int64_t)slot * kDecRows + gi) * D;
        if (TQ_CHECKED(po, 4 * D, a.ws, (int64_t)a.ws_bytes, 403))
#pragma unroll
        for (int i = 0; i < NT; ++i)
          *reinterpret_cast<float2*>(po + 8 * i + 2 * c) = make_float2(o[i][0], o[i][1]);
        if (c == 0) ws.ml[slot * kDecRows + gi] = make_float2(M, L);
      }
    }
    if (!whole) {
      // the CTA that finishes its part of the unit last joins the parts, in their order
      const int c0 = share_owner(W, C, cur.u0), c1 = share_owner(W, C, ue - 1);
      __syncthreads();
      if (tid == 0) s_last = last_part(&ws.count[c0], c1 - c0);
      __syncthreads();
      if (s_last) {
        // 16 threads per row, each D / 16 channels
        const int r = tid >> 4, k = tid & 15;
        constexpr int CH = D / 16;
        auto slot_of = [&](int p) { return p == c0 ? 2 * p + 1 : 2 * p; };
        float Ma = -INFINITY;
        for (int p = c0; p <= c1; ++p) Ma = fmaxf(Ma, __ldcg(&ws.ml[slot_of(p) * kDecRows + r]).x);
        const float Mb = Ma == -INFINITY ? 0.f : Ma;
        float La = 0.f, oo[CH];
#pragma unroll
        for (int q = 0; q < CH; ++q) oo[q] = 0.f;
        for (int p = c0; p <= c1; ++p) {
          const float2 v = __ldcg(&ws.ml[slot_of(p) * kDecRows + r]);
          const float wt = ex2(v.x - Mb);
          La += v.y * wt;
          const float4* src = reinterpret_cast<const float4*>(ws.o + ((int64_t)slot_of(p) * kDecRows + r) * D) + k;
#pragma unroll
          for (int q = 0; q < CH / 4; ++q) {
            const float4 t = __ldcg(src + 16 * q);
            oo[4 * q] = fmaf(t.x, wt, oo[4 * q]);
            oo[4 * q + 1] = fmaf(t.y, wt, oo[4 * q + 1]);
            oo[4 * q + 2] = fmaf(t.z, wt, oo[4 * q + 2]);
            oo[4 * q + 3] = fmaf(t.w, wt, oo[4 * q + 3]);
          }
        }
        const int row = cur.rg * kDecRows + r;
        const int64_t tok = (int64_t)cur.s.q0 + by_g(row);
        const int hq = cur.h * G + row - by_g(row) * G;
        if (r < rows && tok >= 0 && tok < a.total_q) {
          const bool none = s_vis[r] == 0;
          const float inv = 1.f / La;
          const int64_t at = (tok * a.Hq + hq) * D + 4 * k;
#pragma unroll
          for (int q = 0; q < CH; ++q) oo[q] = none ? 0.f : oo[q] * inv;
#pragma unroll
          for (int q = 0; q < CH; q += 4) {
            if (f32)
              *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + 16 * q) = make_float4(oo[q], oo[q + 1], oo[q + 2], oo[q + 3]);
            else
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at + 16 * q) =
                  make_uint2(pack2(oo[q], oo[q + 1], f16), pack2(oo[q + 2], oo[q + 3], f16));
          }
          if (a.lse && k == 0) a.lse[tok * a.Hq + hq] = none ? -INFINITY : (Ma + log2f(La)) * (1.f / kLog2e);
        }
      }
    }
    x = xe;
    if (x < x1) next_unit<kDecRows, kTile, 0>(g, a, G, cur);
  }
  if (*static_cast<volatile int*>(&s_abort)) {
    // a wait gave up: give the copies in flight a last chance to land before the shared memory goes
    const long long t0 = clock64();
    while (clock64() - t0 < (1ll << 28)) {
    }
  }
}

template <int D, int SUB, int CODE>
cudaError_t decode_t(const PGeom& g, const PagedAttn& a, cudaStream_t s) {
  constexpr size_t smem = dec_smem<D, SUB>();
  static_assert(smem <= (DecCfg<D>::kCtas == 1 ? 226u : 113u) * 1024, "resident CTAs");
  cudaError_t e = paged_allow_smem<k_paged_decode<D, SUB, CODE>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_decode<D, SUB, CODE>, dim3(148 * DecCfg<D>::kCtas), dim3(kDecThreads), smem, s, g, a);
}

template <int D, int SUB>
cudaError_t decode_c(const PGeom& g, const PagedAttn& a, cudaStream_t s) {
  return g.code == TQ_CODE_INT8 ? decode_t<D, SUB, TQ_CODE_INT8>(g, a, s) : decode_t<D, SUB, TQ_CODE_E4M3>(g, a, s);
}

template <int D>
cudaError_t decode_d(const PGeom& g, const PagedAttn& a, cudaStream_t s) {
  if (g.sub == 16) return decode_c<D, 16>(g, a, s);
  if (g.sub == 32) return decode_c<D, 32>(g, a, s);
  return decode_c<D, 64>(g, a, s);
}

}  // namespace

size_t paged_attn_ws_bytes(int d) {
  const size_t decode = kWsHeader + (size_t)2 * kMaxCtas * kDecRows * (8 + 4 * (size_t)d), chunk = paged_chunk_ws_bytes(d);
  return decode > chunk ? decode : chunk;
}
cudaError_t paged_lose_copies(int on) {
#ifdef TQ_DEBUG_BOUNDS
  return cudaMemcpyToSymbol(g_lose_copies, &on, sizeof(on));
#else
  return cudaErrorNotSupported;
#endif
}
cudaError_t paged_launch_ws_init(void* ws, cudaStream_t s) {
  return launch_pdl(k_paged_ws_init, dim3(1), dim3(256), 0, s, static_cast<uint32_t*>(ws));
}

cudaError_t paged_launch_attention(const PGeom& g, const PagedAttn& a, cudaStream_t s) {
  // Up to 24 query rows of a KV head the decode, which reads the codes once for every 8 rows, is the
  // faster; the chunk kernel's time does not depend on the rows up to 128.  Measured on 8 sequences, G = 4,
  // int8, decode / chunk in us:
  //                          16 rows     24 rows     32 rows
  //   d = 128, 32768 tokens  170 / 290   270 / 290   356 / 292        2000 tokens  26 / 39   31 / 38   37 / 38
  //   d = 64,  32768         115 / 243   167 / 243   218 / 241        2000         19 / 30   22 / 30   27 / 29
  //   d = 256, 32768         222 / 259   320 / 259   421 / 258        2000         32 / 45   36 / 45   45 / 45
  // (e4m3, d = 256 263 / 257 at 24 rows; G = 1, 8 as G = 4 at d = 128.)  One limit for all: away from d = 128
  // it is off by one group of 8 rows and costs 10 % (d = 64, 32 rows) to 24 % (d = 256, 24 rows) there.
  // fp32 stays with the decode, whose split halves keep its precision.
  if (a.max_q * (a.Hq / g.Hkv) > 24 && g.dtype != TQ_F32) return paged_launch_chunk(g, a, s);
  if (g.d == 64) return decode_d<64>(g, a, s);
  if (g.d == 128) return decode_d<128>(g, a, s);
  return decode_d<256>(g, a, s);
}

TQ_BOUNDS_READER(bounds_flag_paged_attn)

}  // namespace tq
