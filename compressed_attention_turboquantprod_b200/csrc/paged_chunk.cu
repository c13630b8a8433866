// Attention of many query rows over the paged 8-bit cache (chunks, prompts, cross attention
// of bf16 / f16 models) on the fifth-generation tensor cores.
//
// A CTA works on R = 128 MT query rows of one KV head (row r: query r / G, head r mod G, so that
// grouped heads share every tile) and walks its share of their tiles of T tokens:
//   S_w = Q_w K^T       A = Q_w (128 x D, shared memory), B = K (T x D), fp32 in tensor memory
//   P_w = 2^(f S_w + log2 s_v - M)      a thread per row, f16 back into tensor memory over S_w (two S take turns)
//   O_w += P_w V        A = P_w (tensor memory), B = V (D x T, shared memory)
// A warpgroup per row block runs its softmax, four converter warps read the next tile's codes
// into registers while they expand the last one's into the f16 operands, three warps bring the next
// unit's queries, and one warp issues the products: Q K^T a tile ahead of P V, so that S of the next
// tile is there when a softmax has finished one.  The roles meet at mbarriers only: converters, queries
// and the first Q K^T run ahead into the next unit while the softmax warps write out the last.
//
// The scales enter exactly and at no cost per element: a page's key scale multiplies the row's
// factor f (one per 16 tokens), its value scale is added to the exponent, so that O sums code
// products only.  M is a running reference of f S + log2 s_v, raised only when a tile passes it by
// more than 2^4 (O is rescaled then); p is at most 2^15, and p <= 2^11 when M is fresh.  The
// weights' sum l, taken in fp32 before p is rounded to f16, is held against a reference R of f S alone:
// a weight is p 2^(M - R - 11 - log2 s_v), a factor per 16 tokens.  While the value scales in sight lie in
// 2^-60 .. 2^40 (every f16 scale does), M - R does too, and p and the factor stay in fp32's range.  Tiles
// with a scale outside, those behind them, and tiles with a block of zero values, which has no scale and
// must not enter M, take their weights from the logits instead.  Rounding p to f16 (2^-11 relative, as fine as the
// output's own rounding) is the one loss beside q's, which is held to 2^-11 of a f16 entry's own
// bits or exactly (bf16, f16 entries have at most 11 bits; q is scaled by a power of two per row).
//
// Measured (one B200, bf16 peak 1644 TFLOP/s): 64 queries on each of 8 x 32768 tokens, 32 / 8 heads, d =
// 128, int8: 350 us, 786 TFLOP/s; prompts of 8192 and 6001 tokens on themselves, e4m3: 1021 us, 827
// TFLOP/s.  A tile of 64 tokens takes about 2050 cycles on the prompts, whose codes come from L2, and about
// 2400 on the long caches, where its products need 1280 and its exponentials 1024.  The limit is the shared
// issue of 16 warps in four roles, each near its own serial time: leaving out the exponentials, the
// expansion, the products or the loads alone gained 2, 0, 10 and 7 %, all four together 43 % (before the
// folding of O and the reference R, which cost 3 and 2 %).  Tried in the states of the time: T = 128 with one S a row block took 3.0 ms on the prompts (each softmax waited for its own
// products), S single and P apart 1.06 ms, products from a branch of one thread 3.2 ms, two converters
// for the keys and two for the values 1.04 ms, requests into L2 four tiles ahead 1.03 ms.
#include "paged_split.cuh"
#include "tc_common.cuh"

namespace tq {
namespace {
using namespace paged;

constexpr int kChunkCtas = 148;
constexpr int kConv = 4;                   // converter warps
constexpr int kLoad = 3;                   // query warps
constexpr float kNone = -1e30f;            // reference of a row that has seen no token
constexpr float kBias = 11.f;              // p is held times 2^11
constexpr float kScaleLo = -60.f, kScaleHi = 40.f;    // log2 s_v of ordinary tiles
constexpr float kZeros = -3e38f;           // log2 s_v of a block of zeros: below any M, kNone too
constexpr float kSlack = 4.f;

constexpr int kTokens = 64;                // tokens of a tile
constexpr int kUnitCost = 8;               // places of a unit besides its tiles (16k cycles, 2k a tile)
// The tensor core's fp32 sums truncate: a row of O loses up to 2^-23 of itself, always towards zero, with
// every k-step of 16 tokens (measured 1e-7 a step: 0.7 % after 2^20 tokens).  So O is added, rounded to
// nearest, to a sum in the workspace and begun anew after this many tiles: 8192 tokens, 512 steps, 2^-14 at
// most, an eighth of what rounding p to f16 may cost.  64 queries on 8 x 32768 tokens (shares of 222 tiles):
// 342 us, without folding 344, folded after 64 tiles 366 (three folds in place of one).
constexpr int kFold = 128;
template <int D>
__host__ __device__ constexpr int chunk_max_mt() { return D == 256 ? 1 : 2; }
// Query operands: this unit's and the next one's, where they fit.
template <int D>
__host__ __device__ constexpr int chunk_q_bufs() { return D == 256 ? 1 : 2; }
template <int D, int MT>
__host__ __device__ constexpr size_t chunk_smem() {
  return 1024 + (size_t)chunk_q_bufs<D>() * MT * 128 * D * 2 + 4 * (size_t)kTokens * D * 2;
}

// Operands lie in shared memory K-major in the 128-byte swizzle: slabs of 64 f16 along K, a row
// of a slab 128 bytes, its 16-byte piece c at place c ^ (row mod 8); 8 rows are 1024 bytes.
// (The plain core-matrix layout took 190 cycles a 128 x 128 x 16 product here.)
// Byte offset of 16-byte piece c (along all of K) of `row` in an operand of ROWS rows.
template <int ROWS>
__device__ __forceinline__ int sw_off(int row, int c) {
  return (c >> 3) * (ROWS * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}
// Descriptor of such an operand at shared address `at` (1024-byte aligned), and what slab k adds to it
// (the start address is its low field, in units of 16 bytes; a k-step of 16 f16 adds 2).
__device__ __forceinline__ uint64_t sw_desc(uint32_t at) {
  return (uint64_t)((at >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
template <int ROWS>
__device__ __forceinline__ constexpr int sw_slab(int k) {
  return k * (ROWS * 8);
}

// The products' warp runs its loop with all lanes, so that descriptors and addresses stay in uniform
// registers (in a branch of one thread each product took 200 cycles to issue); one elected lane, always
// the same, issues them, four k-steps (one 128-byte slab of the operands) to an election.
// D[tmem] (+)= A[smem] * B[smem]^T over four k-steps, f16 operands.
__device__ __forceinline__ void mma4_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T over four k-steps (8 columns of A each).
__device__ __forceinline__ void mma4_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the mbarrier when every product issued so far has completed;
// mma_commit_and_arrive: the issuing lane arrives there itself, too.
__device__ __forceinline__ void mma_commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void mma_commit_and_arrive(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t"
      "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// *p += v, rounded to nearest, without waiting.
__device__ __forceinline__ void red_add4(float4* p, const float4& v) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

struct ChunkWs {
  int* count;          // [CTAs][2] finished parts of the unit that goes on after the CTA, per row block
  float* lse;          // [2 x CTAs][R] log2 of a part's weight sum (-inf: none)
  float* o;            // [2 x CTAs][D / 4][R][4] a part's output
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

template <int MT>
struct ChunkShared {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2], q_full[2], q_free[2], o_free[2];
  uint64_t s_full[2][2], p_ready[2][2], pv_done[2][2];      // [row block][tile mod 2]
  uint64_t done;                           // every product and arrival of the products' warp
  SplitPlan plan;
  float sk[4][4], lv[4][4];                // a tile's scales per 16 tokens: of the keys, log2 of the values' (or kZeros)
  float fr[2][128 * MT];                   // a row's factor on S, per query operand
  Cursor cur;
  uint32_t tmem;
  int abort, last[2];
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// 16 columns of this thread's lane, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Wait for the tensor-memory loads of this thread, tied to the registers they fill, so that no use
// of those is moved before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27])
               :
               : "memory");
  asm volatile("" : "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31]) : : "memory");
}

template <int D, int CODE, int MT>
__global__ void __launch_bounds__(128 * MT + 256, 1) k_paged_chunk(PGeom g, PagedAttn a) {
  constexpr int T = kTokens, R = 128 * MT, NTH = R + 256;
  constexpr int TW = T / kConv;                       // tokens of a tile a converter warp expands
  constexpr int NK = T * D / 16 / 128;                // 16-byte pieces of a tile's keys (values) per converter lane
  constexpr uint32_t kTb = T * D * 2;                 // bytes of an f16 operand tile
  constexpr uint32_t cO = 0, cS = MT * D;             // tensor memory columns
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ ChunkShared<MT> sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);       // known to be the same in all lanes
  const int wg = warp >> 2;                           // < MT: softmax of row block wg
  const bool is_soft = wg < MT, is_conv = wg == MT, is_mma = warp == 4 * MT + kConv;
  constexpr int NQ = chunk_q_bufs<D>();
  constexpr uint32_t kQb = R * D * 2;                 // bytes of a query operand
  const uint32_t sQ = smem_u32(smem), sK = sQ + NQ * kQb, sV = sK + 2 * kTb;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], kConv);
      mbar_init(&sh.k_free[i], 1);
      mbar_init(&sh.v_full[i], kConv);
      mbar_init(&sh.v_free[i], 1);
      mbar_init(&sh.q_full[i], kLoad);
      mbar_init(&sh.q_free[i], 4 * MT);
      mbar_init(&sh.o_free[i], 4);
      for (int w = 0; w < 2; ++w) {
        mbar_init(&sh.s_full[w][i], 2);       // the products, and the warp that saw the tile's scales
        mbar_init(&sh.p_ready[w][i], 4);
        mbar_init(&sh.pv_done[w][i], 1);
      }
    }
    mbar_init(&sh.done, 1);
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
  const int64_t W = count_places<R, T, kUnitCost, NTH>(g, a, G, sh.plan);
  if (W == 0) return;
  const int64_t C = share_ctas(W, gridDim.x, kUnitCost + 2);
  const int cta = blockIdx.x;
  if (cta >= C) return;
  const int64_t x0 = share_begin(W, C, cta), x1 = share_begin(W, C, cta + 1);
  if (warp == 0) {
    const Cursor f = find_unit<R, T, kUnitCost>(g, a, G, x0, sh.plan);
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
  auto wait = [&](uint64_t* bar, int index) {         // completion `index` (0, 1, ...) of a barrier
    if (!mbar_wait_timed(bar, (uint32_t)(index & 1), &sh.abort)) atomicOr(&g.state->status, kPagedWait);
  };
  // Each role walks the CTA's units by itself: f(tiles of the unit in this CTA's share, how many of
  // them are to be worked on (none in a unit that sees nothing), such tiles before, segments with such tiles before).
  auto walk = [&](auto f) {
    int64_t x = x0;
    int n0 = 0, seg = 0;
    while (x < x1) {
      const Segment<kUnitCost> sg(cur, x, x1);
      if (!sg.empty()) {
        const int nt = group_visible<R>(cur.s, G, cur.rg, a.causal) > 0 ? sg.last - sg.first : 0;
        f(sg, nt, n0, seg);
        n0 += nt;
        seg += nt > 0;
      }
      x = min(x1, cur.u0 + kUnitCost + cur.nt);
      if (x < x1) next_unit<R, T, kUnitCost>(g, a, G, cur);
    }
  };

  const DivG by_g(G);
  // Place of row i of the unit in an array of tokens `stride` entries apart (a token's heads lie side
  // by side), in entries; -1: none.
  auto place = [&](int i, int64_t stride) {
    const int row0 = cur.rg * R, q = by_g(row0 + i);
    const int64_t tok = (int64_t)cur.s.q0 + q;
    return row0 + i < cur.s.nq * G && i < R && tok >= 0 && tok < a.total_q
               ? tok * stride + (cur.h * G + row0 + i - q * G) * D
               : (int64_t)-1;
  };
  // rows of D / 8 16-byte pieces: RL lanes a row, RI rows an instruction
  constexpr int RL = D / 8, RI = 32 / RL;

  // The unit's rows into query operand qb, by warp w of nw: the largest entry of a row into [2^14,
  // 2^15) by a power of two; a negative scale turns the row's sign.
  const bool f16 = g.dtype == TQ_F16;
  auto bring_queries = [&](int qb, int w, int nw) {
    constexpr int BI = 8;                            // reads in flight (a store between them would hold them up)
    const int c = lane % RL;
#pragma unroll 1
    for (int i0 = w * BI; i0 < R / RI; i0 += nw * BI) {
      uint4 q[BI];
#pragma unroll
      for (int i = 0; i < BI; ++i) {
        const int64_t at = place((i0 + i) * RI + lane / RL, a.q_stride);
        q[i] = at >= 0 ? reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.Q) + at)[c] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < BI; ++i) {
        const int rr = (i0 + i) * RI + lane / RL;
        const uint32_t u[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
        // |entries| compare as integers in both types (a NaN or infinity spoils its own row only)
        uint32_t m2 = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) m2 = __vmaxu2(m2, u[k] & 0x7fff7fffu);
        uint32_t m1 = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
        for (int o = RL / 2; o > 0; o >>= 1) m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, o));
        const float mx = unpack2(m1, f16).x;
        const int e = min(mx > 0.f ? 141 - (int)(__float_as_uint(mx) >> 23) : 0, 120);
        const float up = copysignf(__int_as_float((127 + e) << 23), a.scale);
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = unpack2(u[k], f16);
          o[k] = pack_half(v.x * up, v.y * up);
        }
        *reinterpret_cast<uint4*>(smem + qb * kQb + (rr >> 7) * (128 * D * 2) + sw_off<128>(rr & 127, c)) =
            make_uint4(o[0], o[1], o[2], o[3]);
        if (c == 0) sh.fr[qb][rr] = fabsf(a.scale) * kLog2e * __int_as_float((127 - e) << 23);
      }
    }
  };

  if (is_conv) {
    // =================================================================== converters
    // Warp cw expands tokens 16 cw ... of the tile, which lie in one sub-block.  A warp instruction takes 8
    // rows of 4 pieces (keys) or a piece of 32 channels (values), so that its 16-byte stores hit all banks;
    // rows are 128 bytes of the swizzled operand.
    const int cw = warp & 3, l7 = lane & 7, l3 = lane >> 3, par = lane & 1;
    const int lsub = 31 - __clz(g.sub), lpage = 31 - __clz(g.page);
    const int64_t vofs = (int64_t)g.Hkv * g.hb;
    const int ko[2] = {D == 64 ? l7 * D + 16 * l3 : l7 * D + 16 * l3 + 64 * par,
                       D == 64 ? 0 : l7 * D + 16 * l3 + 64 * (1 - par)};
    const int vch = lane, pc = 2 * cw;                // the first channel of this lane's value pieces, their piece along T
    const int kd0 = (cw * TW + l7) * 128 + (((2 * l3) ^ l7) << 4), kd1 = (cw * TW + l7) * 128 + (((2 * l3 + 1) ^ l7) << 4);
    const int vd0 = sw_off<D>(vch, pc), vd1 = sw_off<D>(vch, pc + 1);
    auto put = [&](unsigned char* to, unsigned char* to2, const uint4& v) {        // 16 codes -> two pieces of a row
      uint32_t o[8];
      expand4<CODE>(v.x, o[0], o[1]);
      expand4<CODE>(v.y, o[2], o[3]);
      expand4<CODE>(v.z, o[4], o[5]);
      expand4<CODE>(v.w, o[6], o[7]);
      *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(to2) = make_uint4(o[4], o[5], o[6], o[7]);
    };
    walk([&](const auto& sg, int nt, int n0, int) {
      if (nt == 0) return;
      const int tok0 = sg.first * T + cw * TW, last = cur.s.len - 1;
      const int* table = g.table + (int64_t)cur.s.slot * g.max_pages;
      uint4 kr[NK], vr[NK];
      int pid, off;                                   // page of the warp's tokens and their offset in it, a tile ahead
      const uint8_t* kp = nullptr;                    // their key sub-block
      const uint8_t* heads = g.pool + (int64_t)a.layer * g.pages * g.page_bytes + (int64_t)cur.h * g.hb;
      float sk = 0.f, sv = 0.f;
      auto look = [&](int t) {
        // past the end: the last sub-block's, masked but finite
        const int tk = min(tok0 + t * T, last & ~15);
        pid = table[tk >> lpage];
        off = tk & (g.page - 1);
      };
      auto load_k = [&]() {
        if ((unsigned)pid >= (unsigned)g.pages) {
          if (lane == 0) atomicOr(&g.state->status, kPagedBadPage);
          pid = 0;
        }
        kp = heads + pid * g.page_bytes + (off >> lsub) * g.sb;
        off &= g.sub - 1;
        const uint8_t* p0 = kp + off * D;
#pragma unroll
        for (int it = 0; it < NK; ++it) {
          const int cg = it % (D / 64), rg = it / (D / 64);          // 64-byte group, 8-row group
          const uint8_t* p = p0 + ko[cg & 1] + (cg >> 1) * 128 + rg * 8 * D;
          kr[it] = TQ_CHECKED(p, 16, g.base, g.total, 421) ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
        }
        const uint8_t* tr = kp + (D << lsub);
        sk = *reinterpret_cast<const float*>(tr);
        sv = *reinterpret_cast<const float*>(tr + vofs);
      };
      auto load_v = [&]() {
        const uint8_t* p = kp + off + vofs + (vch << lsub);
#pragma unroll
        for (int it = 0; it < NK; ++it) {
          const uint8_t* q = p + ((it * 32) << lsub);
          vr[it] = TQ_CHECKED(q, 16, g.base, g.total, 422) ? *reinterpret_cast<const uint4*>(q) : make_uint4(0, 0, 0, 0);
        }
      };
      look(0);
      load_k();
      load_v();
      if (nt > 1) look(1);
      for (int t = 0; t < nt; ++t) {
        const int n = n0 + t, b2 = n & 1;
        unsigned char* K = smem + NQ * kQb + b2 * kTb;
        unsigned char* V = K + 2 * kTb;
        if (n >= 2) wait(&sh.k_free[b2], (n >> 1) - 1);
        // four sets of scales: the products of tile n - 2 are done, so the softmax of tile n - 4 is
        if (lane == 0) {
          sh.sk[n & 3][cw] = sk;
          sh.lv[n & 3][cw] = sv > 0.f ? __log2f(sv) : kZeros;
        }
#pragma unroll
        for (int it = 0; it < NK; ++it) {
          unsigned char* to = K + (it % (D / 64)) * (T * 128) + (it / (D / 64)) * 1024;
          put(to + kd0, to + kd1, kr[it]);
        }
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.k_full[b2]);
        // the next tile's pages were looked up a tile ago; its keys travel while the values expand
        if (t + 1 < nt) load_k();
        if (n >= 2) wait(&sh.v_free[b2], (n >> 1) - 1);
#pragma unroll
        for (int it = 0; it < NK; ++it) put(V + vd0 + it * 32 * 128, V + vd1 + it * 32 * 128, vr[it]);
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.v_full[b2]);
        if (t + 1 < nt) load_v();
        if (t + 2 < nt) look(t + 2);
      }
    });
  } else if (is_mma) {
    // =================================================================== products
    constexpr uint32_t iS = tc::idesc_f16(128, T), iO = tc::idesc_f16(128, D);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dQ = sw_desc(__shfl_sync(0xffffffffu, sQ, 0)), dK = sw_desc(__shfl_sync(0xffffffffu, sK, 0)),
                   dV = sw_desc(__shfl_sync(0xffffffffu, sV, 0));
    auto qk = [&](int w, int b2, int qb) {
#pragma unroll
      for (int k = 0; k < D / 64; ++k)
        mma4_ss(tm + cS + (2 * w + b2) * T, dQ + (uint64_t)(qb * (kQb / 16) + w * (128 * D * 2 / 16) + sw_slab<128>(k)),
                dK + (uint64_t)(b2 * (kTb / 16) + sw_slab<T>(k)), iS, k > 0);
    };
    auto pv = [&](int w, int b2, bool first) {
      mma4_ts(tm + cO + w * D, tm + cS + (2 * w + b2) * T, dV + (uint64_t)(b2 * (kTb / 16)), iO, !first);
    };
    walk([&](const auto&, int nt_, int n0_, int seg_) {
      const int nt = __shfl_sync(0xffffffffu, nt_, 0), n0 = __shfl_sync(0xffffffffu, n0_, 0),
                seg = __shfl_sync(0xffffffffu, seg_, 0);
      // Q K^T of tile n + 1, then P V of tile n: the tensor cores have work while the softmax of n runs
      for (int t = -1; t < nt; ++t) {
        const int n = n0 + t, m = n + 1;
        if (t + 1 < nt) {
          if (t < 0) wait(&sh.q_full[seg % NQ], seg / NQ);
          wait(&sh.k_full[m & 1], m >> 1);
#pragma unroll
          for (int w = 0; w < MT; ++w) {
            // P of tile n - 1, over this S buffer, has been used (in the first tiles of a unit, too)
            if (n >= 1) wait(&sh.pv_done[w][m & 1], (n - 1) >> 1);
            tc::fence_after_sync();
            qk(w, m & 1, seg % NQ);
            mma_commit_and_arrive(&sh.s_full[w][m & 1]);
          }
          mma_commit_elected(&sh.k_free[m & 1]);
        }
        if (t >= 0) {
          wait(&sh.v_full[n & 1], n >> 1);
#pragma unroll
          for (int w = 0; w < MT; ++w) {
            wait(&sh.p_ready[w][n & 1], n >> 1);
            if (t == 0 && seg > 0) wait(&sh.o_free[w], seg - 1);      // the last unit's O has been read
            tc::fence_after_sync();
            pv(w, n & 1, t % kFold == 0);
            mma_commit_elected(&sh.pv_done[w][n & 1]);
          }
          mma_commit_elected(&sh.v_free[n & 1]);
        }
      }
    });
    // Nobody waits for the last k_free and v_free, nor, once a wait has given up, for the products: none
    // may be on its way when the tensor and shared memory go.
    mma_commit_elected(&sh.done);
    for (const long long t0 = clock64(); !mbar_try(&sh.done, 0);)
      if (clock64() - t0 > kWaitCycles) {
        atomicOr(&g.state->status, kPagedWait);
        break;
      }
  } else if (is_soft) {
    // =================================================================== softmax
    const uint32_t lrow = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tO = tmem + lrow + cO + wg * D;
    const int w4 = warp & 3, r = tid;                  // this thread's row of the CTA's
    const ChunkWs ws = chunk_ws<D, MT>(a.ws);
    walk([&](const auto& sg, int nt, int n0, int seg) {
      const int tok0 = sg.first * T;                   // the segment's first token
      const int row0 = cur.rg * R;                     // the CTA's first row of the sequence (below 2^27)
      const bool ok = place(r, 0) >= 0;
      const int vis = ok ? visible(cur.s, by_g(row0 + r), a.causal) : 0;
      float fr = 0.f, M = kNone, l = 0.f, Rw = kNone;
      bool far = false;                                // a scale has been out of range in this segment
      // The sum that O is folded into, for the reference Mf: the row's place in the segment's part.  (A unit
      // that this CTA holds alone uses the part of the unit that goes on after it, which is written last.)
      const int slot = 2 * cta + (sg.first == 0 ? 1 : 0);
      float4* part = reinterpret_cast<float4*>(ws.o + (int64_t)slot * R * D) + r;      // [D / 4][R]
      float Mf = kNone;
      auto folded = [&](int i, float w) {              // channels 4 i ... of that sum, times w
        const float4* from = &part[(int64_t)i * R];
        const float4 v = TQ_CHECKED(from, 16, a.ws, (int64_t)a.ws_bytes, 425) ? __ldcg(from) : make_float4(0.f, 0.f, 0.f, 0.f);
        return make_float4(v.x * w, v.y * w, v.z * w, v.w * w);
      };
      unsigned char* Q = smem + (seg % NQ) * kQb + (size_t)wg * 128 * D * 2;  // the row block's operand, later its output
      if (nt > 0) {
        if (seg == 0) {
          bring_queries(0, warp, 4 * MT);
          tc::fence_async_shared();
          tc::bar_sync(3, 128 * MT);
          if (lane == 0 && warp < kLoad) mbar_arrive(&sh.q_full[0]);
        }
        wait(&sh.q_full[seg % NQ], seg / NQ);
        fr = ok ? sh.fr[seg % NQ][r] : 0.f;
      }
      // A parity tells a completion only from its neighbours, so every waiter has to be within one of
      // it: S of tile n came after P V of n - 2 only, hence a barrier per buffer.
      auto pv_wait = [&](int n) { wait(&sh.pv_done[wg][n & 1], n >> 1); };
      // the rows of the warp see at least wmin tokens
      const int wmin = __reduce_min_sync(0xffffffffu, vis);
      // S of the next tile is requested as the registers of this one's halves come free, and P is
      // handed over when the next tile's work has begun: neither latency is waited for
      uint32_t v[2][32];                               // the row of S
      auto s_at = [&](int n) { return tmem + lrow + cS + (2 * wg + (n & 1)) * T; };
      auto hand_over = [&](int n) {                    // P of tile n is in place
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        // (a warp may finish tile n + 1 before another has finished n, but not n + 2)
        if (lane == 0) mbar_arrive(&sh.p_ready[wg][n & 1]);
      };
      if (nt > 0) {
        wait(&sh.s_full[wg][n0 & 1], n0 >> 1);
        tc::fence_after_sync();
        tc::tmem_ld32(s_at(n0), v[0]);
        tc::tmem_ld32(s_at(n0) + 32, v[1]);
      }
      for (int t = 0; t < nt; ++t) {
        const int n = n0 + t, sc = n & 3;
        const uint32_t tS = s_at(n);
        const int base = tok0 + t * T;                 // the tile's first token
        tmem_wait_ld(v[0]);
        tmem_wait_ld(v[1]);
        if (t > 0) hand_over(n - 1);
        if (base + T > wmin) {                         // a tile that not every row of the warp sees in full
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (base + 32 * c + i >= vis) v[c][i] = 0xff800000u;
        }
        float f[T / 16], lv[T / 16], zmax = -INFINITY;  // the largest exponent f S + log2 s_v
#pragma unroll
        for (int h = 0; h < T / 16; ++h) {
          f[h] = fr * sh.sk[sc][h];
          lv[h] = sh.lv[sc][h];
          auto S = [&](int i) { return __uint_as_float(v[h >> 1][16 * (h & 1) + i]); };
          const float m = max3(max3(max3(S(0), S(1), S(2)), max3(S(3), S(4), S(5)), max3(S(6), S(7), S(8))),
                               max3(max3(S(9), S(10), S(11)), S(12), S(13)), fmaxf(S(14), S(15)));
          zmax = fmaxf(zmax, fmaf(m, f[h], lv[h]));    // (nothing visible and f = 0: NaN, which fmaxf drops)
        }
        const float top = fmaxf(fmaxf(lv[0], lv[1]), fmaxf(lv[2], lv[3]));
        const bool odd = far || top > kScaleHi || fminf(fminf(lv[0], lv[1]), fminf(lv[2], lv[3])) < kScaleLo;
        if (t > 0 && t % kFold == 0) {                 // (P V of this tile begins O anew)
          pv_wait(n - 1);
          tc::fence_after_sync();
          // the first O as it is; later ones added where they lie (nothing is waited for), unless a
          // row's reference has moved on since
          const int how = t == kFold ? 0 : __all_sync(0xffffffffu, Mf == M) ? 1 : 2;
          const float w = ex2(Mf - M);
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(tO + 16 * c, o);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float4* to = &part[(int64_t)(4 * c + k) * R];
              if (!TQ_CHECKED(to, 16, a.ws, (int64_t)a.ws_bytes, 426)) continue;
              float4 v = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                     __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
              if (how == 1) {
                red_add4(to, v);
                continue;
              }
              if (how == 2) {
                const float4 u = __ldcg(to);
                v = make_float4(fmaf(u.x, w, v.x), fmaf(u.y, w, v.y), fmaf(u.z, w, v.z), fmaf(u.w, w, v.w));
              }
              *to = v;
            }
          }
          Mf = M;
        }
        const bool raise = __any_sync(0xffffffffu, zmax > M + kSlack);
        float e0 = M - Rw - kBias;                     // p to weight: 2^(e0 - log2 s_v)
        if (raise || odd) {
          if (raise) {
            // each row by itself: what it gives must not depend on the rows that share its warp
            const float Mn = zmax > M + kSlack ? zmax : M;
            const float alpha = ex2(M - Mn);           // (M = kNone: 0, or 1 of nothing)
            M = Mn;
            // R never passes the largest f S: that of M's token is at least M less the tile's largest scale
            const float Rn = alpha == 1.f ? Rw : fmaxf(Rw, M - top);
            l *= ex2(Rw - Rn);
            Rw = Rn;
            if (t % kFold != 0) {
              pv_wait(n - 1);
              tc::fence_after_sync();
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(tO + 16 * c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st16(tO + 16 * c, o);
              }
            }
            e0 = M - Rw - kBias;
          }
          if (odd) {
#pragma unroll
            for (int h = 0; h < T / 16; ++h) far = far || lv[h] > kScaleHi || (lv[h] < kScaleLo && lv[h] != kZeros);
            // rare, so in little code: S once more from tensor memory, 16 tokens at a time
#pragma unroll 1
            for (int h = 0; h < T / 16; ++h) {
              uint32_t u[16];
              tmem_ld16(tS + 16 * h, u);
              const float ff = fr * sh.sk[sc][h];
              float x[16], hi = Rw;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                x[i] = base + 16 * h + i < vis ? __uint_as_float(u[i]) * ff : -INFINITY;
                hi = fmaxf(hi, x[i]);
              }
              l *= ex2(Rw - hi);
              Rw = hi;
#pragma unroll
              for (int i = 0; i < 16; ++i) l += ex2(x[i] - Rw);
            }
            e0 = -INFINITY;                            // they are counted
          }
        }
        // p and its sum.  A masked S is -inf: its product with f = 0 (an unused row, a block of
        // zeros) would be NaN, so such a row's f counts as the smallest factor instead
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = 2 * c + e;
            const float ff = fmaxf(f[h], 1.1754944e-38f), cst = lv[h] - M + kBias;
            const float2 f2 = make_float2(ff, ff), c2 = make_float2(cst, cst);
            float2 ls = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 z = fma2(make_float2(__uint_as_float(v[c][16 * e + 2 * i]), __uint_as_float(v[c][16 * e + 2 * i + 1])), f2, c2);
              const float2 p = make_float2(ex2(z.x), ex2(z.y));
              ls = add2(ls, p);
              pk[8 * e + i] = pack_half(p.x, p.y);
            }
            l = fmaf(ls.x + ls.y, ex2(e0 - lv[h]), l);
          }
          tmem_st16(tS + 16 * c, pk);
          if (t + 1 < nt) {
            if (c == 0) {
              wait(&sh.s_full[wg][(n + 1) & 1], (n + 1) >> 1);
              tc::fence_after_sync();
            }
            tc::tmem_ld32(s_at(n + 1) + 32 * c, v[c]);
          }
        }
      }
      if (nt > 0) hand_over(n0 + nt - 1);
      // ---- the row's output, or its part
      const bool whole = sg.whole(cur);
      // Only a row that sees nothing (of a part: whose weights are all 0) gives 0: a NaN in l, from a query
      // that is not finite, is passed on.
      const bool none = whole ? vis == 0 : l == 0.f;
      const float inv = 1.f / l, up = ex2(M - Rw - kBias);
      const float lse2 = none ? -INFINITY : log2f(l) + Rw;
      const int64_t lse_at = ((int64_t)cur.s.q0 + by_g(row0 + r)) * a.Hq + cur.h * G + row0 + r - by_g(row0 + r) * G;
      if (nt > 0) {
        pv_wait(n0 + nt - 1);                          // (and so the row block's products with Q are done)
        tc::fence_after_sync();
      }
      // the warp's rows from the operand's place to the output, whole rows at a time
      auto rows_out = [&]() {
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < 32 / RI; ++i) {
          const int rr = 32 * w4 + i * RI + lane / RL, c = lane % RL;
          const int64_t at = place(128 * wg + rr, (int64_t)a.Hq * D);
          const uint4 v = nt > 0 ? *reinterpret_cast<const uint4*>(Q + sw_off<128>(rr, c)) : make_uint4(0, 0, 0, 0);
          if (at >= 0 && TQ_CHECKED(static_cast<uint16_t*>(a.out) + at, 2 * D, a.out, a.total_q * a.Hq * D * 2, 423))
            reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at)[c] = v;
        }
        __syncwarp();
      };
      const float wf = ex2(Mf - M);
#pragma unroll 1
      for (int c = 0; c < D / 32 && nt > 0; ++c) {
        uint32_t v[32];
        tc::tmem_ld32(tO + 32 * c, v);
        tmem_wait_ld(v);
        if (nt > kFold)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 s = folded(8 * c + i, wf);
            v[4 * i] = __float_as_uint(__uint_as_float(v[4 * i]) + s.x);
            v[4 * i + 1] = __float_as_uint(__uint_as_float(v[4 * i + 1]) + s.y);
            v[4 * i + 2] = __float_as_uint(__uint_as_float(v[4 * i + 2]) + s.z);
            v[4 * i + 3] = __float_as_uint(__uint_as_float(v[4 * i + 3]) + s.w);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = none ? 0.f : __uint_as_float(v[8 * i + k]) * inv * up;
          if (whole) {
            *reinterpret_cast<uint4*>(Q + sw_off<128>(r & 127, 4 * c + i)) =
                make_uint4(pack2(o[0], o[1], f16), pack2(o[2], o[3], f16), pack2(o[4], o[5], f16), pack2(o[6], o[7], f16));
          } else if (TQ_CHECKED(&part[(int64_t)(8 * c + 2 * i + 1) * R], 16, a.ws, (int64_t)a.ws_bytes, 424)) {
            part[(int64_t)(8 * c + 2 * i) * R] = make_float4(o[0], o[1], o[2], o[3]);
            part[(int64_t)(8 * c + 2 * i + 1) * R] = make_float4(o[4], o[5], o[6], o[7]);
          }
        }
      }
      if (nt > 0) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.o_free[wg]);
      }
      if (whole) {
        rows_out();
        if (ok && a.lse) a.lse[lse_at] = lse2 * (1.f / kLog2e);
      } else {
        ws.lse[slot * R + r] = lse2;
        // the CTA that finishes its part of the unit last joins the parts, in their order
        const int c0 = share_owner(W, C, cur.u0 + kUnitCost), c1 = share_owner(W, C, cur.u0 + kUnitCost + cur.nt - 1);
        tc::bar_sync(1 + wg, 128);
        if ((r & 127) == 0) sh.last[wg] = last_part(&ws.count[2 * c0 + wg], c1 - c0);
        tc::bar_sync(1 + wg, 128);
        if (sh.last[wg]) {
          auto slot_of = [&](int p) { return p == c0 ? 2 * p + 1 : 2 * p; };
          float m = -INFINITY, L = 0.f;
          for (int p = c0; p <= c1; ++p) m = fmaxf(m, __ldcg(&ws.lse[slot_of(p) * R + r]));
          const float mu = m == -INFINITY ? 0.f : m;
          for (int p = c0; p <= c1; ++p) L += ex2(__ldcg(&ws.lse[slot_of(p) * R + r]) - mu);
          const float iL = vis == 0 ? 0.f : 1.f / L;
          // 32 channels at a time: eight reads in flight per part
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float4 o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int p = c0; p <= c1; ++p) {
              const float4* src = reinterpret_cast<const float4*>(ws.o + (int64_t)slot_of(p) * R * D) + (int64_t)(8 * c) * R + r;
              float4 u[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) u[k] = __ldcg(src + (int64_t)k * R);
              const float w = ex2(__ldcg(&ws.lse[slot_of(p) * R + r]) - mu) * iL;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                o[k].x = fmaf(u[k].x, w, o[k].x);
                o[k].y = fmaf(u[k].y, w, o[k].y);
                o[k].z = fmaf(u[k].z, w, o[k].z);
                o[k].w = fmaf(u[k].w, w, o[k].w);
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(Q + sw_off<128>(r & 127, 4 * c + k)) =
                  make_uint4(pack2(o[2 * k].x, o[2 * k].y, f16), pack2(o[2 * k].z, o[2 * k].w, f16),
                             pack2(o[2 * k + 1].x, o[2 * k + 1].y, f16), pack2(o[2 * k + 1].z, o[2 * k + 1].w, f16));
          }
          rows_out();
          if (ok && a.lse)
            a.lse[lse_at] =
                vis == 0 ? -INFINITY : (m + log2f(L)) * (1.f / kLog2e);
        }
      }
      if (nt > 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_free[seg % NQ]);
      }
    });
  } else {
    // =================================================================== queries
    // the first unit's come from the softmax warps, which would only wait for them
    const int lw = warp - (4 * MT + kConv + 1);
    walk([&](const auto&, int nt, int, int seg) {
      if (nt == 0 || seg == 0) return;
      const int qb = seg % NQ;
      if (seg >= NQ) wait(&sh.q_free[qb], seg / NQ - 1);
      bring_queries(qb, lw, kLoad);
      tc::fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[qb]);
    });
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
  cudaError_t e = paged_allow_smem<k_paged_chunk<D, CODE, MT>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_chunk<D, CODE, MT>, dim3(kChunkCtas), dim3(128 * MT + 256), smem, s, g, a);
}

template <int D>
cudaError_t chunk_d(const PGeom& g, const PagedAttn& a, cudaStream_t s) {
  const bool i8 = g.code == TQ_CODE_INT8;
  if constexpr (chunk_max_mt<D>() == 2) {
    // one row block where no sequence has more rows than it holds.  Measured with one block and with two, in
    // us, for 128 and 256 rows of a head: 8 x 32768 tokens, 8 heads, int8, d = 128 284 / 332 and 567 / 346, d =
    // 64 236 / 278 and 464 / 259; 8 x 1200 tokens, 16 heads, d = 64 30 / 39 and 45 / 39
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
