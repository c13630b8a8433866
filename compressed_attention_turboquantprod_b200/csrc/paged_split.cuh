// How a paged attention call is divided over CTAs, shared by its kernel files.
#pragma once

#include "mma_common.cuh"
#include "paged.cuh"

namespace tq {
namespace paged {
using namespace mmadec;

// A workspace begins with this word (tq_paged_workspace_init), so that one that was never made
// ready is reported instead of used; the counters behind it are zero between calls.
constexpr uint32_t kWsMagic = 0x70384b56u;
constexpr size_t kWsHeader = 4096;

// ---------------------------------------------------------------- the split over CTAs
// The work of a call is a list of tiles of T tokens, in the order (sequence, group of query
// rows, head, tile); a unit is one (sequence, group, head), at least one tile long so that a
// unit that sees nothing is also written.  Every CTA takes an equal, contiguous share of the
// list, whatever the lengths: a CTA's share may begin and end inside a unit, and then leaves a
// partial (m, l, o) for the CTA that finishes that unit last.  Lengths are read on the device,
// so a captured call follows them.
struct Seq {
  int slot, len, nq, q0;
};

__device__ __forceinline__ Seq load_seq(const PGeom& g, const PagedAttn& a, int i) {
  Seq s;
  s.slot = a.slots[i];
  s.q0 = a.cu[i];
  s.nq = min(max(a.cu[i + 1] - s.q0, 0), a.max_q);
  s.len = paged_len(g, s.slot);
  return s;
}

// Tokens that query j of the sequence sees.
__device__ __forceinline__ int visible(const Seq& s, int j, int causal) {
  return causal ? max(0, min(s.len, s.len - s.nq + j + 1)) : s.len;
}

// Row groups of R rows (row r: query r / G, head r mod G of the KV head) and their tiles.
template <int R>
__device__ __forceinline__ int seq_groups(const Seq& s, int G) {
  return (int)(((int64_t)s.nq * G + R - 1) / R);
}
template <int R>
__device__ __forceinline__ int group_visible(const Seq& s, int G, int rg, int causal) {
  return visible(s, (int)(min((int64_t)(rg + 1) * R, (int64_t)s.nq * G) - 1) / G, causal);
}
template <int R, int T>
__device__ __forceinline__ int group_tiles(const Seq& s, int G, int rg, int causal) {
  return max(1, (group_visible<R>(s, G, rg, causal) + T - 1) / T);
}

// Whether this thread of CTA 0 found a row with offsets that decrease or pass max_q or total_q.
__device__ __forceinline__ bool cta_first_checks(const PGeom& g, const PagedAttn& a) {
  bool bad = false;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
      const int b = a.cu[i], e = a.cu[i + 1];
      bad |= b < 0 || e < b || e > a.total_q || e - b > a.max_q;
    }
  return bad;
}

struct Cursor {      // a unit: its place in the list, and what it is
  int64_t u0;
  int nt, i, rg, h;
  Seq s;
};

// Tiles of sequence i, by one thread: a causal sequence's groups see one run of lengths.
template <int R, int T>
__device__ int64_t seq_tiles(const PGeom& g, const PagedAttn& a, int i, int G) {
  const Seq s = load_seq(g, a, i);
  const int ng = seq_groups<R>(s, G);
  if (ng == 0) return 0;
  if (!a.causal || s.nq == 1) return (int64_t)g.Hkv * ng * group_tiles<R, T>(s, G, 0, a.causal);
  int64_t t = 0;
  for (int rg = 0; rg < ng; ++rg) t += group_tiles<R, T>(s, G, rg, a.causal);
  return g.Hkv * t;
}

// All threads of the CTA (NT): the number of tiles of the call.
template <int R, int T, int NT>
__device__ int64_t count_tiles(const PGeom& g, const PagedAttn& a, int G, int64_t* s_sum) {
  int64_t t = 0;
  for (int i = threadIdx.x; i < a.n; i += NT) t += seq_tiles<R, T>(g, a, i, G);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = t;
  __syncthreads();
  t = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) t += s_sum[w];
  return t;
}

// One warp: the unit that holds tile x of the list.
template <int R, int T>
__device__ Cursor find_unit(const PGeom& g, const PagedAttn& a, int G, int64_t x) {
  const int lane = threadIdx.x & 31;
  int64_t base = 0;
  Cursor c{};
  int i = 0;
  for (int i0 = 0; i0 < a.n; i0 += 32) {
    const int64_t t = i0 + lane < a.n ? seq_tiles<R, T>(g, a, i0 + lane, G) : 0;
    int64_t v = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + v > x);
    if (hit) {
      const int l = __ffs(hit) - 1;
      base += __shfl_sync(0xffffffffu, v - t, l);
      i = i0 + l;
      break;
    }
    base += __shfl_sync(0xffffffffu, v, 31);
  }
  c.i = i;
  c.s = load_seq(g, a, i);
  const int ng = seq_groups<R>(c.s, G);
  for (int r0 = 0; r0 < ng; r0 += 32) {
    const int64_t t = r0 + lane < ng ? (int64_t)g.Hkv * group_tiles<R, T>(c.s, G, r0 + lane, a.causal) : 0;
    int64_t v = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + v > x);
    if (hit) {
      const int l = __ffs(hit) - 1;
      base += __shfl_sync(0xffffffffu, v - t, l);
      c.rg = r0 + l;
      break;
    }
    base += __shfl_sync(0xffffffffu, v, 31);
  }
  c.nt = group_tiles<R, T>(c.s, G, c.rg, a.causal);
  c.h = (int)((x - base) / c.nt);
  c.u0 = base + (int64_t)c.h * c.nt;
  return c;
}

// The next unit of the list (the caller knows that there is one).
template <int R, int T>
__device__ __forceinline__ void next_unit(const PGeom& g, const PagedAttn& a, int G, Cursor& c) {
  c.u0 += c.nt;
  if (++c.h < g.Hkv) return;
  c.h = 0;
  if (++c.rg >= seq_groups<R>(c.s, G)) {
    c.rg = 0;
    do {
      c.s = load_seq(g, a, ++c.i);
    } while (c.s.nq == 0 && c.i + 1 < a.n);
  }
  c.nt = group_tiles<R, T>(c.s, G, c.rg, a.causal);
}

// CTAs that take part in W tiles (at least `least` tiles each), the first tile of CTA c, and
// the CTA that holds tile x.
__device__ __forceinline__ int64_t share_ctas(int64_t W, int ctas, int least) {
  return max((int64_t)1, min((int64_t)ctas, (W + least - 1) / least));
}
__device__ __forceinline__ int64_t share_begin(int64_t W, int64_t C, int64_t c) { return W * c / C; }
__device__ __forceinline__ int share_owner(int64_t W, int64_t C, int64_t x) { return (int)(((x + 1) * C - 1) / W); }

// Wait on phase `parity` of an mbarrier for at most 2^31 cycles (about a second).
__device__ __forceinline__ bool mbar_wait_timed(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const long long t0 = clock64();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    if (ok) return true;
    if (clock64() - t0 > (1ll << 31)) return false;
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 4 stored bytes -> two f16 pairs, exact.  int8: byte u under 0x64 is the half 1024 + u.
template <int CODE>
__device__ __forceinline__ void expand4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (CODE == TQ_CODE_INT8) {
    const __half2 off = __half2half2(__ushort_as_half((unsigned short)0x6480));     // 1152
    const uint32_t a = prmt(w, 0x64646464u, 0x4140), b = prmt(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace paged
}  // namespace tq
