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
// The work of a call is a list of places, in the order (sequence, group of query rows, head); a
// unit is one (sequence, group, head) and has KO + nt places, nt its tiles of T tokens (at least one, so
// that a unit that sees nothing is also written).  The KO places before a unit's tiles stand for
// what a unit costs besides them (queries in, output out), in tiles.  Every CTA takes an equal, contiguous
// share of the list, whatever the lengths: a share may begin and end inside a unit, and then leaves
// a partial output for the CTA that finishes that unit last.  Lengths are read on the device, so a
// captured call follows them.
// row / G for row < 2^27 and G <= 8: the reciprocal's error times row stays below 1 / G.
struct DivG {
  int G;
  uint32_t m;
  __device__ __forceinline__ explicit DivG(int g) : G(g), m((uint32_t)(0x100000000ull / (uint32_t)g) + 1u) {}
  __device__ __forceinline__ int operator()(int row) const { return G == 1 ? row : (int)__umulhi((uint32_t)row, m); }
};

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

struct Cursor {      // a unit: its first place in the list, its tiles, and what it is
  int64_t u0;
  int nt, i, rg, h;
  Seq s;
};

// Places of one head of sequence i: by one thread, or by a whole warp (every lane gets the sum).
template <int R, int T, int KO>
__device__ __forceinline__ int64_t head_places(const PGeom& g, const PagedAttn& a, int i, int G) {
  const Seq s = load_seq(g, a, i);
  const int ng = seq_groups<R>(s, G);
  if (ng == 0) return 0;
  if (ng == 1 || !a.causal) return (int64_t)ng * (KO + group_tiles<R, T>(s, G, 0, a.causal));
  int64_t t = 0;
  for (int rg = 0; rg < ng; ++rg) t += KO + group_tiles<R, T>(s, G, rg, a.causal);
  return t;
}
template <int R, int T, int KO>
__device__ __forceinline__ int64_t head_places_warp(const PGeom& g, const PagedAttn& a, int i, int G) {
  const Seq s = load_seq(g, a, i);
  const int ng = seq_groups<R>(s, G);
  if (ng == 0) return 0;
  if (!a.causal) return (int64_t)ng * (KO + group_tiles<R, T>(s, G, 0, a.causal));
  int64_t t = 0;
  for (int rg = threadIdx.x & 31; rg < ng; rg += 32) t += KO + group_tiles<R, T>(s, G, rg, a.causal);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// Shared memory of the plan: the sequences' places, when there are at most kPlanSeqs of them.
constexpr int kPlanSeqs = 128;
struct SplitPlan {
  int64_t sum[16];
  int64_t places[kPlanSeqs];
};

// All threads of the CTA (NT): the places of the call.
template <int R, int T, int KO, int NT>
__device__ int64_t count_places(const PGeom& g, const PagedAttn& a, int G, SplitPlan& sp) {
  int64_t t = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int64_t)a.max_q * G > R) {               // several groups: a warp per sequence
    for (int i = warp; i < a.n; i += NT / 32) {
      const int64_t v = g.Hkv * head_places_warp<R, T, KO>(g, a, i, G);
      if (lane == 0) {
        t += v;
        if (i < kPlanSeqs) sp.places[i] = v;
      }
    }
  } else {
    for (int i = threadIdx.x; i < a.n; i += NT) {
      const int64_t v = g.Hkv * head_places<R, T, KO>(g, a, i, G);
      t += v;
      if (i < kPlanSeqs) sp.places[i] = v;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) sp.sum[warp] = t;
  __syncthreads();
  t = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) t += sp.sum[w];
  return t;
}

// Over 32 values, one per lane: the lane whose running sum (from `base`) first passes x, and the
// sum before it in `base`; -1: none, all of them are in `base`.
__device__ __forceinline__ int find_lane(int64_t t, int64_t& base, int64_t x) {
  const int lane = threadIdx.x & 31;
  int64_t v = t;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  const unsigned hit = __ballot_sync(0xffffffffu, base + v > x);
  const int l = hit ? __ffs(hit) - 1 : 31;
  base += __shfl_sync(0xffffffffu, hit ? v - t : v, l);
  return hit ? l : -1;
}

// One warp, after count_places: the unit that holds place x of the list.
template <int R, int T, int KO>
__device__ Cursor find_unit(const PGeom& g, const PagedAttn& a, int G, int64_t x, const SplitPlan& sp) {
  const int lane = threadIdx.x & 31;
  int64_t base = 0;
  Cursor c{};
  for (int i0 = 0; i0 < a.n; i0 += 32) {
    const int i = i0 + lane;
    const int64_t t = i >= a.n ? 0 : i < kPlanSeqs ? sp.places[i] : g.Hkv * head_places<R, T, KO>(g, a, i, G);
    const int l = find_lane(t, base, x);
    if (l >= 0) {
      c.i = i0 + l;
      break;
    }
  }
  c.s = load_seq(g, a, c.i);
  const int ng = seq_groups<R>(c.s, G);
  for (int r0 = 0; r0 < ng; r0 += 32) {
    const int rg = r0 + lane;
    const int64_t t = rg < ng ? (int64_t)g.Hkv * (KO + group_tiles<R, T>(c.s, G, rg, a.causal)) : 0;
    const int l = find_lane(t, base, x);
    if (l >= 0) {
      c.rg = r0 + l;
      break;
    }
  }
  c.nt = group_tiles<R, T>(c.s, G, c.rg, a.causal);
  c.h = (int)((x - base) / (KO + c.nt));
  c.u0 = base + (int64_t)c.h * (KO + c.nt);
  return c;
}

// Both at once for at most 32 sequences, by every warp for itself (one round of loads, no barrier):
// the call's places, then, for the place that `at` makes of them, its unit (`at` < 0: none is sought).
template <int R, int T, int KO, typename F>
__device__ __forceinline__ int64_t plan_in_warp(const PGeom& g, const PagedAttn& a, int G, Cursor& c, F at) {
  const int lane = threadIdx.x & 31;
  Seq s{-1, 0, 0, 0};
  int64_t t = 0;
  if (lane < a.n) {
    s = load_seq(g, a, lane);
    const int ng = seq_groups<R>(s, G);
    if (ng == 1 || (ng > 1 && !a.causal)) {
      t = (int64_t)ng * (KO + group_tiles<R, T>(s, G, 0, a.causal));
    } else {
      for (int rg = 0; rg < ng; ++rg) t += KO + group_tiles<R, T>(s, G, rg, a.causal);
    }
    t *= g.Hkv;
  }
  int64_t W = t;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
  const int64_t x = W > 0 ? at(W) : (int64_t)-1;
  if (x < 0) return W;
  int64_t base = 0;
  c.i = max(find_lane(t, base, x), 0);
  c.s.slot = __shfl_sync(0xffffffffu, s.slot, c.i);
  c.s.len = __shfl_sync(0xffffffffu, s.len, c.i);
  c.s.nq = __shfl_sync(0xffffffffu, s.nq, c.i);
  c.s.q0 = __shfl_sync(0xffffffffu, s.q0, c.i);
  c.rg = 0;
  const int ng = seq_groups<R>(c.s, G);
  for (int r0 = 0; r0 < ng; r0 += 32) {
    const int rg = r0 + lane;
    const int64_t u = rg < ng ? (int64_t)g.Hkv * (KO + group_tiles<R, T>(c.s, G, rg, a.causal)) : 0;
    const int l = find_lane(u, base, x);
    if (l >= 0) {
      c.rg = r0 + l;
      break;
    }
  }
  c.nt = group_tiles<R, T>(c.s, G, c.rg, a.causal);
  c.h = (int)((x - base) / (KO + c.nt));
  c.u0 = base + (int64_t)c.h * (KO + c.nt);
  return W;
}

// The next unit of the list (the caller knows that there is one).
template <int R, int T, int KO>
__device__ __forceinline__ void next_unit(const PGeom& g, const PagedAttn& a, int G, Cursor& c) {
  c.u0 += KO + c.nt;
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

// The tiles [first, last) of a unit in a share [x0, x1) of the list, and the CTAs that hold its tiles.
template <int KO>
struct Segment {
  int first, last;
  __device__ __forceinline__ Segment(const Cursor& c, int64_t x0, int64_t x1) {
    first = (int)max((int64_t)0, x0 - c.u0 - KO);
    last = (int)max((int64_t)0, min(x1 - c.u0, (int64_t)KO + c.nt) - KO);
  }
  __device__ __forceinline__ bool empty() const { return last <= first; }
  __device__ __forceinline__ bool whole(const Cursor& c) const { return first == 0 && last == c.nt; }
};

// CTAs that take part in W places (at least `least` each), the first place of CTA c, and the CTA
// that holds place x.
__device__ __forceinline__ int64_t share_ctas(int64_t W, int ctas, int least) {
  return max((int64_t)1, min((int64_t)ctas, (W + least - 1) / least));
}
__device__ __forceinline__ int64_t share_begin(int64_t W, int64_t C, int64_t c) { return W * c / C; }
__device__ __forceinline__ int share_owner(int64_t W, int64_t C, int64_t x) { return (int)(((x + 1) * C - 1) / W); }

// One thread, after a barrier of the threads that wrote a part of a unit in `others` + 1 parts: whether
// this was the last to be written.  The release and acquire at device scope carry the other threads'
// writes with them; the counter wraps to 0 for the next call.
__device__ __forceinline__ bool last_part(int* count, int others) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(count), "r"((uint32_t)others) : "memory");
  return old == (uint32_t)others;
}

// Whether phase `parity` of an mbarrier is complete (the thread may sleep a little for it).
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Wait on phase `parity` for at most `cycles`; once a wait of the CTA has given up (*abort), none waits
// any more.  False: the phase is not complete.
constexpr long long kWaitCycles = 1ll << 31;           // about a second
__device__ __forceinline__ bool mbar_wait_slow(uint64_t* bar, uint32_t parity, int* abort, long long cycles) {
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (*static_cast<volatile int*>(abort)) return false;
    if (clock64() - t0 > cycles) {
      *static_cast<volatile int*>(abort) = 1;
      return false;
    }
  }
  return true;
}
// The same with the usual case, a completed phase, inline (a clock read costs more than the test).
__device__ __forceinline__ bool mbar_wait_timed(uint64_t* bar, uint32_t parity, int* abort, long long cycles = kWaitCycles) {
  return mbar_try(bar, parity) || mbar_wait_slow(bar, parity, abort, cycles);
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

// Two entries of a model type as floats, and back.
__device__ __forceinline__ float2 unpack2(uint32_t u, bool f16) {
  return f16 ? __half22float2(*reinterpret_cast<const __half2*>(&u))
             : make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, bool f16) {
  if (f16) return pack_half(a, b);
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace paged
}  // namespace tq
