// Quantisation into the pages of the 8-bit cache, and reading them back.
//
// A block (the tokens of a page in one KV head; keys and values apart) has one scale, from
// the largest magnitude a over its finite entries:
//   int8   code = round-half-even(127 x / a), scale = a / 127 (IEEE fp32);
//   e4m3   scale = 2^k, the smallest with a / scale <= 448, code = e4m3(x / scale), exact
//          but for that one rounding.
// The partly filled last page of a sequence also keeps its tokens as they came (the tail), so
// its codes are always those of the exact tokens under the present a, however the tokens
// were split into appends.  When a new token does not raise a, only its own codes are
// written; when it does, the page's codes are formed again from the tail.
#include <cuda_fp8.h>

#include <type_traits>

#include "paged.cuh"

namespace tq {
namespace {

constexpr int kWThreads = 128;
// A block whose largest magnitude is below this is stored as zeros: 127 / a and 2^-k stay
// far from the ends of the fp32 range.
constexpr float kMinMax = 7.8886090522101181e-31f;   // 2^-100

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// |x| of a finite entry, 0 of an infinity or NaN: what a block's largest magnitude is
// taken over, so that one bad entry does not erase its block.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// The smallest 2^k with a / 2^k <= 448 = 0.875 * 2^9: with a = m 2^e, m in [0.5, 1),
// k = e - 9 when m <= 0.875, else e - 8.
__device__ __forceinline__ int e4m3_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 126;
  return (u & 0x7fffffu) <= 0x600000u ? e - 9 : e - 8;     // 0.875 = 0.5 * 1.75
}

struct BlockScale {
  float scale;      // what a code is multiplied by
  float inv;        // int8: fl32(127 / a); e4m3: 2^-k
  float a;
};

__device__ __forceinline__ BlockScale block_scale(float a, int code) {
  BlockScale b;
  b.a = a;
  if (a < kMinMax) {
    b.scale = 0.f;
    b.inv = 0.f;
  } else if (code == TQ_CODE_INT8) {
    b.scale = __fdiv_rn(a, 127.f);
    b.inv = __fdiv_rn(127.f, a);
  } else {
    const int k = e4m3_exponent(a);
    b.scale = __int_as_float((127 + k) << 23);
    b.inv = __int_as_float((127 - k) << 23);
  }
  return b;
}

// Stored byte of x, in full.  int8: inv is off by 2^-24 at most, so x * inv is within 127 * 2^-24 <
// 8e-6 of 127 x / a; next to a rounding border the exact products 127 x and (2 n + 1) a / 2 (at most 32 significant bits each) are
// compared in fp64, a tie going to the even code.  An infinity saturates, a NaN is 0.
template <int CODE>
__device__ __noinline__ uint32_t encode_slow(float x, float a, float inv) {
  if constexpr (CODE == TQ_CODE_INT8) {
    if (x != x || inv == 0.f) return 128u;
    if (!(fabsf(x) <= a)) return x > 0.f ? 255u : 1u;
    const double h = floor((double)(x * inv)) + 0.5;
    const double diff = 127.0 * (double)x - h * (double)a;
    const double lo = h - 0.5, even = ((int)lo & 1) == 0 ? lo : lo + 1.0;
    return (uint32_t)((int)(diff < 0.0 ? lo : diff > 0.0 ? lo + 1.0 : even) + 128);
  } else {
    return 0u;
  }
}

// Stored bytes of four entries.  int8: 1.5 * 2^23 added in one rounding leaves the nearest integer in
// the low bits; the remainder tells whether x is plain (finite and not next to a border).
template <int CODE>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], const BlockScale& b) {
  if constexpr (CODE == TQ_CODE_INT8) {
    uint32_t u[4];
    bool plain = true;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float m = fmaf(x[k], b.inv, 12582912.f);
      const float rest = fmaf(x[k], b.inv, 12582912.f - m);
      plain = plain && fabsf(rest) < 0.5f - 1e-5f;
      u[k] = __float_as_uint(m);
    }
    // bytes of the integers, + 128 each
    uint32_t w = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410) ^ 0x80808080u;
    if (!plain) {
      w = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float m = fmaf(x[k], b.inv, 12582912.f);
        const float rest = fmaf(x[k], b.inv, 12582912.f - m);
        w |= (fabsf(rest) < 0.5f - 1e-5f ? (__float_as_uint(m) + 128u) & 255u : encode_slow<CODE>(x[k], b.a, b.inv)) << (8 * k);
      }
    }
    return w;
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const float2 y = make_float2(x[k] == x[k] ? x[k] * b.inv : 0.f, x[k + 1] == x[k + 1] ? x[k + 1] * b.inv : 0.f);
      w |= (uint32_t)__nv_cvt_float2_to_fp8x2(b.inv == 0.f ? make_float2(0.f, 0.f) : y, __NV_SATFINITE, __NV_E4M3) << (8 * k);
    }
    return w;
  }
}

template <int CODE>
__device__ __forceinline__ float decode_byte(uint32_t u) {
  if constexpr (CODE == TQ_CODE_INT8) {
    return __uint_as_float(0x4b000000u | u) - 8388736.f;       // 2^23 + u, less 2^23 + 128
  } else {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)u, __NV_E4M3)));
  }
}

__device__ __forceinline__ float cta_max(float v, float* s) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = s[0];
#pragma unroll
  for (int i = 1; i < kWThreads / 32; ++i) r = fmaxf(r, s[i]);
  return r;
}

// A plan that the write cannot serve (it reaches past the input, or was made for more rows than this
// launch): its tokens are stored as zeros, so that nothing of a page's former owner is left in their places.
template <int D, int CODE>
__device__ __noinline__ void write_zeros(const PGeom& g, int layer, int h, int kv, int n_items, int n_rows) {
  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    int lo = 0, hi = n_rows;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g.rows[mid].item <= item) lo = mid; else hi = mid;
    }
    const PagedRow row = g.rows[lo];
    const int p = row.start / g.page + (item - row.item), t0 = p * g.page, end = row.start + row.count;
    const int n0 = max(row.start, t0) - t0, n1 = min(end, t0 + g.page) - t0;
    if (n1 <= n0) continue;
    const int pid = g.table[(int64_t)row.slot * g.max_pages + p];
    if (g.len[row.slot] != end) continue;                              // (freed since: its pages are not its own)
    if ((unsigned)pid >= (unsigned)g.pages) {
      if (threadIdx.x == 0) atomicOr(&g.state->status, kPagedBadPage);
      continue;
    }
    uint8_t* blk = paged_block(g, layer, pid, kv, h, 0);
    uint8_t* tail = paged_tail(g, layer, row.slot, kv, h);
    const int es = paged_esize(g.dtype);
    if (!TQ_CHECKED(blk, g.hb, g.base, g.total, 437) || !TQ_CHECKED(tail, g.tail_head, g.base, g.total, 438)) continue;
    for (int i = threadIdx.x; i < (n1 - n0) * D; i += kWThreads) {
      const int t = n0 + i / D, j = i % D, tb = t % g.sub;
      blk[(int64_t)(t / g.sub) * g.sb + (kv ? j * g.sub + tb : paged_k_off(D, tb, j))] = CODE == TQ_CODE_INT8 ? 128 : 0;
    }
    if (n0 == 0 && threadIdx.x < g.page / g.sub)
      *reinterpret_cast<float2*>(blk + (int64_t)threadIdx.x * g.sb + (int64_t)g.sub * D) = make_float2(0.f, 0.f);
    if (p == end / g.page)                                             // the page that stays open
      for (int i = threadIdx.x; i < (n1 - n0) * D * es / 4; i += kWThreads)
        reinterpret_cast<uint32_t*>(tail + (int64_t)n0 * D * es)[i] = 0;
  }
}

// One CTA per (page of the plan, head, K / V): the page's new tokens come once from the
// input into shared memory, where their largest magnitude is formed and from where they
// are encoded; codes leave as 16-byte words.  Measured: 32.8 k tokens of 8 heads, d = 128, bf16 to int8: 78 us
// for 201 MB (0.40 of the copy peak, 49 % issue at 9 CTAs an SM; 12 of them, with spills, took 86 us).
template <typename T, int D, int CODE>
__global__ void __launch_bounds__(kWThreads) k_paged_write(const __grid_constant__ PGeom g, int layer, const T* K, const T* V, int64_t k_stride,
                                                           int64_t v_stride, int64_t total, int max_rows) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float s_red[kWThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int item = blockIdx.x, h = blockIdx.y, kv = blockIdx.z;
  // the row whose items hold this one: up to 32 rows by one load each, more by bisection
  const int n_items = g.state->n_items, n_rows = g.state->n_rows, lane = tid & 31;
  PagedRow row = g.rows[lane < max_rows ? lane : 0];
  if (g.state->end > total || n_rows > max_rows) {
    if (tid == 0 && item < n_items) atomicOr(&g.state->status, kPagedBadOffsets);
    write_zeros<D, CODE>(g, layer, h, kv, n_items, n_rows);
    return;
  }
  if (item >= n_items) return;
  if (n_rows <= 32) {
    const unsigned below = __ballot_sync(0xffffffffu, lane < n_rows && row.item <= item);
    const int l = 31 - __clz(below);
    row.slot = __shfl_sync(0xffffffffu, row.slot, l);
    row.src = __shfl_sync(0xffffffffu, row.src, l);
    row.start = __shfl_sync(0xffffffffu, row.start, l);
    row.count = __shfl_sync(0xffffffffu, row.count, l);
    row.item = __shfl_sync(0xffffffffu, row.item, l);
  } else {
    int lo = 0, hi = n_rows;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g.rows[mid].item <= item) lo = mid; else hi = mid;
    }
    row = g.rows[lo];
  }
  const int p = row.start / g.page + (item - row.item);
  const int t0 = p * g.page;
  const int n0 = max(row.start, t0) - t0, n1 = min(row.start + row.count, t0 + g.page) - t0;
  if (n1 <= n0) return;
  const int pid = g.table[(int64_t)row.slot * g.max_pages + p];
  if (g.len[row.slot] != row.start + row.count) {   // freed since the plan: its pages may be another sequence's
    if (tid == 0) atomicOr(&g.state->status, kPagedBadSlot);
    return;
  }
  if ((unsigned)pid >= (unsigned)g.pages) {
    if (tid == 0) atomicOr(&g.state->status, kPagedBadPage);
    return;
  }
  const int64_t src0 = (int64_t)row.src + (t0 + n0 - row.start);    // input token of page token n0
  constexpr int CH = D * (int)sizeof(T) / 16;      // 16-byte pieces of a token
  constexpr int EP = 16 / (int)sizeof(T);
  T* S = reinterpret_cast<T*>(smem);               // [page][D]
  uint4* S4 = reinterpret_cast<uint4*>(smem);
  uint4* tail = reinterpret_cast<uint4*>(paged_tail(g, layer, row.slot, kv, h));
  const T* in = kv ? V : K;
  const int64_t stride = kv ? v_stride : k_stride;
  // The exact tokens of the page that stays open go to the tail.  When the row begins inside
  // an older open page, that page's CTA may read the tail, so it also writes it, afterwards.
  const int end = row.start + row.count, p_open = end / g.page;
  const bool old_first = row.start % g.page != 0 && p_open != row.start / g.page;
  const bool keep = p == p_open && !old_first;
  // The largest magnitude, as bits: entries without their sign compare as integers; one that is not
  // finite shows itself past the largest finite number, and only then are they sorted out.
  constexpr uint32_t kFinite = std::is_same_v<T, float> ? 0x7f7fffffu : std::is_same_v<T, __half> ? 0x7bffu : 0x7f7fu;
  auto bits = [&](uint32_t m, uint32_t u) {
    if constexpr (sizeof(T) == 4) return max(m, u & 0x7fffffffu);
    else return __vmaxu2(m, u & 0x7fff7fffu);
  };
  uint32_t m = 0;
#pragma unroll 4
  for (int i = tid; i < (n1 - n0) * CH; i += kWThreads) {
    const int t = i / CH, c = i % CH;
    const T* from = in + (src0 + t) * stride + (int64_t)h * D + c * EP;
    const uint4 v = TQ_CHECKED(from, 16, in, ((total - 1) * stride + (int64_t)g.Hkv * D) * (int64_t)sizeof(T), 431)
                        ? *reinterpret_cast<const uint4*>(from)
                        : make_uint4(0, 0, 0, 0);
    S4[(n0 + t) * CH + c] = v;
    if (keep && TQ_CHECKED(&tail[(n0 + t) * CH + c], 16, g.base, g.total, 432)) tail[(n0 + t) * CH + c] = v;
    m = bits(bits(bits(bits(m, v.x), v.y), v.z), v.w);
  }
  if constexpr (sizeof(T) == 2) m = max(m & 0xffffu, m >> 16);
  float a = 0.f;
  if (m <= kFinite) {
    if constexpr (sizeof(T) == 4) {
      a = __uint_as_float(m);
    } else {
      const uint16_t m16 = (uint16_t)m;
      a = to_f<T>(*reinterpret_cast<const T*>(&m16));
    }
  } else {
    for (int i = tid; i < (n1 - n0) * CH; i += kWThreads)
      for (int k = 0; k < EP; ++k) a = fmaxf(a, finite_abs(to_f<T>(S[(n0 * CH + i) * EP + k])));
  }
  a = cta_max(a, s_red);
  int first = n0;
  uint8_t* blk = paged_block(g, layer, pid, kv, h, 0);
  const int64_t cbytes = (int64_t)g.sub * D;
  if (n0 > 0) {
    const float old = reinterpret_cast<const float*>(blk + cbytes)[1];
    if (a > old) {
      first = 0;
      for (int i = tid; i < n0 * CH; i += kWThreads) S4[i] = tail[i];
    } else {
      a = old;
    }
  } else {
    first = 0;
  }
  __syncthreads();
  if (old_first && n0 > 0) {
    const int kept = end % g.page;
    for (int i = tid; i < kept * CH; i += kWThreads) {
      const int64_t t = (int64_t)row.src + row.count - kept + i / CH;
      tail[i] = *reinterpret_cast<const uint4*>(in + t * stride + (int64_t)h * D + (i % CH) * EP);
    }
  }
  const BlockScale b = block_scale(a, g.code);
  if (first == 0 && tid < g.page / g.sub) {
    float2* t = reinterpret_cast<float2*>(blk + (int64_t)tid * g.sb + cbytes);
    *t = make_float2(b.scale, b.a);
  }
  if (kv == 0) {
    constexpr int C16 = D / 16;
    for (int i = first * C16 + tid; i < n1 * C16; i += kWThreads) {
      const int t = i / C16, c = i % C16;
      T e[16];
#pragma unroll
      for (int k = 0; k < (int)sizeof(T); ++k) reinterpret_cast<uint4*>(e)[k] = S4[t * CH + c * (int)sizeof(T) + k];
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x[4] = {to_f<T>(e[4 * k]), to_f<T>(e[4 * k + 1]), to_f<T>(e[4 * k + 2]), to_f<T>(e[4 * k + 3])};
        w[k] = encode4<CODE>(x, b);
      }
      const int tb = t % g.sub;
      uint8_t* to = blk + (int64_t)(t / g.sub) * g.sb + paged_k_off(D, tb, c * 16);
      if (TQ_CHECKED(to, 16, g.base, g.total, 433)) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    // a lane takes 16 tokens of four neighbouring channels: four 16-byte stores
    struct alignas(4 * sizeof(T)) Four {
      T e[4];
    };
    const int g0 = first / 16, g1 = (n1 + 15) / 16;
    for (int i = tid; i < (g1 - g0) * (D / 4); i += kWThreads) {
      const int j = 4 * (i % (D / 4)), t16 = (g0 + i / (D / 4)) * 16;
      uint8_t* to = blk + (int64_t)(t16 / g.sub) * g.sb + (int64_t)j * g.sub + t16 % g.sub;
      if (!TQ_CHECKED(to, 3 * g.sub + 16, g.base, g.total, 434)) continue;
      if (t16 >= first && t16 + 16 <= n1) {
        uint32_t w[4][4];                          // [channel][four tokens]
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          Four f[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) f[q] = *reinterpret_cast<const Four*>(S + (t16 + 4 * k + q) * D + j);
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            const float x[4] = {to_f<T>(f[0].e[ch]), to_f<T>(f[1].e[ch]), to_f<T>(f[2].e[ch]), to_f<T>(f[3].e[ch])};
            w[ch][k] = encode4<CODE>(x, b);
          }
        }
#pragma unroll
        for (int ch = 0; ch < 4; ++ch)
          *reinterpret_cast<uint4*>(to + ch * g.sub) = make_uint4(w[ch][0], w[ch][1], w[ch][2], w[ch][3]);
      } else {
        // a group that this append fills in part: byte by byte
        for (int t = max(t16, first); t < min(t16 + 16, n1); ++t) {
          const Four f = *reinterpret_cast<const Four*>(S + t * D + j);
          const float x[4] = {to_f<T>(f.e[0]), to_f<T>(f.e[1]), to_f<T>(f.e[2]), to_f<T>(f.e[3])};
          const uint32_t w = encode4<CODE>(x, b);
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) to[ch * g.sub + t - t16] = (uint8_t)(w >> (8 * ch));
        }
      }
    }
  }
}

// The first cu[i + 1] - cu[i] tokens of slot slots[i] as floats (zeros past its length).
// One CTA per (up to 64 tokens of one sequence, head, K / V); no shared memory: a lane's 16 key codes
// are neighbours in the output already, and of values it takes 16 tokens of four neighbouring channels and
// turns them around in 4 x 4 bytes.  Measured: the same tokens 46 us (0.67 of the copy peak).
constexpr int kReadTokens = 64;
template <typename T, int D, int CODE>
__global__ void __launch_bounds__(kWThreads) k_paged_read(PGeom g, int layer, const int* slots, const int* cu, int n,
                                                          int64_t total, T* K, T* V) {
  constexpr int RT = kReadTokens;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int h = blockIdx.y, kv = blockIdx.z;
  if (blockIdx.x == 0 && h == 0 && kv == 0) {
    bool bad = false;
    for (int r = tid; r < n; r += kWThreads) bad |= cu[r] < 0 || cu[r + 1] < cu[r] || cu[r + 1] > total;
    if (bad) atomicOr(&g.state->status, kPagedBadOffsets);
  }
  // the sequence and tile of this CTA: rows in groups of 32, one per lane
  int item = blockIdx.x, i = -1;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int r = i0 + lane;
    const int c = r < n ? (max(0, cu[r + 1] - cu[r]) + RT - 1) / RT : 0;
    int v = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, item < v);
    if (hit) {
      const int l = __ffs(hit) - 1;
      item -= __shfl_sync(0xffffffffu, v - c, l);
      i = i0 + l;
      break;
    }
    item -= __shfl_sync(0xffffffffu, v, 31);
  }
  if (i < 0) return;
  const int slot = slots[i], c0 = cu[i], count = cu[i + 1] - c0;
  const int len = paged_len(g, slot);
  const int t0 = RT * item, nt = min(RT, count - t0);
  T* out = kv ? V : K;
  if (c0 < 0 || (int64_t)c0 + count > total) return;
  // four codes to four outputs
  struct alignas(4 * sizeof(T)) Four {
    T e[4];
  };
  auto four = [&](uint32_t w, float scale) {
    Four f;
#pragma unroll
    for (int k = 0; k < 4; ++k) f.e[k] = from_f<T>(decode_byte<CODE>((w >> (8 * k)) & 255u) * scale);
    return f;
  };
  auto page_of = [&](int t) {                        // -1: no such token
    return t < len ? g.table[(int64_t)slot * g.max_pages + t / g.page] : -1;
  };
  auto row = [&](int t) { return out + (((int64_t)c0 + t0 + t) * g.Hkv + h) * D; };
  if (kv == 0) {
    constexpr int C16 = D / 16;
    for (int k = tid; k < nt * C16; k += kWThreads) {
      const int t = k / C16, c = k % C16, pid = page_of(t0 + t);
      uint4 raw = make_uint4(0, 0, 0, 0);
      float scale = 0.f;
      if ((unsigned)pid < (unsigned)g.pages) {
        const int tp = (t0 + t) % g.page;
        const uint8_t* blk = paged_block(g, layer, pid, 0, h, tp / g.sub);
        scale = *reinterpret_cast<const float*>(blk + g.sub * D);
        if (TQ_CHECKED(blk, g.sb, g.base, g.total, 435))
          raw = *reinterpret_cast<const uint4*>(blk + paged_k_off(D, tp % g.sub, 16 * c));
      }
      Four* to = reinterpret_cast<Four*>(row(t) + 16 * c);
      if (!TQ_CHECKED(to, 4 * sizeof(Four), out, total * g.Hkv * D * (int64_t)sizeof(T), 436)) continue;
      to[0] = four(raw.x, scale);
      to[1] = four(raw.y, scale);
      to[2] = four(raw.z, scale);
      to[3] = four(raw.w, scale);
    }
  } else {
    for (int k = tid; k < (nt + 15) / 16 * (D / 4); k += kWThreads) {
      const int j = 4 * (k % (D / 4)), t = 16 * (k / (D / 4)), pid = page_of(t0 + t);
      uint4 raw[4] = {};
      float scale = 0.f;
      if ((unsigned)pid < (unsigned)g.pages) {
        const int tp = (t0 + t) % g.page;
        const uint8_t* blk = paged_block(g, layer, pid, 1, h, tp / g.sub);
        scale = *reinterpret_cast<const float*>(blk + g.sub * D);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) raw[ch] = *reinterpret_cast<const uint4*>(blk + (j + ch) * g.sub + tp % g.sub);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t a0 = reinterpret_cast<const uint32_t*>(&raw[0])[q], a1 = reinterpret_cast<const uint32_t*>(&raw[1])[q],
                       a2 = reinterpret_cast<const uint32_t*>(&raw[2])[q], a3 = reinterpret_cast<const uint32_t*>(&raw[3])[q];
        const uint32_t l01 = __byte_perm(a0, a1, 0x5140), l23 = __byte_perm(a2, a3, 0x5140),
                       h01 = __byte_perm(a0, a1, 0x7362), h23 = __byte_perm(a2, a3, 0x7362);
        const uint32_t w[4] = {__byte_perm(l01, l23, 0x5410), __byte_perm(l01, l23, 0x7632),
                               __byte_perm(h01, h23, 0x5410), __byte_perm(h01, h23, 0x7632)};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t + 4 * q + e < nt)
            *reinterpret_cast<Four*>(row(t + 4 * q + e) + j) = four(w[e], t0 + t + 4 * q + e < len ? scale : 0.f);
      }
    }
  }
}

template <typename T, int D, int CODE>
cudaError_t write_t(const PGeom& g, int layer, const void* K, const void* V, int64_t ks, int64_t vs, int64_t total,
                    int n_rows, cudaStream_t s) {
  const size_t smem = (size_t)g.page * D * sizeof(T);
  cudaError_t e = paged_allow_smem<k_paged_write<T, D, CODE>>((size_t)128 * D * sizeof(T));     // the largest page's
  if (e != cudaSuccess) return e;
  // a row of c tokens touches at most c / page + 2 pages
  const int64_t items = total / g.page + 2 * (int64_t)n_rows;
  return launch_pdl(k_paged_write<T, D, CODE>, dim3((unsigned)items, g.Hkv, 2), dim3(kWThreads), smem, s, g, layer,
                    static_cast<const T*>(K), static_cast<const T*>(V), ks, vs, total, n_rows);
}

template <typename T, int D, int CODE>
cudaError_t read_t(const PGeom& g, int layer, const int* slots, const int* cu, int n, int64_t total, void* K, void* V,
                   cudaStream_t s) {
  const int64_t items = total / kReadTokens + n;
  return launch_pdl(k_paged_read<T, D, CODE>, dim3((unsigned)items, g.Hkv, 2), dim3(kWThreads), 0, s, g, layer, slots,
                    cu, n, total, static_cast<T*>(K), static_cast<T*>(V));
}

template <typename F>
cudaError_t by_shape(const PGeom& g, F f) {
  auto by_code = [&](auto t, auto d) {
    return g.code == TQ_CODE_INT8 ? f(t, d, std::integral_constant<int, TQ_CODE_INT8>())
                                  : f(t, d, std::integral_constant<int, TQ_CODE_E4M3>());
  };
  auto by_d = [&](auto t) {
    if (g.d == 64) return by_code(t, std::integral_constant<int, 64>());
    if (g.d == 128) return by_code(t, std::integral_constant<int, 128>());
    return by_code(t, std::integral_constant<int, 256>());
  };
  if (g.dtype == TQ_F32) return by_d(float());
  if (g.dtype == TQ_F16) return by_d(__half());
  return by_d(__nv_bfloat16());
}

}  // namespace

cudaError_t paged_launch_write(const PGeom& g, int layer, const void* K, const void* V, int64_t k_stride,
                               int64_t v_stride, int64_t total, int n_rows, cudaStream_t s) {
  return by_shape(g, [&](auto t, auto d, auto c) {
    return write_t<decltype(t), decltype(d)::value, decltype(c)::value>(g, layer, K, V, k_stride, v_stride, total,
                                                                        n_rows, s);
  });
}

cudaError_t paged_launch_read(const PGeom& g, int layer, const int* slots, const int* cu, int n, int64_t total,
                              void* K, void* V, cudaStream_t s) {
  return by_shape(g, [&](auto t, auto d, auto c) {
    return read_t<decltype(t), decltype(d)::value, decltype(c)::value>(g, layer, slots, cu, n, total, K, V, s);
  });
}

TQ_BOUNDS_READER(bounds_flag_paged_quant)

}  // namespace tq
