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

// Stored byte of x.  int8: x * inv is within 127 * 2^-22.9 < 2e-5 of 127 x / a; where that
// is next to a rounding border the exact products 127 x and (2 n + 1) a / 2 (at most 32
// significant bits each) are compared in fp64, a tie going to the even code.
template <int CODE>
__device__ __forceinline__ uint32_t encode(float x, const BlockScale& b) {
  if constexpr (CODE == TQ_CODE_INT8) {
    if (!(fabsf(x) <= b.a)) {                        // an infinity saturates, NaN is 0
      return x != x || b.inv == 0.f ? 128u : x > 0.f ? 255u : 1u;
    }
    const float t = x * b.inv;
    float r = rintf(t);
    if (fabsf(fabsf(t - r) - 0.5f) < 4e-5f) {
      const double h = floor((double)t) + 0.5;
      const double diff = 127.0 * (double)x - h * (double)b.a;
      const double lo = h - 0.5;
      const double even = fmod(lo, 2.0) == 0.0 ? lo : lo + 1.0;
      r = b.inv == 0.f ? 0.f : (float)(diff < 0.0 ? lo : diff > 0.0 ? lo + 1.0 : even);
    }
    return (uint32_t)((int)r + 128);
  } else {
    if (x != x || b.inv == 0.f) return 0u;
    return (uint32_t)__nv_cvt_float_to_fp8(x * b.inv, __NV_SATFINITE, __NV_E4M3);
  }
}

template <int CODE>
__device__ __forceinline__ float decode_byte(uint32_t u) {
  if constexpr (CODE == TQ_CODE_INT8) {
    return (float)((int)u - 128);
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

// One CTA per (page of the plan, head, K / V): the page's new tokens come once from the
// input into shared memory, where their largest magnitude is formed and from where they
// are encoded; codes leave as 16-byte words.
template <typename T, int D, int CODE>
__global__ void __launch_bounds__(kWThreads) k_paged_write(PGeom g, int layer, const T* K, const T* V, int64_t k_stride,
                                                           int64_t v_stride, int64_t total) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float s_red[kWThreads / 32];
  pdl_wait();
  const int tid = threadIdx.x;
  const int item = blockIdx.x, h = blockIdx.y, kv = blockIdx.z;
  const PagedState* st = g.state;
  if (item >= st->n_items) return;
  int lo = 0, hi = st->n_rows;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.rows[mid].item <= item) lo = mid; else hi = mid;
  }
  const PagedRow row = g.rows[lo];
  const int p = row.start / g.page + (item - row.item);
  const int t0 = p * g.page;
  const int n0 = max(row.start, t0) - t0, n1 = min(row.start + row.count, t0 + g.page) - t0;
  if (n1 <= n0) return;
  const int pid = g.table[(int64_t)row.slot * g.max_pages + p];
  if ((unsigned)pid >= (unsigned)g.pages) {
    if (tid == 0) atomicOr(&g.state->status, kPagedBadPage);
    return;
  }
  const int64_t src0 = (int64_t)row.src + (t0 + n0 - row.start);    // input token of page token n0
  if (src0 + (n1 - n0) > total) {                                    // offsets past the arrays
    if (tid == 0) atomicOr(&g.state->status, kPagedBadOffsets);
    return;
  }
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
  auto amax4 = [](uint4 v) {
    const T* e = reinterpret_cast<const T*>(&v);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < EP; ++i) m = fmaxf(m, finite_abs(to_f<T>(e[i])));
    return m;
  };
  float a = 0.f;
#pragma unroll 4
  for (int i = tid; i < (n1 - n0) * CH; i += kWThreads) {
    const int t = i / CH, c = i % CH;
    const uint4 v = *reinterpret_cast<const uint4*>(in + (src0 + t) * stride + (int64_t)h * D + c * EP);
    S4[(n0 + t) * CH + c] = v;
    if (keep) tail[(n0 + t) * CH + c] = v;
    a = fmaxf(a, amax4(v));
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
      if (t < total) tail[i] = *reinterpret_cast<const uint4*>(in + t * stride + (int64_t)h * D + (i % CH) * EP);
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
      uint32_t w[4];
      const T* e = S + t * D + c * 16;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = encode<CODE>(to_f<T>(e[4 * k]), b) | encode<CODE>(to_f<T>(e[4 * k + 1]), b) << 8 |
               encode<CODE>(to_f<T>(e[4 * k + 2]), b) << 16 | encode<CODE>(to_f<T>(e[4 * k + 3]), b) << 24;
      const int tb = t % g.sub;
      *reinterpret_cast<uint4*>(blk + (int64_t)(t / g.sub) * g.sb + paged_k_off(D, tb, c * 16)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    // lanes take neighbouring channels; 16 tokens of a channel are one 16-byte store
    const int g0 = first / 16, g1 = (n1 + 15) / 16;
    for (int i = tid; i < (g1 - g0) * D; i += kWThreads) {
      const int j = i % D, t16 = (g0 + i / D) * 16;
      uint8_t* to = blk + (int64_t)(t16 / g.sub) * g.sb + (int64_t)j * g.sub + t16 % g.sub;
      if (t16 >= first && t16 + 16 <= n1) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k] = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) w[k] |= encode<CODE>(to_f<T>(S[(t16 + 4 * k + q) * D + j]), b) << (8 * q);
        }
        *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        for (int t = max(t16, first); t < min(t16 + 16, n1); ++t)
          to[t - t16] = (uint8_t)encode<CODE>(to_f<T>(S[t * D + j]), b);
      }
    }
  }
}

// The first cu[i + 1] - cu[i] tokens of slot slots[i] as floats (zeros past its length).
// One CTA per (up to read_tokens tokens of one sequence, head, K / V).
template <typename T, int D>
constexpr int read_tokens() { return D * sizeof(T) >= 1024 ? 32 : 64; }     // static shared memory
template <typename T, int D, int CODE>
__global__ void __launch_bounds__(kWThreads) k_paged_read(PGeom g, int layer, const int* slots, const int* cu, int n,
                                                          int64_t total, T* K, T* V) {
  constexpr int RT = read_tokens<T, D>();
  __shared__ __align__(16) T s_t[RT * (D + 8)];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int h = blockIdx.y, kv = blockIdx.z;
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
  if (c0 < 0 || (int64_t)c0 + count > total) {
    if (tid == 0) atomicOr(&g.state->status, kPagedBadOffsets);
    return;
  }
  // groups of 16 tokens lie in one sub-block; thread = (group, 16-byte piece)
  for (int k = tid; k < RT / 16 * D; k += kWThreads) {
    const int grp = k / D, x = k % D;
    const int t = t0 + 16 * grp;
    if (16 * grp >= nt) continue;
    uint4 raw = make_uint4(0, 0, 0, 0);
    float scale = 0.f;
    const int pid = t < len ? g.table[(int64_t)slot * g.max_pages + t / g.page] : -1;
    const int tb = t % g.page % g.sub;
    if ((unsigned)pid < (unsigned)g.pages) {
      const uint8_t* blk = paged_block(g, layer, pid, kv, h, t % g.page / g.sub);
      scale = *reinterpret_cast<const float*>(blk + (int64_t)g.sub * D);
      // keys: token tb + x / (D / 16), channels 16 (x mod D / 16)...; values: channel x, 16 tokens
      const int64_t off = kv ? (int64_t)x * g.sub + tb : paged_k_off(D, tb + x / (D / 16), 16 * (x % (D / 16)));
      raw = *reinterpret_cast<const uint4*>(blk + off);
    }
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int tok = kv ? 16 * grp + e : 16 * grp + x / (D / 16);
      const int ch = kv ? x : 16 * (x % (D / 16)) + e;
      const float v = decode_byte<CODE>((w[e >> 2] >> (8 * (e & 3))) & 255u) * scale;
      s_t[tok * (D + 8) + ch] = from_f<T>(t0 + tok < len ? v : 0.f);
    }
  }
  __syncthreads();
  constexpr int CH = D * (int)sizeof(T) / 16;
  constexpr int EP = 16 / (int)sizeof(T);
  for (int k = tid; k < nt * CH; k += kWThreads) {
    const int t = k / CH, c = k % CH;
    *reinterpret_cast<uint4*>(out + (((int64_t)c0 + t0 + t) * g.Hkv + h) * D + c * EP) =
        *reinterpret_cast<const uint4*>(&s_t[t * (D + 8) + c * EP]);
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
                    static_cast<const T*>(K), static_cast<const T*>(V), ks, vs, total);
}

template <typename T, int D, int CODE>
cudaError_t read_t(const PGeom& g, int layer, const int* slots, const int* cu, int n, int64_t total, void* K, void* V,
                   cudaStream_t s) {
  const int64_t items = total / read_tokens<T, D>() + n;
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
