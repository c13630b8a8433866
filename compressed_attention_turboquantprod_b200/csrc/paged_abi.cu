// C ABI of the paged 8-bit cache: layout, host checks, dispatch.  Every host check runs
// before any launch.
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "paged.cuh"

namespace {

using tq::set_error;

#define TQ_FAULT_POINT(name) \
  do {                       \
    if (tq::fault_injected(name)) return set_error(TQ_ERR_CUDA, "injected fault"); \
  } while (0)

int cuda_fail(cudaError_t e, const char* where) {
  return set_error(TQ_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

// A CUDA error left pending by earlier asynchronous work.
int check_pending(const char* where) {
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, where);
}

int done(cudaError_t e, const char* where) { return e == cudaSuccess ? tq::clear_error() : cuda_fail(e, where); }

// Whether two arrays share bytes.
struct Extent {
  const void* p;
  int64_t bytes;
};
bool meet(const Extent& a, const Extent& b) {
  const char *x = static_cast<const char*>(a.p), *y = static_cast<const char*>(b.p);
  return x && y && x < y + b.bytes && y < x + a.bytes;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int layout_status(const tq_paged_desc* d, tq_paged* out) {
  if (!d) return set_error(TQ_ERR_INVALID_ARG, "null descriptor");
  if (d->layers < 1 || d->layers > 1024 || d->Hkv < 1 || d->Hkv > 1024 || d->pages < 1 || d->pages > (1 << 20) ||
      d->slots < 1 || d->slots > 65536 || d->max_pages < 1)
    return set_error(TQ_ERR_INVALID_ARG, "bad descriptor (layers=%d Hkv=%d pages=%d slots=%d max_pages=%d)", d->layers,
                     d->Hkv, d->pages, d->slots, d->max_pages);
  if (d->dtype != TQ_F32 && d->dtype != TQ_F16 && d->dtype != TQ_BF16)
    return set_error(TQ_ERR_INVALID_ARG, "bad dtype %d", d->dtype);
  if (d->d != 64 && d->d != 128 && d->d != 256)
    return set_error(TQ_ERR_UNSUPPORTED, "head dim d=%d not in {64,128,256}", d->d);
  if (d->page != 16 && d->page != 32 && d->page != 64 && d->page != 128)
    return set_error(TQ_ERR_UNSUPPORTED, "page=%d not in {16,32,64,128}", d->page);
  if (d->code != TQ_CODE_INT8 && d->code != TQ_CODE_E4M3)
    return set_error(TQ_ERR_UNSUPPORTED, "code=%d is neither int8 nor e4m3", d->code);
  if ((int64_t)d->max_pages * d->page > (1 << 30))
    return set_error(TQ_ERR_UNSUPPORTED, "max_pages * page = %lld tokens, more than 2^30",
                     (long long)d->max_pages * d->page);
  tq_paged c;
  std::memset(&c, 0, sizeof(c));
  c.desc = *d;
  const int64_t sub = d->page < 64 ? d->page : 64;
  c.sub_bytes = sub * d->d + tq::kPagedTrailer;
  c.block_bytes = d->page / sub * c.sub_bytes;
  c.page_bytes = 2 * (int64_t)d->Hkv * c.block_bytes;
  int64_t o = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  c.o_state = take(sizeof(tq::PagedState));
  c.o_len = take(4 * (int64_t)d->slots);
  c.o_table = take(4 * (int64_t)d->slots * d->max_pages);
  c.o_ref = take(4 * (int64_t)d->pages);
  c.o_claim = take(4 * (int64_t)d->slots);
  c.o_rows = take((int64_t)sizeof(tq::PagedRow) * d->slots);
  c.o_scan = take(4 * ((int64_t)d->slots + 1));
  c.o_moves = take(8 * (int64_t)d->pages);
  c.o_remap = take(4 * (int64_t)d->pages);
  c.o_tail = take((int64_t)d->layers * d->slots * 2 * d->Hkv * d->page * d->d * tq::paged_esize(d->dtype));
  c.o_pool = take((int64_t)d->layers * d->pages * c.page_bytes);
  c.bytes = (size_t)o;
  if (out) *out = c;
  return TQ_OK;
}

int check(const tq_paged* c, const char* name) {
  if (!c || !c->base) return set_error(TQ_ERR_INVALID_ARG, "%s: null cache or cache without memory", name);
  tq_paged ref;
  const int st = layout_status(&c->desc, &ref);
  if (st != TQ_OK) return st;
  if (ref.o_pool != c->o_pool || ref.o_tail != c->o_tail || ref.page_bytes != c->page_bytes || c->bytes < ref.bytes)
    return set_error(TQ_ERR_INVALID_ARG, "%s: cache struct does not match its descriptor (not initialised?)", name);
  return TQ_OK;
}

int check_layer(const tq_paged* c, int layer, const char* name) {
  const int st = check(c, name);
  if (st != TQ_OK) return st;
  if (layer < 0 || layer >= c->desc.layers)
    return set_error(TQ_ERR_INVALID_ARG, "%s: layer=%d of %d", name, layer, c->desc.layers);
  return TQ_OK;
}

// A device int32 array of n >= 1 entries.
int check_ints(const void* a, const void* b, int n, int most, const char* name) {
  if (!a || !b || !aligned(a, 4) || !aligned(b, 4))
    return set_error(TQ_ERR_INVALID_ARG, "%s: null or misaligned index array", name);
  if (n < 1 || n > most) return set_error(TQ_ERR_INVALID_ARG, "%s: n=%d not in 1..%d", name, n, most);
  return TQ_OK;
}

tq::PGeom geom(const tq_paged* c) {
  tq::PGeom g;
  const tq_paged_desc& d = c->desc;
  g.layers = d.layers;
  g.Hkv = d.Hkv;
  g.d = d.d;
  g.page = d.page;
  g.sub = d.page < 64 ? d.page : 64;
  g.pages = d.pages;
  g.slots = d.slots;
  g.max_pages = d.max_pages;
  g.dtype = d.dtype;
  g.code = d.code;
  g.sb = c->sub_bytes;
  g.hb = c->block_bytes;
  g.page_bytes = c->page_bytes;
  g.tail_head = (int64_t)d.page * d.d * tq::paged_esize(d.dtype);
  g.base = static_cast<uint8_t*>(c->base);
  g.total = (int64_t)c->bytes;
  g.pool = g.base + c->o_pool;
  g.tail = g.base + c->o_tail;
  g.state = reinterpret_cast<tq::PagedState*>(g.base + c->o_state);
  g.len = reinterpret_cast<int*>(g.base + c->o_len);
  g.table = reinterpret_cast<int*>(g.base + c->o_table);
  g.ref = reinterpret_cast<int*>(g.base + c->o_ref);
  g.claim = reinterpret_cast<int*>(g.base + c->o_claim);
  g.rows = reinterpret_cast<tq::PagedRow*>(g.base + c->o_rows);
  g.scan = reinterpret_cast<int*>(g.base + c->o_scan);
  g.moves = reinterpret_cast<int2*>(g.base + c->o_moves);
  g.remap = reinterpret_cast<int*>(g.base + c->o_remap);
  return g;
}

int extend(tq_paged* c, const int32_t* slots, const int32_t* cu, int n, int64_t total, void* stream, const char* name) {
  int st = check(c, name);
  if (st == TQ_OK) st = check_ints(slots, cu, n, c->desc.slots, name);
  if (st == TQ_OK) st = check_pending(name);
  if (st != TQ_OK) return st;
  const cudaError_t e = tq::paged_launch_extend(geom(c), slots, cu, n, total, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) c->plan_rows = n;
  return done(e, name);
}

// A token stride in elements: whole 16-byte pieces, no token inside another.
bool bad_stride(const tq_paged* c, int64_t stride, int64_t heads) {
  return stride < heads * c->desc.d || stride * tq::paged_esize(c->desc.dtype) % 16 != 0;
}

int check_tokens(const tq_paged* c, const void* K, const void* V, int64_t k_stride, int64_t v_stride, int64_t total,
                 const char* name) {
  if (total < 0 || total > INT_MAX) return set_error(TQ_ERR_INVALID_ARG, "%s: total=%lld", name, (long long)total);
  if (total == 0) return TQ_OK;
  if (!K || !V || !aligned(K, 16) || !aligned(V, 16))
    return set_error(TQ_ERR_INVALID_ARG, "%s: K and V must be non-null, 16-byte aligned", name);
  if (bad_stride(c, k_stride, c->desc.Hkv) || bad_stride(c, v_stride, c->desc.Hkv))
    return set_error(TQ_ERR_INVALID_ARG, "%s: token strides %lld, %lld: at least Hkv * d, multiples of 16 bytes", name,
                     (long long)k_stride, (long long)v_stride);
  return TQ_OK;
}

}  // namespace

extern "C" {

size_t tq_paged_bytes(const tq_paged_desc* desc) {
  tq_paged c;
  return layout_status(desc, &c) == TQ_OK ? c.bytes : 0;
}

int tq_paged_layout(const tq_paged_desc* desc, tq_paged* out) {
  if (!out) return set_error(TQ_ERR_INVALID_ARG, "null output");
  const int st = layout_status(desc, out);
  return st == TQ_OK ? tq::clear_error() : st;
}

int tq_paged_init(tq_paged* c, const tq_paged_desc* desc, void* dev_mem, size_t bytes, void* stream) {
  TQ_FAULT_POINT("tq_paged_init");
  if (!c) return set_error(TQ_ERR_INVALID_ARG, "tq_paged_init: null cache");
  tq_paged l;
  int st = layout_status(desc, &l);
  if (st != TQ_OK) return st;
  if (!dev_mem || !aligned(dev_mem, 256))
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_init: device memory must be non-null, 256-byte aligned");
  if (bytes < l.bytes)
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_init: %zu bytes, the layout needs %zu", bytes, l.bytes);
  st = check_pending("tq_paged_init");
  if (st != TQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  l.base = dev_mem;
  const cudaError_t e = tq::paged_launch_init(geom(&l), s);
  if (e != cudaSuccess) return cuda_fail(e, "tq_paged_init");
  *c = l;
  return tq::clear_error();
}

int tq_paged_extend(tq_paged* c, const int32_t* slots, const int32_t* cu, int n, void* stream) {
  TQ_FAULT_POINT("tq_paged_extend");
  return extend(c, slots, cu, n, -1, stream, "tq_paged_extend");
}

int tq_paged_extend_within(tq_paged* c, const int32_t* slots, const int32_t* cu, int n, int64_t total, void* stream) {
  TQ_FAULT_POINT("tq_paged_extend_within");
  if (total < 0 || total > INT_MAX)
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_extend_within: total=%lld", (long long)total);
  return extend(c, slots, cu, n, total, stream, "tq_paged_extend_within");
}

int tq_paged_write(const tq_paged* c, int layer, const void* K, const void* V, int64_t k_stride, int64_t v_stride,
                   int64_t total, void* stream) {
  TQ_FAULT_POINT("tq_paged_write");
  int st = check_layer(c, layer, "tq_paged_write");
  if (st != TQ_OK) return st;
  st = check_tokens(c, K, V, k_stride, v_stride, total, "tq_paged_write");
  if (st != TQ_OK) return st;
  if (total == 0) return tq::clear_error();
  if (c->plan_rows < 1) return set_error(TQ_ERR_INVALID_ARG, "tq_paged_write: no tq_paged_extend before it");
  st = check_pending("tq_paged_write");
  if (st != TQ_OK) return st;
  return done(tq::paged_launch_write(geom(c), layer, K, V, k_stride, v_stride, total, c->plan_rows,
                                     static_cast<cudaStream_t>(stream)),
              "tq_paged_write");
}

int tq_paged_append(tq_paged* c, const int32_t* slots, const int32_t* cu, int n, const void* K, const void* V,
                    int64_t k_stride, int64_t v_stride, int64_t total, void* stream) {
  TQ_FAULT_POINT("tq_paged_append");
  int st = check_layer(c, 0, "tq_paged_append");
  if (st == TQ_OK && c->desc.layers != 1)
    st = set_error(TQ_ERR_INVALID_ARG, "tq_paged_append: layers=%d, not 1", c->desc.layers);
  if (st == TQ_OK) st = check_tokens(c, K, V, k_stride, v_stride, total, "tq_paged_append");
  if (st == TQ_OK) st = extend(c, slots, cu, n, total, stream, "tq_paged_append");
  if (st != TQ_OK || total == 0) return st;
  return done(tq::paged_launch_write(geom(c), 0, K, V, k_stride, v_stride, total, n, static_cast<cudaStream_t>(stream)),
              "tq_paged_append");
}

int tq_paged_read(const tq_paged* c, int layer, const int32_t* slots, const int32_t* cu, int n, int64_t total, void* K,
                  void* V, void* stream) {
  TQ_FAULT_POINT("tq_paged_read");
  int st = check_layer(c, layer, "tq_paged_read");
  if (st == TQ_OK) st = check_ints(slots, cu, n, INT_MAX / 4, "tq_paged_read");
  if (st != TQ_OK) return st;
  if (total < 0 || total > INT_MAX) return set_error(TQ_ERR_INVALID_ARG, "tq_paged_read: total=%lld", (long long)total);
  if (total == 0) return tq::clear_error();
  if (!K || !V || !aligned(K, 16) || !aligned(V, 16))
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_read: K and V must be non-null, 16-byte aligned");
  const int64_t bytes = total * c->desc.Hkv * c->desc.d * tq::paged_esize(c->desc.dtype);
  const Extent k{K, bytes}, v{V, bytes}, m{c->base, (int64_t)c->bytes};
  if (meet(k, v) || meet(k, m) || meet(v, m))
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_read: K, V and the cache overlap");
  st = check_pending("tq_paged_read");
  if (st != TQ_OK) return st;
  return done(tq::paged_launch_read(geom(c), layer, slots, cu, n, total, K, V, static_cast<cudaStream_t>(stream)),
              "tq_paged_read");
}

int tq_paged_table(const tq_paged* c, const int32_t* slots, int n, int32_t* out, void* stream) {
  TQ_FAULT_POINT("tq_paged_table");
  int st = check(c, "tq_paged_table");
  if (st == TQ_OK) st = check_ints(slots, out, n, INT_MAX / 4, "tq_paged_table");
  if (st == TQ_OK) st = check_pending("tq_paged_table");
  if (st != TQ_OK) return st;
  return done(tq::paged_launch_table(geom(c), slots, n, out, static_cast<cudaStream_t>(stream)), "tq_paged_table");
}

size_t tq_paged_workspace_bytes(const tq_paged* c) {
  return check(c, "tq_paged_workspace_bytes") == TQ_OK ? tq::paged_attn_ws_bytes(c->desc.d) : 0;
}

int tq_paged_workspace_init(const tq_paged* c, void* workspace, size_t ws_bytes, void* stream) {
  TQ_FAULT_POINT("tq_paged_workspace_init");
  int st = check(c, "tq_paged_workspace_init");
  if (st != TQ_OK) return st;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < tq::paged_attn_ws_bytes(c->desc.d))
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_workspace_init: workspace must be 256-byte aligned, %zu bytes",
                     tq::paged_attn_ws_bytes(c->desc.d));
  st = check_pending("tq_paged_workspace_init");
  if (st != TQ_OK) return st;
  return done(tq::paged_launch_ws_init(workspace, static_cast<cudaStream_t>(stream)), "tq_paged_workspace_init");
}

int tq_paged_attention(const tq_paged* c, int layer, const void* Q, int64_t q_stride, int Hq, const int32_t* slots,
                       const int32_t* cu, int n, int max_q, int64_t total_q, int causal, float softmax_scale, void* out,
                       float* lse, void* workspace, size_t ws_bytes, void* stream) {
  TQ_FAULT_POINT("tq_paged_attention");
  int st = check_layer(c, layer, "tq_paged_attention");
  if (st == TQ_OK) st = check_ints(slots, cu, n, 1 << 20, "tq_paged_attention");
  if (st != TQ_OK) return st;
  const int Hkv = c->desc.Hkv;
  if (Hq < Hkv || Hq % Hkv != 0 || Hq / Hkv > tq::kMaxG)
    return set_error(TQ_ERR_UNSUPPORTED, "Hq=%d must be a multiple of Hkv=%d with at most %d heads per KV head", Hq, Hkv,
                     tq::kMaxG);
  // (a call without queries has no longest row)
  if (total_q < 0 || total_q > INT_MAX || max_q < (total_q > 0 ? 1 : 0) || max_q > (1 << 24))
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_attention: total_q=%lld max_q=%d", (long long)total_q, max_q);
  if (!std::isfinite(softmax_scale)) return set_error(TQ_ERR_INVALID_ARG, "tq_paged_attention: softmax_scale not finite");
  if (total_q == 0) return tq::clear_error();
  if (!Q || !out || !aligned(Q, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_attention: Q and out must be non-null, 16-byte aligned");
  if (bad_stride(c, q_stride, Hq))
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_attention: q_stride=%lld: at least Hq * d, a multiple of 16 bytes",
                     (long long)q_stride);
  // several CTAs read a query, and the codes, that one of them answers: nothing that is written may lie
  // over what is read
  const int64_t es = tq::paged_esize(c->desc.dtype), row = (int64_t)Hq * c->desc.d * es;
  const Extent q{Q, (total_q - 1) * q_stride * es + row}, o{out, total_q * row}, l{lse, total_q * Hq * 4},
      w{workspace, (int64_t)tq::paged_attn_ws_bytes(c->desc.d)}, m{c->base, (int64_t)c->bytes};
  if (meet(o, q) || meet(o, l) || meet(o, w) || meet(o, m) || meet(l, q) || meet(l, w) || meet(l, m) || meet(w, q) ||
      meet(w, m))
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_attention: out, lse or workspace overlaps another array");
  if (!workspace || !aligned(workspace, 256) || ws_bytes < tq::paged_attn_ws_bytes(c->desc.d))
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_attention: workspace must be 256-byte aligned, %zu bytes",
                     tq::paged_attn_ws_bytes(c->desc.d));
  st = check_pending("tq_paged_attention");
  if (st != TQ_OK) return st;
  tq::PagedAttn a{};
  a.Q = Q;
  a.q_stride = q_stride;
  a.out = out;
  a.lse = lse;
  a.slots = slots;
  a.cu = cu;
  a.n = n;
  a.Hq = Hq;
  a.max_q = max_q;
  a.layer = layer;
  a.total_q = total_q;
  a.causal = causal != 0;
  a.scale = softmax_scale;
  a.ws = workspace;
  a.ws_bytes = ws_bytes;
  return done(tq::paged_launch_attention(geom(c), a, static_cast<cudaStream_t>(stream)), "tq_paged_attention");
}

int tq_paged_fork(tq_paged* c, const int32_t* from, const int32_t* to, int n, void* stream) {
  TQ_FAULT_POINT("tq_paged_fork");
  int st = check(c, "tq_paged_fork");
  if (st == TQ_OK) st = check_ints(from, to, n, c->desc.slots, "tq_paged_fork");
  if (st == TQ_OK) st = check_pending("tq_paged_fork");
  if (st != TQ_OK) return st;
  const tq::PGeom g = geom(c);
  return done(tq::paged_launch_branch(g, g, from, to, n, true, static_cast<cudaStream_t>(stream)), "tq_paged_fork");
}

int tq_paged_copy(const tq_paged* src, tq_paged* dst, const int32_t* from, const int32_t* to, int n, void* stream) {
  TQ_FAULT_POINT("tq_paged_copy");
  int st = check(src, "tq_paged_copy");
  if (st == TQ_OK) st = check(dst, "tq_paged_copy");
  if (st == TQ_OK) st = check_ints(from, to, n, dst->desc.slots, "tq_paged_copy");
  if (st != TQ_OK) return st;
  const tq_paged_desc &a = src->desc, &b = dst->desc;
  if (a.layers != b.layers || a.Hkv != b.Hkv || a.d != b.d || a.page != b.page || a.dtype != b.dtype || a.code != b.code)
    return set_error(TQ_ERR_INVALID_ARG, "tq_paged_copy: the caches differ in layers, Hkv, d, page, dtype or code");
  st = check_pending("tq_paged_copy");
  if (st != TQ_OK) return st;
  return done(tq::paged_launch_branch(geom(src), geom(dst), from, to, n, false, static_cast<cudaStream_t>(stream)),
              "tq_paged_copy");
}

int tq_paged_free(tq_paged* c, const int32_t* slots, int n, void* stream) {
  TQ_FAULT_POINT("tq_paged_free");
  int st = check(c, "tq_paged_free");
  if (st == TQ_OK) st = check_ints(slots, slots, n, INT_MAX / 4, "tq_paged_free");
  if (st == TQ_OK) st = check_pending("tq_paged_free");
  if (st != TQ_OK) return st;
  return done(tq::paged_launch_free(geom(c), slots, n, static_cast<cudaStream_t>(stream)), "tq_paged_free");
}

int tq_paged_compact(tq_paged* c, void* stream) {
  TQ_FAULT_POINT("tq_paged_compact");
  int st = check(c, "tq_paged_compact");
  if (st == TQ_OK) st = check_pending("tq_paged_compact");
  if (st != TQ_OK) return st;
  return done(tq::paged_launch_compact(geom(c), static_cast<cudaStream_t>(stream)), "tq_paged_compact");
}

int tq_paged_check(tq_paged* c, int32_t* free_pages, void* stream) {
  TQ_FAULT_POINT("tq_paged_check");
  int st = check(c, "tq_paged_check");
  if (st != TQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int v[2];
  const tq::PGeom g = geom(c);
  static_assert(offsetof(tq::PagedState, status) == 0 && offsetof(tq::PagedState, n_free) == 4, "read together");
  cudaError_t e = cudaMemcpyAsync(v, g.state, sizeof(v), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  // (only what is reported: a call on another stream may fail meanwhile)
  if (e == cudaSuccess && v[0] != 0) e = tq::paged_launch_clear(g, v[0], s);
  if (e != cudaSuccess) return cuda_fail(e, "tq_paged_check");
  if (free_pages) *free_pages = v[1];
  if (v[0] == 0) return tq::clear_error();
  const struct {
    int bit, status;
    const char* what;
  } reasons[] = {{tq::kPagedWait, TQ_ERR_CUDA, "a paged attention's bounded wait gave up"},
                 {tq::kPagedNoPages, TQ_ERR_CAPACITY, "not enough free pages"},
                 {tq::kPagedTooLong, TQ_ERR_CAPACITY, "a sequence would outgrow max_pages"},
                 {tq::kPagedBadSlot, TQ_ERR_INVALID_ARG, "a slot out of range, named twice, or freed before its write"},
                 {tq::kPagedBadOffsets, TQ_ERR_INVALID_ARG, "token offsets that decrease, leave the arrays or pass max_q"},
                 {tq::kPagedNotEmpty, TQ_ERR_INVALID_ARG, "a fork or copy into a slot that is not empty"},
                 {tq::kPagedBadWorkspace, TQ_ERR_INVALID_ARG, "an attention workspace that was not initialised"},
                 {tq::kPagedBadPage, TQ_ERR_INVALID_ARG, "a page table entry out of range"}};
  char text[512] = "";
  int status = TQ_OK;
  for (const auto& r : reasons)
    if (v[0] & r.bit) {
      if (status == TQ_OK) status = r.status;
      const size_t at = std::strlen(text);
      std::snprintf(text + at, sizeof(text) - at, "%s%s", at ? "; " : "", r.what);
    }
  return set_error(status == TQ_OK ? TQ_ERR_CUDA : status, "%s (%d pages free, max_pages=%d)", text, v[1],
                   c->desc.max_pages);
}

}  // extern "C"
