// Geometry and address arithmetic of the paged 8-bit cache, shared by its kernel files.
//
// A page holds `page` tokens of one sequence.  Its tokens of one KV head are a block: for
// the keys and for the values one scale each.  A block is stored as sub-blocks of
// sub = min(page, 64) tokens, each sub * d code bytes followed by a 32-byte trailer (the
// block's scale, then its largest magnitude, as floats), so that one bulk copy brings the
// codes and their scale and every sub-block starts on a 32-byte boundary:
//   keys    [token][d], the two 64-byte halves of each 128 bytes exchanged for odd tokens
//           (two adjacent tokens then fill all shared-memory banks of a 16-byte-per-lane read);
//   values  [d][token] (a lane's 16 bytes are 16 tokens of one channel: the B operand of P V).
// int8 codes are stored with 128 added (an unsigned byte c turns into the half 1024 + c by
// one byte permutation), e4m3 codes as they are.
#pragma once

#include <atomic>

#include "common.cuh"

namespace tq {

constexpr int kPagedTrailer = 32;

// Status bits of a cache, set by the kernels, read and cleared by tq_paged_check.
enum PagedStatus : int {
  kPagedNoPages = 1,       // not enough free pages
  kPagedTooLong = 2,       // a sequence would outgrow its page table
  kPagedBadSlot = 4,       // a slot out of range, or named twice where it may not be
  kPagedBadOffsets = 8,    // token offsets that decrease or leave the arrays
  kPagedNotEmpty = 16,     // fork / copy into a slot that holds tokens
  kPagedBadWorkspace = 32, // an attention workspace that was not initialised
  kPagedWait = 64,         // a bounded wait gave up
  kPagedBadPage = 128      // a page table entry out of range
};

struct PagedState {
  int status;
  int n_free;      // pages with reference count 0
  int n_rows;      // rows of the last extend's plan
  int n_items;     // (row, page) items of that plan
  int n_moves;     // page copies of the last fork / copy / compact
  int n_pairs;     // pairs of the last fork / copy
  int compacted;   // 1: the last plan renumbers pages (compact)
  int low;         // every page below this one is in use
  int end;         // input tokens that the last extend's plan reaches to
};

struct PagedRow {  // one row of an extend: `count` tokens from row `src` of the input
  int slot, src, start, count, item;
};

struct PGeom {
  int layers, Hkv, d, page, sub, pages, slots, max_pages, dtype, code;
  int64_t sb, hb, page_bytes;       // sub-block, block, page (one layer)
  int64_t tail_head;                // bytes of one (slot, K/V, head) of the exact tail
  uint8_t* base;
  int64_t total;                    // extent of the buffer
  uint8_t* pool;
  uint8_t* tail;
  PagedState* state;
  int* len;                         // [slots] tokens
  int* table;                       // [slots][max_pages]
  int* ref;                         // [pages]
  int* claim;                       // [slots] scratch of the planning kernels (all -1 between calls)
  PagedRow* rows;                   // [slots]
  int* scan;                        // [slots + 1]
  int2* moves;                      // [pages] (from, to)
  int* remap;                       // [pages]
};

__host__ __device__ __forceinline__ int paged_esize(int dtype) { return dtype == TQ_F32 ? 4 : 2; }

// Sub-block `sub_i` of the block (layer, page, keys 0 / values 1, head).
__device__ __forceinline__ uint8_t* paged_block(const PGeom& g, int layer, int pid, int kv, int h,
                                                int sub_i) {
  return g.pool + ((int64_t)layer * g.pages + pid) * g.page_bytes +
         ((int64_t)kv * g.Hkv + h) * g.hb + (int64_t)sub_i * g.sb;
}

// Byte offset in a key sub-block of channel j of its token t.
__device__ __forceinline__ int paged_k_off(int d, int t, int j) {
  return d == 64 ? t * d + j : t * d + (j ^ ((t & 1) << 6));
}

__device__ __forceinline__ uint8_t* paged_tail(const PGeom& g, int layer, int slot, int kv, int h) {
  return g.tail + (((int64_t)layer * g.slots + slot) * 2 * g.Hkv + (int64_t)kv * g.Hkv + h) * g.tail_head;
}

// Tokens of a slot (0 for a slot out of range: callers treat it as an empty sequence).
__device__ __forceinline__ int paged_len(const PGeom& g, int slot) {
  return (unsigned)slot < (unsigned)g.slots ? g.len[slot] : 0;
}

// The kernel's dynamic shared memory limit, set once per device and kernel.
template <auto Kernel>
cudaError_t paged_allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ---- host launchers ----
cudaError_t paged_launch_init(const PGeom& g, cudaStream_t s);      // every slot empty, every page free
// total: input tokens there are (the plan is refused if a row goes past them), or -1: not known yet
cudaError_t paged_launch_extend(const PGeom& g, const int* slots, const int* cu, int n, int64_t total, cudaStream_t s);
cudaError_t paged_launch_write(const PGeom& g, int layer, const void* K, const void* V, int64_t k_stride,
                               int64_t v_stride, int64_t total, int n_rows, cudaStream_t s);
cudaError_t paged_launch_read(const PGeom& g, int layer, const int* slots, const int* cu, int n,
                              int64_t total, void* K, void* V, cudaStream_t s);
cudaError_t paged_launch_free(const PGeom& g, const int* slots, int n, cudaStream_t s);
// src and dst may be the same cache; share: full pages are shared instead of copied
cudaError_t paged_launch_branch(const PGeom& src, const PGeom& dst, const int* from, const int* to, int n,
                                bool share, cudaStream_t s);
cudaError_t paged_launch_compact(const PGeom& g, cudaStream_t s);
cudaError_t paged_launch_clear(const PGeom& g, int bits, cudaStream_t s);      // of the status
cudaError_t paged_launch_table(const PGeom& g, const int* slots, int n, int* out, cudaStream_t s);

struct PagedAttn {
  const void* Q;
  int64_t q_stride;        // elements between query tokens
  void* out;               // [total_q][Hq][d]
  float* lse;              // [total_q][Hq] or null
  const int* slots;
  const int* cu;           // [n + 1]
  int n, Hq, max_q, layer;
  int64_t total_q;
  int causal;
  float scale;
  void* ws;
  size_t ws_bytes;
};
size_t paged_attn_ws_bytes(int d);
// many query rows (paged_chunk.cu)
size_t paged_chunk_ws_bytes(int d);
cudaError_t paged_launch_chunk(const PGeom& g, const PagedAttn& a, cudaStream_t s);
cudaError_t paged_lose_copies(int on);                                          // see tq_debug_paged_lose_copies
cudaError_t paged_launch_ws_init(void* ws, cudaStream_t s);
cudaError_t paged_launch_attention(const PGeom& g, const PagedAttn& a, cudaStream_t s);

int bounds_flag_paged_pages();
int bounds_flag_paged_quant();
int bounds_flag_paged_attn();
int bounds_flag_paged_chunk();

// Shared with abi.cu: success (clears the thread's message), the fault injector.
int clear_error();
bool fault_injected(const char* name);

}  // namespace tq
