// The paged key/value cache as the kernels address it.
#pragma once
#include "pi_host.hpp"
#include "pi_types.hpp"

struct pi_kv {
  pi_kv_desc desc;
  pi_ctx* ctx;
};

namespace pi {

// n / page for n in [0, 2^31): the product with floor(2^32 / page) is short of the quotient by
// at most one.
struct PageDiv {
  uint32_t page, mul;
};
inline PageDiv page_div(uint32_t page) {
  return PageDiv{page, page == 1 ? 0xFFFFFFFFu : (uint32_t)((1ull << 32) / page)};
}
__device__ __forceinline__ uint32_t page_of(PageDiv d, uint32_t n, uint32_t* off) {
  uint32_t q = __umulhi(n, d.mul), r = n - q * d.page;
  if (r >= d.page) {
    ++q;
    r -= d.page;
  }
  *off = r;
  return q;
}

struct KvDev {
  void *k, *v;
  long long page_stride, token_stride, head_stride;
  const int32_t* table;  // NULL: sequence b has page b
  long long table_stride;
  PageDiv div;
  int pages, capacity;   // pages of the cache; positions of a sequence
};

// The page of sequence b's positions from i * page_tokens on, or -1 outside the cache.
__device__ __forceinline__ int kv_page(const KvDev& c, int b, uint32_t i) {
  const int id = c.table == nullptr ? b : c.table[(long long)b * c.table_stride + i];
  return (unsigned)id < (unsigned)c.pages ? id : -1;
}

__device__ __forceinline__ int kv_len(const KvDev& c, const int32_t* ctx_len, int b) {
  return min(max(ctx_len[b], 0), c.capacity);
}

// The arguments that the calls on a cache share.
inline pi_status check_paging(pi_ctx* c, const pi_kv* kv, const int32_t* table, int64_t table_stride, int32_t width,
                              const int32_t* ctx_len, int32_t B, int32_t N) {
  if (kv == nullptr) return fail(c, PI_ERR_INVALID, "kv is NULL");
  if (kv->ctx != c) return fail(c, PI_ERR_INVALID, "the cache belongs to another context");
  if (B < 1 || N < 1) return fail(c, PI_ERR_INVALID, "bad shape B=%d N=%d", B, N);
  if (ctx_len == nullptr) return fail(c, PI_ERR_INVALID, "ctx_len is NULL");
  if (table != nullptr) {
    if (width < 1 || (B > 1 && table_stride < width))
      return fail(c, PI_ERR_INVALID, "bad page table: width %d, stride %lld", width, (long long)table_stride);
    if ((int64_t)width * kv->desc.page_tokens >= (1ll << 31) - 64)
      return fail(c, PI_ERR_INVALID, "a page table of %d pages of %d tokens is too long", width, kv->desc.page_tokens);
  } else if (B > kv->desc.pages) {
    return fail(c, PI_ERR_INVALID, "%d sequences without a page table need as many pages (have %d)", B, kv->desc.pages);
  }
  return PI_OK;
}

inline KvDev kv_dev(const pi_kv* kv, const int32_t* table, int64_t table_stride, int32_t width) {
  const pi_kv_desc& d = kv->desc;
  return KvDev{d.k, d.v, d.page_stride, d.token_stride, d.head_stride, table, table_stride,
               page_div((uint32_t)d.page_tokens), d.pages, table != nullptr ? width * d.page_tokens : d.page_tokens};
}

// Strides of a [B][N][heads][D] tensor of 16-bit elements whose rows are 16-byte aligned.
inline pi_status check_bnh(pi_ctx* c, const char* name, const void* p, int64_t sb, int64_t sn, int64_t sh) {
  PI_TRY(check_dev_ptr(c, p, name));
  if ((sb | sn | sh) & 7) return fail(c, PI_ERR_INVALID, "%s: strides must be multiples of 8 elements", name);
  return PI_OK;
}

}  // namespace pi
