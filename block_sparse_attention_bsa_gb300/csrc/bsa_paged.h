// Host-side declarations of the position, cache and paged-attention calls.
#pragma once

#include <string>

#include "../../include/bsa_paged.h"
#include "bsa_internal.h"

namespace bsa {

// Bit of the device error words of bsa_rope.cu, bsa_paged.cu and the 4-bit cache's
// files: a page table entry that names no page, or a length without pages (bit 0:
// a bounded wait gave up).
constexpr unsigned int kErrPage = 2u;
// The same in the word of bsa_paged.cu where its kernel works for bsaq_forward.
constexpr unsigned int kErrQuantPage = 4u;
unsigned int read_and_clear_rope_error();
unsigned int read_and_clear_paged_error();
bsa_status launch_paged_wait_probe(unsigned long long limit_ns, cudaStream_t stream);

constexpr int kMaxPagedBatch = 4096;

// [B, S, H, D] bf16 input of the calls of bsa_paged.h.  Strides of axes of
// length 1 are replaced by 0; `cache`: strides of longer axes must be positive.
bsa_status check_view(const bsa_tensor* t, const char* fn, const char* name, bool cache, bsa_tensor* view);

// Refuses an array whose elements of `size` bytes the kernels could not read or
// write where it lies (a misaligned access is a fault); NULL passes.
bsa_status check_aligned(const char* fn, const char* name, const void* ptr, int size);

// Refuses memory that a call writes while it reads or writes it elsewhere:
// from the first to behind the last byte of each view.  `in_place`: the same
// memory is fine where x, contiguous, starts where y does.
bsa_status check_apart(const char* fn, const char* x_name, const bsa_tensor& x, const char* y_name,
                       const bsa_tensor& y, bool in_place = false);
// The same for the bytes [lo, hi) that a call writes, against others.
struct Bytes {
  const char* name;
  uintptr_t lo, hi;
};
Bytes bytes_at(const char* name, const void* ptr, int64_t n);
Bytes bytes_of(const char* name, const bsa_tensor& t);
bsa_status check_apart(const char* fn, const Bytes& x, const Bytes& y);
// The view of a contiguous output of x's shape.
bsa_tensor contiguous_like(const bsa_tensor& x, void* ptr);

// The paged cache and its tables, checked.
struct PagedArgs {
  bsa_tensor k, v;
  const int32_t* page_table; int64_t table_stride; int max_pages;
  const int32_t* kv_lens; const int32_t* new_lens;
};
// Key tiles at most of an attention over pages, with the keys that the tables could
// hold: what bsap_forward and bsaq_forward limit (32 bits count them on the device).
int64_t most_tiles_of(const bsa_tensor& qv, int64_t Hkv, int64_t page, int64_t max_pages, int64_t prefix_len);
bsa_status check_paged(const char* fn, const bsa_tensor* k_cache, const bsa_tensor* v_cache,
                       const int32_t* page_table, int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                       const int32_t* new_lens, int64_t B, PagedArgs* a);

}  // namespace bsa
