// Index arithmetic of the paged key-value cache, shared by the kernels and
// by a host-compiled test. Every function returns a value that is safe to
// use, or -1, whatever the page table, the lengths and the offsets hold.
#pragma once

#include <cstdint>

// OSS_ROLLED: a loop that is not to be unrolled (what runs once per call should
// not push a kernel's main loop out of the instruction cache).
#if defined(__CUDACC__)
#define OSS_HD __host__ __device__ __forceinline__
#define OSS_ROLLED _Pragma("unroll 1")
#else
#define OSS_HD inline
#define OSS_ROLLED
#endif

namespace oss {

// Sites of the error word's kernel 3 (an index outside the cache).
enum PagedSite : unsigned int { kSiteBadPage = 1, kSiteBadPosition = 2, kSiteBadOffsets = 3 };

// The pools and tables of an os_paged_cache, by value for kernels.
struct PagedCache {
  const uint16_t* k;
  const uint16_t* v;
  int64_t ld_page, ld_head, ld_slot;  // elements
  const int32_t* table;
  int64_t ld_table;
  const int32_t* kv_len;
  int32_t num_pages, page_shift, max_pages, heads, batch;
};

// Tokens of a sequence: its kv_len, clamped to what its pages hold.
OSS_HD int32_t paged_length(int32_t kv_len, int32_t max_pages, int32_t page_shift) {
  const int32_t cap = max_pages << page_shift;
  return kv_len < 0 ? 0 : (kv_len > cap ? cap : kv_len);
}

// Whether a page number of the table may be followed.
OSS_HD bool page_ok(int32_t page, int32_t num_pages) {
  return static_cast<uint32_t>(page) < static_cast<uint32_t>(num_pages);
}

// Element offset of (page, head, slot) in a pool, in 64 bits.
OSS_HD int64_t pool_offset(int32_t page, int32_t head, int32_t slot, int64_t ld_page,
                           int64_t ld_head, int64_t ld_slot) {
  return static_cast<int64_t>(page) * ld_page + static_cast<int64_t>(head) * ld_head +
         static_cast<int64_t>(slot) * ld_slot;
}

// The sequence that row `token` belongs to: the b with cu[b] <= token <
// cu[b + 1], or -1. For offsets that are not ascending the answer may be -1
// for a token that some sequence has; it never names a sequence whose range
// the token is outside of.
OSS_HD int32_t sequence_of(int64_t token, const int32_t* cu, int32_t batch) {
  int32_t lo = 0, hi = batch;  // the first b in [0, batch] with cu[b] > token is in (lo, hi]
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (cu[mid + 1] > token)
      hi = mid;
    else
      lo = mid + 1;
  }
  if (lo >= batch || cu[lo] > token) return -1;
  return lo;
}

// A sequence's range of packed rows, clamped to 0 .. tokens.
struct RowRange {
  int32_t start, len;
  bool clamped;
};

OSS_HD RowRange row_range(int32_t begin, int32_t end, int32_t tokens) {
  RowRange r;
  int32_t b = begin < 0 ? 0 : (begin > tokens ? tokens : begin);
  int32_t e = end < b ? b : (end > tokens ? tokens : end);
  r.start = b;
  r.len = e - b;
  r.clamped = b != begin || e != end;
  return r;
}

// The prefixes that groups of sequences share: group g is sequences cu[g] .. cu[g + 1] - 1
// (cu null: one group of all), and its tokens are those of row g of the table.
struct PrefixTables {
  const int32_t* table;
  int64_t ld_table;
  const int32_t* len;
  const int32_t* cu;
  int32_t groups, max_pages;
};

// Group of sequence b, or -1.
OSS_HD int32_t prefix_group(const PrefixTables& p, int32_t b) {
  return p.cu ? sequence_of(b, p.cu, p.groups) : 0;
}

// Order of fp32 weights as unsigned integers: a larger weight has a larger
// key, -0 equals 0, NaN is above infinity.
OSS_HD uint32_t weight_key_bits(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;  // NaN
  if (u == 0x80000000u) u = 0u;                             // -0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The scale byte e + 127 of a row of the 8-bit cache, from the fp32 bits of its largest
// magnitude f * 2^n, f in [1, 2). With 448 = 1.75 * 2^8, e = n - 8, or n - 7 for f >
// 1.75, which is where adding 2^21 - 1 to the 23 bits of f carries into n. Magnitudes up
// to 1.75 * 2^-119, 0 among them, take the least scale, 2^-127; infinity and NaN 255.
constexpr uint32_t kFp8ScaleNan = 255;

OSS_HD uint32_t fp8_scale_byte(uint32_t bits) {
  if (bits >= 0x7f800000u) return kFp8ScaleNan;
  const uint32_t field = (bits + 0x1fffffu) >> 23;
  return field > 8 ? field - 8 : 0;
}

// The fp32 bits of the scale that a byte stands for.
OSS_HD uint32_t fp8_scale_bits(uint32_t byte) {
  if (byte == kFp8ScaleNan) return 0x7fffffffu;
  return byte ? byte << 23 : 0x00400000u;  // 2^-127 is subnormal
}

}  // namespace oss
