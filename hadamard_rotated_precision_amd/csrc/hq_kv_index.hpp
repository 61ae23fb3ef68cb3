// hq_kv_index.hpp — where a token of a paged cache lies, with the checks that keep a wrong slot,
// page or length inside the buffers. Plain arithmetic, for the kernels and for tests on the host.
#pragma once

#include <stdint.h>

#if defined(__HIP__) || defined(__HIPCC__)
#define HQ_BOTH __host__ __device__ inline
#else
#define HQ_BOTH inline
#endif

namespace hq {

// Row of a slot in k_codes' pages x heads x page rows, or -1 for a slot outside the cache. page is
// 2^shift.
HQ_BOTH int64_t kv_row_of_slot(int64_t slot, int64_t pages, int shift, int heads, int head) {
  if (slot < 0 || slot >= (pages << shift)) return -1;
  return ((((slot >> shift) * heads) + head) << shift) + (slot & ((int64_t{1} << shift) - 1));
}

// Whether a sequence's table has this entry.
HQ_BOTH bool kv_entry_in_table(int64_t entry, int64_t table_ld) { return entry >= 0 && entry < table_ld; }
// The entry of a sequence's table that names the page of its token `at`, or -1 where the table ends before.
HQ_BOTH int64_t kv_entry_of_token(int at, int64_t table_ld, int shift) {
  const int64_t p = at >> shift;
  return kv_entry_in_table(p, table_ld) ? p : -1;
}
// Row of token `at` in the page that the entry names, or -1 where that is no page of the cache.
HQ_BOTH int64_t kv_row_in_page(int at, int32_t page, int64_t pages, int shift, int heads, int head) {
  if (page < 0 || page >= pages) return -1;
  return (((static_cast<int64_t>(page) * heads) + head) << shift) + (at & ((int64_t{1} << shift) - 1));
}
HQ_BOTH int64_t kv_row_of_token(int at, const int32_t* table, int64_t table_ld, int64_t pages, int shift, int heads,
                                int head) {
  const int64_t p = kv_entry_of_token(at, table_ld, shift);
  return p < 0 ? -1 : kv_row_in_page(at, table[p], pages, shift, heads, head);
}

// A sequence's query rows [first, first + n) of the tensor's `tokens`, at most max_q of them, and its
// length, at most max_len. `behind`: new tokens that lie beyond the bounds count as seen by nobody,
// but row i keeps its position len - (end - first) + i.
struct KvSequence {
  int64_t first;
  int n;          // rows to compute
  int64_t pos0;   // position of row 0
  int len;        // tokens that may be seen
};
HQ_BOTH KvSequence kv_sequence(int32_t start, int32_t end, int32_t len, int64_t tokens, int max_q, int max_len) {
  KvSequence s;
  s.first = start;
  const int64_t all = static_cast<int64_t>(end) - start;
  const bool ok = start >= 0 && all > 0;
  int64_t n = ok ? all : 0;
  if (ok && s.first + n > tokens) n = tokens > s.first ? tokens - s.first : 0;
  s.n = static_cast<int>(n < max_q ? n : max_q);
  const int64_t l = len > 0 ? len : 0;
  s.pos0 = l - (ok ? all : 0);
  s.len = static_cast<int>(l < max_len ? l : max_len);
  return s;
}

// Tokens [kv_start_of, kv_end_of) are those that query row i sees; both lie in [0, s.len], whatever the
// position (a length that the bound cuts may be any).
HQ_BOTH int kv_cut(const KvSequence& s, int64_t at) { return static_cast<int>(at < 0 ? 0 : at < s.len ? at : s.len); }
HQ_BOTH int kv_end_of(const KvSequence& s, int i) { return kv_cut(s, s.pos0 + i + 1); }
HQ_BOTH int kv_start_of(const KvSequence& s, int i, int window) { return window ? kv_cut(s, s.pos0 + i + 1 - window) : 0; }

// The chunks of `size` tokens that one of the query rows first .. last sees.
struct KvChunks {
  int first, count;
};
HQ_BOTH KvChunks kv_chunks(const KvSequence& s, int first, int last, int window, int size) {
  const int from = kv_start_of(s, first, window), to = kv_end_of(s, last);
  return KvChunks{from / size, from < to ? (to + size - 1) / size - from / size : 0};
}

}  // namespace hq
