"""Host-side AddressSanitizer and UndefinedBehaviorSanitizer runs (CPU only, no GPU code) of what
include/hq_mx.h stands on: the argument checks (hq_mx_api.cpp with stand-ins for the kernel launchers,
under tests/test_mx_abi.py), and the arithmetic that finds a token's row in the cache
(hq_kv_index.hpp), with slots, pages, lengths and query rows of every wrong kind."""
import os
import subprocess

import pytest

from test_sanitizers import CSRC, LIBASAN, ROOT, SAN, _run_pytest

needs_asan = pytest.mark.skipif(LIBASAN is None, reason="gcc's libasan is not available")


@needs_asan
def test_mx_abi_checks_under_sanitizers(tmp_path):
    objs = []
    for src in (os.path.join(CSRC, "hq_api.cpp"), os.path.join(CSRC, "hq_profile.cpp"),
                os.path.join(CSRC, "hq_mx_api.cpp"),
                os.path.join(ROOT, "tests", "sanitize", "launcher_stubs.cpp"),
                os.path.join(ROOT, "tests", "sanitize", "mx_launcher_stubs.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        subprocess.run(["g++", "-std=c++17", "-w", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                        "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include")] + SAN +
                       ["-c", src, "-o", obj], check=True)
        objs.append(obj)
    lib = str(tmp_path / "libhq_mx_san.so")
    subprocess.run(["g++", "-shared"] + SAN + objs +
                   ["-L/opt/rocm/lib", "-lamdhip64", "-o", lib], check=True)
    _run_pytest({"HQ_LIB_PATH": lib, "HQ_MX_LIB_PATH": lib}, [os.path.join("tests", "test_mx_abi.py")])


PROGRAM = r'''
#include "hq_kv_index.hpp"
#include <cstdio>
#include <vector>
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
using namespace hq;
int main() {
  const int64_t wild[] = {INT64_MIN, INT64_MIN + 1, -(int64_t{1} << 40), -2147483649LL, -2147483648LL, -65, -1,
                          int64_t{1} << 31, (int64_t{1} << 31) + 5, int64_t{1} << 40, INT64_MAX - 1, INT64_MAX};
  for (int shift = 4; shift <= 20; shift += 4)
    for (int heads : {1, 3, 1024})
      for (int64_t pages : {int64_t{0}, int64_t{1}, int64_t{7}, int64_t{2048}}) {
        const int64_t slots = pages << shift, rows = slots * heads;
        for (int head : {0, heads - 1}) {
          for (int64_t s : wild) CHECK(kv_row_of_slot(s, pages, shift, heads, head) == -1 || s < slots);
          CHECK(kv_row_of_slot(slots, pages, shift, heads, head) == -1);
          for (int64_t s = 0; s < slots; s += 1 + slots / 97) {
            const int64_t r = kv_row_of_slot(s, pages, shift, heads, head);
            CHECK(r >= 0 && r < rows && (r >> shift) % heads == head && (r >> shift) / heads == s >> shift);
          }
          // a table of its own allocation: reading past it would be reported
          for (int64_t ld : {0, 1, 5}) {
            for (int32_t entry : {INT32_MIN, -1, 0, static_cast<int32_t>(pages) - 1, static_cast<int32_t>(pages), INT32_MAX}) {
              std::vector<int32_t> table(ld, entry);
              for (int at : {INT32_MIN, -1, 0, 15, 16, (1 << shift) - 1, 1 << shift, 5 << shift, 1 << 30, INT32_MAX}) {
                const int64_t r = kv_row_of_token(at, table.data(), ld, pages, shift, heads, head);
                const bool named = at >= 0 && (at >> shift) < ld && entry >= 0 && entry < pages;
                CHECK(named ? r >= 0 && r < rows : r == -1);
                // sixteen tokens from a multiple of 16 on lie in one page
                if (named && at % 16 == 0) CHECK(r % 16 == 0 && r + 16 <= rows);
              }
            }
          }
        }
      }
  const int32_t ends[] = {INT32_MIN, -7, -1, 0, 1, 5, 9, 10, 11, 1000, INT32_MAX};
  for (int32_t a : ends)
    for (int32_t b : ends)
      for (int32_t len : ends)
        for (int64_t tokens : {int64_t{0}, int64_t{1}, int64_t{10}})
          for (int max_q : {0, 1, 4, 100})
            for (int max_len : {0, 3, 2000, INT32_MAX}) {
              const KvSequence s = kv_sequence(a, b, len, tokens, max_q, max_len);
              CHECK(s.n >= 0 && s.n <= max_q && s.len >= 0 && s.len <= max_len);
              if (s.n > 0) CHECK(s.first >= 0 && s.first + s.n <= tokens && s.first + s.n <= b);
              if (s.n > 0) CHECK(s.pos0 == static_cast<int64_t>(len > 0 ? len : 0) - (static_cast<int64_t>(b) - a));
            }
  std::puts("ok");
  return 0;
}
'''


def test_wrong_slots_pages_and_lengths_stay_inside(tmp_path):
    src, exe = tmp_path / "index.cpp", str(tmp_path / "index")
    src.write_text(PROGRAM)
    san = SAN if LIBASAN else []
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I" + CSRC, str(src), "-o", exe] + san, check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    print(r.stdout + r.stderr)
    assert r.returncode == 0 and r.stdout.strip() == "ok"


# What a wave of the attention kernel does before its first load: the chunks of a tile of rows, the wave's
# first one (waves that share rows take every eighth), and the 64 entries of the table around it.
CHUNKS = r'''
#include "hq_kv_index.hpp"
#include <cstdio>
#include <vector>
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
using namespace hq;
int main() {
  const int kSize = 64;
  long waves = 0;
  for (int32_t len : {INT32_MIN, -1, 0, 1, 63, 64, 65, 1000, 1 << 30, INT32_MAX - 64, INT32_MAX - 1, INT32_MAX})
    for (int32_t rows : {1, 2, 9, 1000})
      for (int window : {0, 1, 16, 64, 65, 1000, INT32_MAX - 1, INT32_MAX})
        for (int max_len : {0, 1, 63, 64, 200, 5000, 1 << 30})
          for (int max_q : {1, 4, 1000}) {
            const KvSequence s = kv_sequence(5, 5 + rows, len, 2000, max_q, max_len);
            CHECK(s.n == (rows < max_q ? rows : max_q));
            for (int first = 0; first < s.n; first += 1 + s.n / 3) {
              const int last = first + 15 < s.n ? first + 15 : s.n - 1;
              for (int i : {first, last, last + 2000000000}) {      // rows behind the last are asked about too
                const int from = kv_start_of(s, i, window), to = kv_end_of(s, i);
                CHECK(from >= 0 && from <= s.len && to >= 0 && to <= s.len);
                const int64_t p = s.pos0 + i;
                for (int64_t j : {int64_t{0}, int64_t{1}, int64_t{from} - 1, int64_t{from}, int64_t{to} - 1, int64_t{to}})
                  if (j >= 0 && j < s.len) CHECK((j >= from && j < to) == (j <= p && (!window || j > p - window)));
              }
              const KvChunks c = kv_chunks(s, first, last, window, kSize);
              CHECK(c.first >= 0 && c.count >= 0 && c.first <= (1 << 30) / kSize);
              if (max_len == 0) CHECK(c.count == 0);
              for (int w = 0; w < 8; ++w) {
                if (w >= c.count) continue;
                const int at = (c.first + w) * kSize;
                CHECK(at >= 0 && at < s.len);
                ++waves;
                for (int shift : {4, 6, 20})
                  for (int64_t ld : {0, 1, 7}) {
                    std::vector<int32_t> table(ld, 0);
                    for (int lane = 0; lane < 64; ++lane) {
                      const int64_t entry = (at >> shift) + static_cast<int64_t>(lane);
                      if (kv_entry_in_table(entry, ld)) CHECK(table.at(entry) == 0);
                    }
                  }
              }
            }
          }
  for (int64_t e : {INT64_MIN, -(int64_t{1} << 31), int64_t{-1}, int64_t{7}, int64_t{1} << 31, INT64_MAX}) CHECK(!kv_entry_in_table(e, 7));
  CHECK(waves > 1000);
  std::puts("ok");
  return 0;
}
'''


def test_no_chunk_of_any_length_and_window_lies_outside(tmp_path):
    """Lengths up to 2^31 - 1 with windows: positions past the bound on the lengths give no chunk, and no
    arithmetic on them overflows."""
    src, exe = tmp_path / "chunks.cpp", str(tmp_path / "chunks")
    src.write_text(CHUNKS)
    san = SAN if LIBASAN else []
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I" + CSRC, str(src), "-o", exe] + san, check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    print(r.stdout + r.stderr)
    assert r.returncode == 0 and r.stdout.strip() == "ok"
