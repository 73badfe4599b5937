// rld_grad_chunks and rld_grad_pack at their edges, built together with
// routed_lora_delta_amd/csrc/rld_host.cpp under AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_grad_pack_sanitize.py (no GPU involved):
// heap arrays of the exact size, empty gradients and groups, addresses and counts next
// to the end of their range.  Last line "ok" if every result is the expected one.
#include <stdio.h>
#include <string.h>

#include <vector>

#include "rld.h"

static int g_fail = 0;

#define EXPECT(cond)                                                      \
  do {                                                                    \
    if (!(cond)) {                                                        \
      fprintf(stderr, "%s:%d: expected %s\n", __FILE__, __LINE__, #cond); \
      ++g_fail;                                                           \
    }                                                                     \
  } while (0)

static rld_grad_entry entry(uint64_t addr, uint64_t out, uint64_t count, uint32_t group, int bf16) {
  rld_grad_entry e;
  memset(&e, 0, sizeof(e));
  e.addr = addr;
  e.out_addr = out;
  e.count = count;
  e.group = group;
  e.bf16 = bf16;
  return e;
}

static void check(const std::vector<rld_grad_entry>& e, uint32_t groups, uint32_t want) {
  uint32_t n = 7;
  EXPECT(rld_grad_chunks(e.data(), e.size(), &n) == RLD_OK && n == want);
  std::vector<rld_grad_chunk> chunks(n);
  std::vector<uint32_t> starts(groups + 1);
  EXPECT(rld_grad_pack(e.data(), e.size(), groups, chunks.data(), n, starts.data()) == RLD_OK);
  EXPECT(starts[0] == 0 && starts[groups] == n);
  uint64_t listed = 0, packed = 0;
  for (const auto& v : e) listed += v.count;
  for (uint32_t i = 0; i < n; ++i) {
    packed += chunks[i].count;
    EXPECT(chunks[i].count > 0 && chunks[i].group < groups);
    EXPECT(starts[chunks[i].group] <= i && i < starts[chunks[i].group + 1]);
  }
  EXPECT(listed == packed);
  if (n)
    EXPECT(rld_grad_pack(e.data(), e.size(), groups, chunks.data(), n - 1, starts.data()) ==
           RLD_ENOSPACE);
}

int main() {
  check({}, 1, 0);
  check({entry(0, 0, 0, 0, 0)}, 1, 0);
  check({entry(16, 0, 1, 0, 0)}, 1, 1);
  check({entry(16, 0, 2048, 0, 0), entry(1 << 20, 0, 4096, 0, 1)}, 1, 2);
  check({entry(16, 0, 2049, 4, 0), entry(1 << 20, 32, 4097, 0, 1), entry(48, 0, 0, 2, 0)}, 5, 4);
  // the highest addresses, and more elements than 32 bits count
  check({entry(0xFFFFFFFFFFFFE000ull, 0, 2048, 0, 0)}, 1, 1);
  check({entry(1ull << 40, 0, (1ull << 32) + 1, 1, 1)}, 2, (1u << 20) + 1);
  uint32_t n = 7;
  const rld_grad_entry huge[2] = {entry(16, 0, 1ull << 41, 0, 0), entry(16, 0, ~0ull, 0, 0)};
  EXPECT(rld_grad_chunks(huge, 1, &n) == RLD_OK && n == 1u << 30);
  EXPECT(rld_grad_chunks(huge, 2, &n) == RLD_EUNSUPPORTED);
  EXPECT(rld_grad_chunks(nullptr, 0, &n) == RLD_OK && n == 0);
  if (g_fail) return 1;
  printf("ok\n");
  return 0;
}
