// Test infrastructure: as trace_main.cpp, for the entry points around a batched round.
// Commands (one per line):
//   device <sms> <smem_optin>
//   pages <B> <T> <max_pages> <maps 0|1>
//   prefix <B> <S> <Hq> <heads> <dim> <page> <prefix_pages> <max_pages>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <string>

#include "sdv.h"

extern "C" void trace_set_device(int sms, int smem);

namespace {

template <typename T = int32_t>
T* addr(uint64_t off) {
  return reinterpret_cast<T*>(0x100000000ull + off);
}

}  // namespace

int main() {
  char line[512];
  while (std::fgets(line, sizeof line, stdin)) {
    char cmd[32] = {0};
    int a[8] = {0};
    const int got = std::sscanf(line, "%31s %d %d %d %d %d %d %d %d", cmd, &a[0], &a[1], &a[2], &a[3], &a[4], &a[5],
                                &a[6], &a[7]);
    if (got < 1) continue;
    line[std::strcspn(line, "\n")] = 0;
    std::printf("call %s\n", line);
    const std::string c = cmd;
    int st = -1;
    if (c == "device") {
      trace_set_device(a[0], a[1]);
      st = 0;
    } else if (c == "pages") {
      const sdv_pagepool pool = {1 << 20, 16, a[2], addr(0x1000), addr(0x800000), addr(0x900000), addr(0xa00000)};
      st = sdv_page_assign(&pool, a[0], a[1], addr(0xb00000), nullptr, addr(0xc00000), a[3] ? addr(0xd00000) : nullptr,
                           a[3] ? addr(0xe00000) : nullptr, addr(0xf00000), sdv_page_assign_workspace_bytes(a[0]),
                           nullptr);
    } else if (c == "prefix") {
      const sdv_kvcache cache = {SDV_F16,        4096,           a[3],           a[5], a[4], a[7],
                                 addr(0x1000000), addr(0x2000000), addr(0x3000000)};
      st = sdv_prefix_attn(&cache, addr(0x4000000), a[6], addr(0x5000000), addr(0x6000000), (int64_t)a[2] * a[4], a[0],
                           a[1], a[2], addr(0x7000000), nullptr, nullptr, 0.1f, addr(0x8000000), nullptr,
                           addr(0x9000000), sdv_prefix_attn_workspace_bytes(a[0], a[1], a[2], a[3], a[4]), nullptr);
    }
    std::printf("status %d\n", st);
  }
  return 0;
}
