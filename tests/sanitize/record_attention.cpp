// A host stand-in for the attention launcher that keeps the arguments which the C entry points derived, for tests of
// what the kernels would be told (linked beside launch_stub.cpp; arrays are host memory, nothing is launched).
#include "launch.h"

namespace w4a4 {

static AttnArgs last;

size_t attention_workspace_bytes(const AttnArgs&, int64_t) { return 256; }

hipError_t launch_attention(AttnArgs a, int, int64_t, void*, hipStream_t) {
  last = a;
  return hipErrorNoDevice;
}

}  // namespace w4a4

// Entries of the page table that the kernels may read: those of the keys below a sequence's length, which they clamp to
// max_len.
extern "C" int64_t attention_table_entries(void) {
  const w4a4::AttnArgs& a = w4a4::last;
  int64_t n = 0;
  for (int s = 0; s < a.batch; ++s) {
    const int64_t len = a.lens[s] < 0 ? 0 : a.lens[s] < a.max_len ? a.lens[s] : a.max_len;
    n += (len + a.page_size - 1) / a.page_size;
  }
  return n;
}
extern "C" int32_t attention_max_len(void) { return w4a4::last.max_len; }
