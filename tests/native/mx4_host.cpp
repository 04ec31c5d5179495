// Host build of the MXFP4 products' index arithmetic (csrc/mx4.h), driven from
// tests/test_mx4_arithmetic.py.
#include "../../fp4_routed_expert_amd/csrc/mx4.h"

// Walks the passes of `rows` rows that start at m0, `stride` apart, up to `end`
// as the streaming product does.  Returns their number, -1 on a pass outside
// [m0, end), -2 where there are more than `most`; *last: the last pass.
extern "C" long host_walk(int m0, int stride, int end, long most, int* last) {
  long n = 0;
  const int begin = m0;
  for (; m0 < end; m0 = moe::next_pass(m0, stride, end)) {
    if (m0 < begin) return -1;
    if (++n > most) return -2;
    *last = m0;
  }
  return n;
}
