// Driver for the AddressSanitizer + UndefinedBehaviorSanitizer build of the
// host code of mxfp4.h, run by tests/test_fp4_sanitizers.py on a machine
// without a GPU.  Sizes come from extreme sets; every call holds at least one
// argument that the header rejects, so that none reaches a launch (one that did
// would report MX_ERR_HIP, a failure here).  Exit status 0: clean.
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "mxfp4.h"

namespace {

int failures = 0;
long calls = 0;

void rejected(mx_status st, const char* what, int64_t a, int64_t b, int64_t c) {
  ++calls;
  if (st == MX_OK || st == MX_ERR_HIP || st < MX_OK || st > MX_ERR_WORKSPACE) {
    fprintf(stderr, "%s(%lld, %lld, %lld) -> %d\n", what, (long long)a, (long long)b, (long long)c, (int)st);
    ++failures;
  }
}

// no size of any argument
const std::vector<int64_t> kBad = {-1, -32, ((int64_t)1 << 40) + 32, (int64_t)1 << 41, INT64_MAX, INT64_MIN,
                                   INT64_MAX - 127, INT64_MAX - 31, (int64_t)1 << 62, -((int64_t)1 << 62)};
const std::vector<int64_t> kAny = {0, 32, 64, 4096, INT32_MAX - 31, (int64_t)1 << 31, INT64_MAX - 31, INT64_MIN};
const std::vector<int32_t> kTypes = {0, 1};

uint8_t* const P = reinterpret_cast<uint8_t*>(0x10000);   // aligned, never dereferenced
const int32_t* const E = reinterpret_cast<int32_t*>(0x10000);

// bad in one place, any in the others
void sizes(int64_t a, int64_t b, int64_t c) {
  for (int32_t f : kTypes) {
    rejected(mx_gemm_mxfp4(P, P, f, P, P, a, b, c, P, 0, nullptr), "mx_gemm_mxfp4", a, b, c);
    rejected(mx_grouped_gemm_mxfp4(P, P, f, P, P, E, 1024, a, b, c, P, 1, nullptr), "mx_grouped_gemm_mxfp4", a, b, c);
    rejected(mx_linear_decode(P, INT32_MAX, P, P, f, a, b, c, P, 0, nullptr), "mx_linear_decode", a, b, c);
    rejected(mx_gated_ffn_decode(P, INT64_MAX, P, P, f, a, b, c, f, P, nullptr), "mx_gated_ffn_decode", a, b, c);
    rejected(mx_gated_ffn(P, P, f, P, P, 1, nullptr, 1, a, b, c, f, P, P, P, nullptr), "mx_gated_ffn", a, b, c);
    rejected(mx_gated_ffn(P, P, 0, P, P, f, E, 1024, a, b, c, f, P, P, P, nullptr), "mx_gated_ffn", a, b, c);
    rejected(mx_gated_ffn_backward(P, P, f, P, P, 1, E, 7, a, b, c, f, P, P, P, P, nullptr), "mx_gated_ffn_backward", a,
             b, c);
    rejected(mx_cast_mxfp4(P, f, a, b, c, c, P, P, P, P, f, nullptr), "mx_cast_mxfp4", a, b, c);
    rejected(mx_dequantize_mxfp4(P, P, a, b, c, f, P, f, nullptr), "mx_dequantize_mxfp4", a, b, c);
  }
}

}  // namespace

int main() {
  for (int64_t bad : kBad)
    for (int64_t x : kAny)
      for (int64_t y : kAny) {
        sizes(bad, x, y);
        sizes(x, bad, y);
        sizes(x, y, bad);
      }
  for (int32_t g : {-1, 0, 1025, INT32_MAX, INT32_MIN})
    for (int64_t x : kAny) {
      rejected(mx_grouped_gemm_mxfp4(P, P, 1, P, P, E, g, x, 32, 32, P, 0, nullptr), "groups", g, x, 0);
      rejected(mx_gated_ffn(P, P, 1, P, P, 1, E, g, x, 32, 32, 0, P, P, P, nullptr), "groups", g, x, 1);
      rejected(mx_gated_ffn_backward(P, P, 1, P, P, 1, E, g, x, 32, 32, 0, P, P, P, P, nullptr), "groups", g, x, 2);
    }
  for (int64_t ld : {INT64_MIN, (int64_t)-1, (int64_t)31, INT64_MAX}) {
    rejected(mx_cast_mxfp4(P, 0, 1, 32, 32, ld, P, P, P, P, 0, nullptr), "ldx", ld, 0, 0);
    rejected(mx_linear_decode(P, ld, P, P, 1, 1, 32, 32, P, 0, nullptr), "ldx", ld, 0, 1);
  }
  if (failures) {
    fprintf(stderr, "%d of %ld calls not rejected\n", failures, calls);
    return 1;
  }
  printf("fp4 sanitizer run clean (%ld calls)\n", calls);
  return 0;
}
