/* Host-side driver of the validation of the short convolution, the selective scan
 * and the gated feed-forward projections, for a build of the library whose host code
 * carries AddressSanitizer and UndefinedBehaviorSanitizer.  Every call below returns
 * before any HIP call (a query, or arguments that the host refuses: an output lies over
 * an input), so no GPU is needed.  "Device" pointers are aligned fake addresses that the
 * host code never dereferences.  Exit status 0 when every expectation holds. */
#include <stdint.h>
#include <stdio.h>

#include "m3ssm.h"

static int fails = 0;
static size_t calls = 0;
#define REFUSED(c)                                                                        \
  do {                                                                                    \
    const m3_status st_ = (c);                                                            \
    ++calls;                                                                              \
    if (st_ != M3_ERR_INVALID_VALUE && st_ != M3_ERR_NOT_SUPPORTED && st_ != M3_ERR_WORKSPACE) { \
      fprintf(stderr, "FAIL %s:%d: %s gave %d\n", __FILE__, __LINE__, #c, (int)st_);      \
      ++fails;                                                                            \
    }                                                                                     \
  } while (0)

#define N_OF(a) (sizeof(a) / sizeof *(a))
static const int64_t sizes[] = {-1, 0, 1, 3, 64, 1001, 1ll << 22, 1ll << 31, 1ll << 40, INT64_MAX};
static const int64_t lds[] = {-1, 0, 64, 1001, 4194303, 1ll << 40, INT64_MAX};
static const int64_t small[] = {-1, 0, 1, 2, 4, 5, 16, 64, 65, INT64_MAX};

/* The i-th array of a call, 2^44 bytes from the next. */
static void* at(int i) { return (void*)(uintptr_t)(((uintptr_t)(i + 1) << 44) + 0x10000u); }
static float* fat(int i) { return (float*)at(i); }
static const int32_t* iat(int i) { return (const int32_t*)at(i); }

static void convs(void) {
  for (size_t b = 0; b < N_OF(sizes); ++b)
    for (size_t t = 0; t < N_OF(sizes); ++t)
      for (size_t d = 0; d < N_OF(sizes); ++d)
        for (size_t w = 0; w < N_OF(small); ++w)
          for (int dt = 0; dt < 2; ++dt) {
            m3_conv_dims s = {sizes[b], sizes[t], sizes[d], small[w], lds[(t + d) % N_OF(lds)], lds[d % N_OF(lds)]};
            if (sizes[b] == 0) continue; /* an empty batch passes */
            /* state_out over state_in, y over x */
            REFUSED(m3_causal_conv(&s, (m3_dtype)dt, at(0), fat(1), fat(2), 1, at(3), iat(4), at(5), at(3), NULL));
            if (sizes[t] > 0)
              REFUSED(m3_causal_conv(&s, (m3_dtype)dt, at(0), fat(1), fat(2), 1, at(3), iat(4), at(0), at(6), NULL));
            if (sizes[t] != 0) /* (a pool of none passes) */
              REFUSED(m3_causal_conv_step(&s, (m3_dtype)dt, at(0), iat(1), sizes[t], at(0), fat(3), fat(4), 0, at(5),
                                          NULL));
          }
}

static void scans(void) {
  for (size_t b = 0; b < N_OF(sizes); ++b)
    for (size_t t = 0; t < N_OF(sizes); ++t)
      for (size_t d = 0; d < N_OF(sizes); ++d)
        for (size_t n = 0; n < N_OF(small); ++n)
          for (int dt = 0; dt < 2; ++dt) {
            const int64_t l = lds[(t + d) % N_OF(lds)], k = lds[n % N_OF(lds)];
            m3_select_dims s = {sizes[b], sizes[t], sizes[d], small[n], l, 0, l, 0, k, 0};
            (void)m3_selective_scan_workspace_size(&s, (m3_dtype)dt);
            ++calls;
            if (sizes[b] == 0 || sizes[t] == 0) continue;
            /* y over x, h_last over h0, the workspace over B */
            REFUSED(m3_selective_scan(&s, (m3_dtype)dt, at(0), at(1), fat(2), at(3), at(4), fat(5), at(6), fat(7), 1,
                                      fat(8), iat(9), at(0), fat(11), at(12), SIZE_MAX, NULL));
            REFUSED(m3_selective_scan(&s, (m3_dtype)dt, at(0), at(1), fat(2), at(3), at(4), fat(5), at(6), fat(7), 1,
                                      fat(8), iat(9), at(10), fat(8), at(12), SIZE_MAX, NULL));
            REFUSED(m3_selective_scan_step(&s, (m3_dtype)dt, fat(0), iat(1), sizes[t], at(2), at(3), fat(4), at(5),
                                           at(6), fat(7), at(8), fat(9), 1, at(0), NULL));
          }
}

static void ffns(void) {
  for (size_t m = 0; m < N_OF(sizes); ++m)
    for (size_t k = 0; k < N_OF(sizes); ++k)
      for (size_t f = 0; f < N_OF(sizes); ++f)
        for (size_t l = 0; l < N_OF(lds); ++l)
          for (int dt = 0; dt < 2; ++dt) {
            m3_ffn_dims s = {sizes[m], sizes[k], sizes[f], lds[l], 0, lds[l], 0, lds[l], 0, 0, lds[l], 0, lds[l]};
            (void)m3_gated_ffn_backward_workspace_size(&s, (m3_dtype)dt);
            ++calls;
            if (sizes[m] != 0)
              REFUSED(m3_gated_ffn(&s, (m3_dtype)dt, at(0), at(1), at(2), at(1), fat(4), fat(5), NULL));
            /* both weights' gradients in one place */
            REFUSED(m3_gated_ffn_backward(&s, (m3_dtype)dt, at(0), at(1), at(2), at(3), fat(4), fat(5), at(6), at(7),
                                          at(7), at(8), SIZE_MAX, NULL));
            if (sizes[m] != 0)
              REFUSED(m3_gated_ffn_backward(&s, (m3_dtype)dt, at(0), at(1), at(2), at(3), fat(4), fat(5), at(6), at(7),
                                            at(8), at(2), SIZE_MAX, NULL));
          }
}

int main(void) {
  convs();
  scans();
  ffns();
  printf("driver_selective_abi: %zu calls, %d failures\n", calls, fails);
  return fails ? 1 : 0;
}
