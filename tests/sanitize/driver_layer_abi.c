/* Host-side driver of the layer operators' validation, for a build of the
 * library whose host code carries AddressSanitizer and UndefinedBehavior-
 * Sanitizer.  Every call below returns before any HIP call (a query, or
 * arguments that the host refuses: an output lies over an input), so no GPU is
 * needed.  "Device" pointers are aligned fake addresses that the host code never
 * dereferences.  Exit status 0 when every expectation holds. */
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

/* The i-th array of a call, 2^44 bytes from the next. */
static void* at(int i) { return (void*)(uintptr_t)(((uintptr_t)(i + 1) << 44) + 0x10000u); }
static float* fat(int i) { return (float*)at(i); }

static void scans(void) {
  for (size_t b = 0; b < N_OF(sizes); ++b)
    for (size_t t = 0; t < N_OF(sizes); ++t)
      for (size_t d = 0; d < N_OF(sizes); ++d)
        for (size_t l = 0; l < N_OF(lds); ++l)
          for (int dt = 0; dt < 2; ++dt) {
            m3_scan_dims s = {sizes[b], sizes[t], sizes[d], lds[l], 0, lds[l], 0, lds[l], 0, lds[l]};
            (void)m3_gated_scan_workspace_size(&s, (m3_dtype)dt);
            ++calls;
            if (sizes[b] == 0) continue; /* an empty batch passes */
            if (sizes[t] != 0) {         /* (no tokens: the states are moved) */
              /* y over x, h_last over h0, states over the workspace, all at one place */
              REFUSED(m3_gated_scan(&s, (m3_dtype)dt, at(0), at(1), at(2), fat(3), at(0), fat(3), fat(7), at(7),
                                    SIZE_MAX, NULL));
              REFUSED(m3_gated_scan(&s, (m3_dtype)dt, at(0), at(1), at(2), fat(3), at(4), fat(4), fat(6), at(7),
                                    SIZE_MAX, NULL));
              REFUSED(m3_gated_scan_backward(&s, (m3_dtype)dt, at(0), at(1), at(2), at(3), fat(4), fat(5), at(6),
                                             at(7), at(7), fat(9), at(10), SIZE_MAX, NULL));
              REFUSED(m3_gated_scan_backward(&s, (m3_dtype)dt, at(0), at(1), at(2), at(3), fat(4), fat(5), at(6),
                                             at(4), at(8), fat(9), at(10), SIZE_MAX, NULL));
            }
            REFUSED(m3_gated_scan_step(&s, (m3_dtype)dt, fat(0), fat(1), at(2), at(3), at(4), at(1), NULL));
          }
}

static void norms(void) {
  for (size_t r = 0; r < N_OF(sizes); ++r)
    for (size_t d = 0; d < N_OF(sizes); ++d)
      for (size_t l = 0; l < N_OF(lds); ++l)
        for (size_t k = 0; k < N_OF(lds); ++k)
          for (int dt = 0; dt < 2; ++dt) {
            m3_norm_dims n = {sizes[r], sizes[d], lds[l], lds[k], lds[l], lds[k], lds[l], lds[k], lds[l]};
            (void)m3_layer_norm_backward_workspace_size(&n, (m3_dtype)dt);
            ++calls;
            if (sizes[r] != 0)
              REFUSED(m3_layer_norm(&n, (m3_dtype)dt, at(0), at(1), fat(2), fat(3), 1e-5f, at(4), at(4), fat(6),
                                    fat(7), NULL));
            REFUSED(m3_layer_norm_backward(&n, (m3_dtype)dt, at(0), at(1), fat(2), fat(3), fat(4), at(5), at(6),
                                           fat(7), fat(7), at(8), SIZE_MAX, NULL));
          }
}

static void caches(void) {
  static const int64_t ns[] = {0, 2, 15, 34, 128, 256, 512};
  static const int64_t ps[] = {8, 16, 64, 128};
  for (size_t b = 0; b < N_OF(sizes); ++b)
    for (size_t h = 0; h < N_OF(sizes); ++h)
      for (size_t n = 0; n < N_OF(ns); ++n)
        for (size_t p = 0; p < N_OF(ps); ++p)
          for (size_t s = 0; s < N_OF(sizes); ++s) {
            m3_dims d = {sizes[b], 1, sizes[h], ps[p], ns[n], 2};
            if (sizes[b] == 0) continue; /* an empty batch passes */
            if (sizes[s] != 0) {         /* and so does an empty pool */
              REFUSED(m3_state_store(&d, M3_CODE_E4M3, fat(0), at(1), fat(1), (int32_t*)at(3), sizes[s], NULL));
              REFUSED(m3_state_load(&d, M3_CODE_INT8, M3_BF16, at(1), fat(2), (int32_t*)at(3), sizes[s], at(2),
                                    NULL));
              REFUSED(m3_decode_step_cached(&d, M3_BF16, M3_CODE_INT8, at(0), fat(1), (int32_t*)at(2), sizes[s],
                                            at(3), at(4), at(5), at(6), at(7), fat(8), fat(9), fat(10), fat(11),
                                            at(11), NULL));
            }
          }
}

int main(void) {
  scans();
  norms();
  caches();
  m3_scan_dims s = {2, 300, 64, 0, 0, 0, 0, 0, 0, 0};
  REFUSED(m3_gated_scan(NULL, M3_F32, at(0), at(1), NULL, NULL, at(4), NULL, NULL, at(5), SIZE_MAX, NULL));
  REFUSED(m3_gated_scan(&s, (m3_dtype)-7, at(0), at(1), NULL, NULL, at(4), NULL, NULL, at(5), SIZE_MAX, NULL));
  /* the last byte of the address space */
  REFUSED(m3_gated_scan_step(&s, M3_BF16, fat(0), fat(1), (void*)(UINTPTR_MAX - 1), at(3), NULL,
                             (void*)(UINTPTR_MAX - 1), NULL));
  printf("driver_layer_abi: %zu calls, %d failures\n", calls, fails);
  return fails ? 1 : 0;
}
