/* A plain C99 caller of the paged cache: include/wall_paged.h must compile as
 * C, every function must resolve at link time, and the host-side checks must
 * answer without a GPU.  Exits 0 when every check holds. */
#include <stdint.h>
#include <stdio.h>

#include "wall_paged.h"

#define CHECK(cond)                                                \
  do {                                                             \
    if (!(cond)) {                                                 \
      fprintf(stderr, "abi_check_paged:%d: %s\n", __LINE__, #cond); \
      return 1;                                                    \
    }                                                              \
  } while (0)

typedef void (*any_fn)(void);

int main(void) {
  void* const fake = (void*)(uintptr_t)4096; /* aligned, never dereferenced */
  int32_t* const fi = (int32_t*)fake;
  int64_t* const fl = (int64_t*)fake;
  float* const ff = (float*)fake;
  const any_fn fns[] = {
      (any_fn)wall_paged_plan,   (any_fn)wall_paged_release, (any_fn)wall_paged_append_workspace,
      (any_fn)wall_paged_append, (any_fn)wall_paged_attn,    (any_fn)wall_paged_attn_workspace,
  };
  for (size_t i = 0; i < sizeof(fns) / sizeof(fns[0]); ++i) CHECK(fns[i] != NULL);
  /* a page size that is not built */
  CHECK(wall_paged_plan(fi, fi, fi, fi, fi, 1, 4, 8, 48, 3, fi, fi, fl, fi, fi, fi, NULL) ==
        WALL_ERR_UNSUPPORTED);
  CHECK(wall_paged_plan(NULL, fi, fi, fi, fi, 1, 4, 8, 64, 3, fi, fi, fl, fi, fi, fi, NULL) ==
        WALL_ERR_INVALID_ARG);
  CHECK(wall_paged_release(fi, fi, fi, fi, fi, -1, 4, 8, 64, NULL) == WALL_ERR_INVALID_ARG);
  CHECK(wall_paged_release(fi, fi, fi, fi, fi, 1, 4, 8, 16, NULL) == WALL_ERR_UNSUPPORTED);
  /* HQ % H != 0; no requests */
  CHECK(wall_paged_append(fake, fake, fake, WALL_BF16, fi, fi, fl, 1, 3, 0, 3, 4, 64, 64, 64, 8,
                          fake, fake, fi, fl, fl, ff, NULL, 0, NULL) == WALL_ERR_INVALID_ARG);
  CHECK(wall_paged_append(fake, fake, fake, WALL_BF16, fi, fi, fl, 0, 0, 0, 2, 4, 64, 64, 64, 8,
                          fake, fake, fi, fl, fl, ff, NULL, 0, NULL) == WALL_OK);
  CHECK(wall_paged_attn(fake, ff, WALL_BF16, fi, fi, fi, 0, 0, 0, 4, 2, 4, 64, 64, 64, 8, fake,
                        fake, fi, NULL, 0.f, 0, fake, NULL, NULL, 0, NULL) == WALL_OK);
  CHECK(wall_paged_attn_workspace(WALL_BF16, 4, 4, 1, 2, 4, 64, 64) > 0);
  CHECK(wall_paged_attn(fake, ff, WALL_BF16, fi, fi, fi, 4, 4, 1, 4, 2, 4, 64, 64, 64, 8, fake,
                        fake, fi, NULL, 0.f, 0, fake, NULL, fake, 8, NULL) == WALL_ERR_INVALID_ARG);
  printf("abi_check_paged: ok (%d entry points)\n", (int)(sizeof(fns) / sizeof(fns[0])));
  return 0;
}
