/*
 * mok_profile.h - optional timing hooks of libmok (no counterpart in the articles; used
 * by benchmarks to attribute time to the library's kernels inside a timed region).
 *
 * When enabled on a context, every kernel launch made by later mok_plan / mok_moe_fwd /
 * mok_moe_bwd calls is bracketed by two CUDA events recorded on the launch stream, and
 * the forward megakernel stamps its phases per CTA (%globaltimer) into a small device
 * buffer that mok_profile_enable allocates once per context (64 launches x SMs x 64 bytes;
 * freed by mok_destroy). Recording adds a few microseconds per launch.
 *
 * mok_lora_get_forms says which of its kernels' forms a call of mok_ops.h would run, for tests
 * that have to reach one and for profiles.
 */
#ifndef MOK_PROFILE_H_
#define MOK_PROFILE_H_

#include <stddef.h>

#include "mok.h"
#include "mok_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* enable != 0: start recording (clears earlier records); 0: stop. */
mok_status mok_profile_enable(mok_ctx_t ctx, int enable);

/* Synchronise the recorded events and write one line per kernel name,
 * "<name> <launches> <total_ms>\n", into buf (NUL-terminated, truncated to len), then
 * the megakernel's phases as "fwd_megakernel:<phase> <launches> <total_ms>" lines
 * (gather, gemm, gemm_spread, combine, total; measured from the kernel's first CTA start).
 * *total_launches receives the number of kernel launches recorded. Records are cleared.
 * Returns MOK_ERR_CUDA if enabling could not allocate the stamp buffer. */
mok_status mok_profile_report(mok_ctx_t ctx, char* buf, size_t len, int* total_launches);

/* A projection: tiles of 128 rows and `columns` columns; `split` CTAs share a tile's contraction;
 * pair: SM pairs, 256 rows, whose last `halved` tiles are run as two halves of the width. */
typedef struct {
  int columns, split, pair, halved;
} mok_lora_proj_form;

typedef struct {
  mok_lora_proj_form proj;     /* the shared projection (y, dX)                              */
  mok_lora_proj_form adapters; /* own_input: the product of its own that gives dXa           */
  int u_ranks;                 /* u (v): ranks a CTA where found row by row, 0: in tiles ... */
  int u_split, u_chunks;       /* ... CTAs that share a contraction, clusters that share a
                                * tile's adapters                                            */
  int grad_columns, grad_split; /* weight gradients: columns of a CTA, CTAs that share rows  */
} mok_lora_forms;

/* The forms of mok_lora_fwd (backward = 0) or mok_lora_bwd for these dims on the current device;
 * own_input != 0: with x_ad. Parts that the call does not have are 0. */
mok_status mok_lora_get_forms(const mok_lora_dims* dims, int backward, int own_input,
                              mok_lora_forms* out);

#ifdef __cplusplus
}
#endif
#endif /* MOK_PROFILE_H_ */
