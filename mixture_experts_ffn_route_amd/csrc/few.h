// Launch interface of the few-token layer (few.hip).
#pragma once

#include "internal.h"

namespace moe {

struct FewArgs {
  const void *x;
  int T, d, E, k, I, G, kept, score, renorm, route_mode;
  float route_scale, limit;
  int has_shared;
  const void *gate_w;
  const float *bias;
  const int32_t *token_ids, *tid2eid;
  int64_t vocab;
  int64_t primes[16];                          // 2-gram hash
  const void *w_gate, *w_up, *w_down;
  const uint8_t *s_gate, *s_up, *s_down;
  const void *sh_gate, *sh_up, *sh_down;
  // workspace
  float *out_w;                                // [T, k] gate values
  int32_t *out_e;                              // [T, k] expert ids
  uint32_t *flags;                             // [4]
  float *scores;                               // [KS, T, E] partial gate logits
  int KS;
  uint8_t *xq, *xq_scales;                     // MXFP8 layers, else null
  void *h, *h_lo;                              // [T*k + T, I] SwiGLU output
  uint8_t *hq, *hq_scales;                     // [T*k, I] MXFP8 layers
  int32_t *plan_slots, *plan_expert;           // the distinct chosen experts
  float *plan_w;                               // [slots, 16]
  int16_t *plan_row;                           // [slots, 16]
  int32_t *plan_mask;                          // [T] choices that hold a row
  float *yrows;                                // [T*k + T, d] weighted expert outputs
  void *y;
  int score_items, small_gate;                 // set by launch_few
};

int few_logit_parts(int d, bool f32);
hipError_t launch_few(FewArgs a, const moe_config &cfg, hipStream_t s);

}  // namespace moe
