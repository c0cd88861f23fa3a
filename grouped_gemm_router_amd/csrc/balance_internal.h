// balance_internal.h -- host launchers of balance.hip.  Arguments are
// validated by the C-ABI layer before these are called.
#pragma once

#include "moe_internal.h"
#include "../../include/moe_balance.h"

size_t balance_loss_ws_bytes(int T, int E, int S);
hipError_t launch_balance_loss(const float *logits, const int32_t *topk_idx, const int32_t *off,
                               const uint8_t *mask, int T, int E, int k, int S, float alpha,
                               int32_t *counts, float *probs, int32_t *tokens, float *loss, void *ws,
                               hipStream_t s);
hipError_t launch_route_backward(const float *logits, const int32_t *topk_idx, const float *dw,
                                 bool renorm, const int32_t *counts, const int32_t *tokens,
                                 float alpha, const float *d_loss, const int32_t *off,
                                 const uint8_t *mask, int T, int E, int k, int S, float *d_logits,
                                 hipStream_t s);
