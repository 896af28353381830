#pragma once
#include "device.h"

namespace gtp {

// Whether D[m_dim, n_dim] goes to the few-rows kernel (the reasons are beside it).
bool few_rows(int64_t m_dim, int64_t n_dim, int sm_count);

// D[m_dim, n_dim] (bf16) = dq(A) dq(B)^T for m_dim <= 4; arguments checked by the caller.
gtp_status run_mxfp4_rows(const uint8_t *Aq, const uint8_t *As, const uint8_t *Bq, const uint8_t *Bs, void *D,
                          int64_t m_dim, int64_t n_dim, int64_t k_dim, cudaStream_t st);

}  // namespace gtp
