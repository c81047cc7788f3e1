// What the translation units of the C ABI (api.cu, api_paged.cu) share.
#pragma once

#include "gqa.h"
#include "kernels.h"

namespace gqa {

// SM count the workspace sizing assumes (GB300); launches use at most this many.
constexpr int REF_SMS = 152;
int sm_count();    // of the current device
int launch_sms();  // min(sm_count(), REF_SMS)

bool aligned16(const void* p);
int fail_cuda(cudaError_t e);                // remembers e for gqa_strerror; GQA_ECUDA
unsigned long long wait_limit_ns();          // gqa_set_wait_limit_ns of this thread
void begin_call();                           // no kernel enqueued yet by the current call
int launched(cudaError_t e);                 // counts a launch that returned e; GQA_OK or GQA_ECUDA
void prof_mark(int i, cudaStream_t s);       // gqa_set_profile_events: event i, if set
bool encode_bf16(CUtensorMap* m, cuuint32_t rank, const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box);
bool encode_bytes(CUtensorMap* m, cuuint32_t rank, const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
                  const cuuint32_t* box);

}  // namespace gqa
