// Token sampling (ql_sample.cu): the internal launch interface.
#pragma once
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace ql {

constexpr int64_t kMaxSampleVocab = 360448;
constexpr float kMinTemperature = 1e-36f;   // below: the arg max (64 log2(e) / T has to be finite)

struct SampleArgs {
    const void* logits;   // [batch][vocab], rows row_stride elements apart
    int dtype;
    int64_t row_stride, batch, vocab;
    const float* temperature;   // [batch] or null, as the next three
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* uniform;       // [batch][uniform_stride]
    int64_t uniform_stride;     // above 1: row b takes number positions[b] % uniform_stride of its row
    const int32_t* positions;
    const int32_t* active;
    int32_t* tokens;
    float* probs;
};
int sample_launch(const SampleArgs& a, cudaStream_t s, bool pdl);

}  // namespace ql
