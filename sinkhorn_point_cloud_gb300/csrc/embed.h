// embed.h -- launch interface of the embedding lookup and of its gradient.
#pragma once
#include <cuda_runtime.h>

namespace sot {

struct EmbedArgs {
    const void* table;  // [V, D], row v at element v * ld
    long long T, ld, ldo;
    int V, D, type, out_type;
    const void* ids;
    int ids_type;
    float scale;
    void* out;  // [T, D]
};

struct EmbedGradArgs {
    const void* g;  // [T, D], row t at element t * ld
    long long T, ld, ldg;
    int V, D, type, grad_type;
    const void* ids;
    int ids_type;
    float scale;
    int accumulate;
    void* grad;  // [V, D]
    int chunk;   // sorted tokens of a chunk
    // scratch: (row, token) sorted by row (two buffers), the chunks where a row begins that goes on in the next and that row,
    // a bit for each row that a token names, partial sums
    uint2* sorted[2];
    unsigned *spans, *named;
    uint2* span;
    float* part;
};

struct EmbedGradPlan {
    int passes, bits;  // of the sort
    long long chunks;
    int chunk;  // tokens of one
    size_t sorted_at[2], spans_at, span_at, named_at, part_at, scratch;
};
EmbedGradPlan embed_grad_plan(long long T, int V, int D);
cudaError_t launch_embed(const EmbedArgs& a, int sms, cudaStream_t st);
cudaError_t launch_embed_grad(EmbedGradArgs a, const EmbedGradPlan& p, unsigned char* scratch, int sms, cudaStream_t st);

}  // namespace sot
