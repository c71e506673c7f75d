// Prompt attention kernels of head dim 128 (one translation unit per head dim, compiled in parallel).
#include "tq_prompt.cuh"

namespace tq {
tq_status launch_prompt_128(const PromptArgs& a, int64_t part_rows, const CUtensorMap& mq, const CUtensorMap& mk,
                            const CUtensorMap& mv, bool bf16, cudaStream_t s) {
    return bf16 ? launch_prompt<PromptCfg<128, true>>(a, part_rows, mq, mk, mv, s)
                : launch_prompt<PromptCfg<128, false>>(a, part_rows, mq, mk, mv, s);
}
}  // namespace tq
