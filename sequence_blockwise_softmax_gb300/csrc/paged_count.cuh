// paged_count.cuh -- counting a cut pair's pieces in a workspace that other calls
// may have written to.
#pragma once
#include <cuda_runtime.h>

namespace ra {

// The pieces of a pair (or of a unit of rows) are counted in the low bits of a word whose others are the
// call's tag, so that whatever other calls left in the workspace counts as
// nothing; the block that counts the last piece sets the word back to the tag
// and no pieces, where a replay of the same call begins.  A tag's upper half
// is, as fp32, a signalling NaN, which no arithmetic leaves behind: floats that
// other entry points keep in a workspace are never taken for a call's count.
constexpr unsigned long long kCountMask = 1023, kTag = 0xffaull << 52;
__host__ __device__ constexpr unsigned long long call_tag(unsigned long long n) { return kTag | ((n << 10) & ~(0xfffull << 52)); }

__device__ __forceinline__ unsigned long long swap_word(unsigned long long *word, unsigned long long old,
                                                        unsigned long long now) {
    unsigned long long seen;
    asm volatile("atom.cas.acq_rel.gpu.global.b64 %0, [%1], %2, %3;" : "=l"(seen) : "l"(word), "l"(old), "l"(now) : "memory");
    return seen;
}
// A block starts its own word (that of the pair whose first piece it may have)
// as early as it can, so that later counts find the call's tag there.
__device__ __forceinline__ void start_word(unsigned long long *word, unsigned long long call) {
    const unsigned long long old = *reinterpret_cast<volatile unsigned long long *>(word);
    if ((old & ~kCountMask) != call) swap_word(word, old, call);
}
// How many pieces were counted in this word before this one: one add where the
// word has the call's tag.  Where it has not, the add fell on what will be
// replaced; whoever replaces it counts itself, the others add again.
__device__ __forceinline__ int count_piece(unsigned long long *word, unsigned long long call) {
    while (true) {
        unsigned long long old;
        asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(old) : "l"(word) : "memory");
        if ((old & ~kCountMask) == call) return (int)(old & kCountMask);
        unsigned long long seen = *reinterpret_cast<volatile unsigned long long *>(word);
        while ((seen & ~kCountMask) != call) {
            old = seen;
            seen = swap_word(word, old, call + 1);
            if (seen == old) return 0;
        }
    }
}

// The tag of a call, another one for every call of the process (attn_paged_tokens.cu).
unsigned long long next_call_tag();

}  // namespace ra
