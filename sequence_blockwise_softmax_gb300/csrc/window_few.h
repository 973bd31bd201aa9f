// window_few.h -- the launch of the windowed forward's few-key form, shared
// between its kernel (attn_window_few.cu) and the entry point (attn_window.cu).
#pragma once
#include "ra_internal.h"

namespace ra {

struct WindowFew {
    const uint16_t *q, *k, *v;
    void *o;
    float *lse;
    const int *cu;
    int n_seqs;
    int S, H, Hkv, window, sinks;
    float scale_log2;
    int blocks, max_chunks, heads, group_parts;     // set by the launch
};

// The most dynamic shared memory of a CTA: 227 KB, less 1 KB for the kernel's static
// part.  The limit set on the kernel is this one whatever a call needs, since host
// threads share it: one lowered by another thread's call would refuse the launch.
constexpr size_t kWindowFewSmem = (size_t)226 << 10;

// 16-key chunks a CTA may hold at these sizes, and its shared memory.
int window_few_chunks(int S, int window, int sinks, bool split);
size_t window_few_smem(int chunks, int d, bool split);

// Whether a CTA's warps share 16 rows: the call's CTAs run at once and have more
// than two chunks.
bool window_few_split(int64_t B, int64_t S, int64_t H, int d, int window, int sinks);

ra_status launch_window_few(WindowFew a, int d, bool o_bf16, int64_t B, cudaStream_t stream);

}  // namespace ra
