// The tree kinds of the chunk kernel: attention of a drafted tree's nodes to the
// cached context and to what their masks name of the tree (pa_tree_attention).
// A file of their own so that they compile beside the other kinds.
#include "pa_prefill_kernel.cuh"

namespace pa {

// type: (stream-K, FP8 cache, head size 64, bf16), highest bit first.
const void *tree_kernel(bool solo, int type)
{
#define PA_TREE_INSTANCES(SK, KIND)                                                              \
    reinterpret_cast<const void *>(&paged_prefill_kernel<false, false, 128, SK, KIND>),          \
        reinterpret_cast<const void *>(&paged_prefill_kernel<true, false, 128, SK, KIND>),       \
        reinterpret_cast<const void *>(&paged_prefill_kernel<false, false, 64, SK, KIND>),       \
        reinterpret_cast<const void *>(&paged_prefill_kernel<true, false, 64, SK, KIND>),        \
        reinterpret_cast<const void *>(&paged_prefill_kernel<false, true, 128, SK, KIND>),       \
        reinterpret_cast<const void *>(&paged_prefill_kernel<true, true, 128, SK, KIND>),        \
        reinterpret_cast<const void *>(&paged_prefill_kernel<false, true, 64, SK, KIND>),        \
        reinterpret_cast<const void *>(&paged_prefill_kernel<true, true, 64, SK, KIND>)
    static const void *const kernels[32] = {PA_TREE_INSTANCES(false, kTree), PA_TREE_INSTANCES(true, kTree),
                                            PA_TREE_INSTANCES(false, kTreeSolo), PA_TREE_INSTANCES(true, kTreeSolo)};
#undef PA_TREE_INSTANCES
    return kernels[(solo ? 16 : 0) + type];
}

int tree_attention_take_device_error(int *bits)
{
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_prefill_error, sizeof(int));
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbol(g_prefill_error, &zero, sizeof(int));
    *bits = e == cudaSuccess ? v : 0;
    return (int)e;
}

}  // namespace pa
