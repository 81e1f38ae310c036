// Launch of a kernel that follows another one of the same call in its stream.
#pragma once
#include <cuda_runtime.h>

namespace m2rnn {

// The kernel may be set up (CTAs placed, prologue run) once every CTA of the
// one before has called cudaTriggerProgrammaticLaunchCompletion() or ended; it
// calls cudaGridDependencySynchronize(), which waits for that kernel's end and
// its writes, before it touches what that kernel reads or writes.  A kernel
// that is launched so waits before its own trigger, so whatever follows it is
// ordered behind everything before it.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, A&&... args) {
    cudaLaunchAttribute a = {};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &a;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

}  // namespace m2rnn
