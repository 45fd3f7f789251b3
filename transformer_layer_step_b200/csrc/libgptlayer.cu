// The library as one translation unit: the layer step, its optimizer and
// building blocks (gptlayer.cu), then the extensions that use the same
// argument checks, device check and launch recorder: gradient clipping and
// accumulation (optim_ext.cuh), stacks of layers (stack_ext.cuh), and the parts
// around the layer: norm and rotation of queries and keys (qk_rope.cuh),
// dropout (dropout.cuh) and token log probabilities (logprob.cuh).
#include "gptlayer.cu"
#include "optim_ext.cuh"
#include "stack_ext.cuh"
#include "qk_rope.cuh"
#include "dropout.cuh"
#include "logprob.cuh"
