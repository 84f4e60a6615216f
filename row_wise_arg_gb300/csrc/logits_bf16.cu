// Vocabulary-row kernels of one element type.
#include "logits_impl.cuh"

ARGR_DEFINE_LOGITS(bf16, argr::TagBF16)
