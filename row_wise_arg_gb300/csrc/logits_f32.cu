// Vocabulary-row kernels of one element type.
#include "logits_impl.cuh"

ARGR_DEFINE_LOGITS(f32, argr::TagF32)
