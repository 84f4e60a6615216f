// Beam selection and routing of one element type.
#include "beam_select.cuh"
#include "route.cuh"

ARGR_DEFINE_SELECT(bf16, argr::TagBF16, ARGR_BF16)
