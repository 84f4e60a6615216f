// Beam selection and routing of one element type.
#include "beam_select.cuh"
#include "route.cuh"

ARGR_DEFINE_SELECT(f16, argr::TagF16, ARGR_F16)
