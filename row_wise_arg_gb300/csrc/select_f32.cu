// Beam selection and routing of one element type.
#include "beam_select.cuh"
#include "route.cuh"

ARGR_DEFINE_SELECT(f32, argr::TagF32, ARGR_F32)
