// C entry points of the vocabulary-row operators: argument checks (all before
// anything is queued), plans and dispatch by element type.
#include "logits_checks.h"

namespace argr {
namespace {

argr_status check_slots(int64_t rows, const int64_t* ids, const float* teacher, int slots) {
    if (slots < 0 || slots > ARGR_LOGITS_MAX_SLOTS) return ARGR_EINVAL;
    if (rows > 0 && slots > 0 && (!ids || !teacher)) return ARGR_EINVAL;
    return misaligned(ids, 8) || misaligned(teacher, 4) ? ARGR_EINVAL : ARGR_OK;
}

argr_status pick_plan(int what, const argr_plan* given, int64_t rows, int64_t cols, int dtype, int k, argr_plan* p) {
    argr_caps caps;
    argr_status s = current_caps(&caps);
    if (s != ARGR_OK) return s;
    if (!given) return make_logits_plan(what, rows, cols, dtype, k, caps, p);
    *p = *given;
    return check_logits_plan(what, *given, rows, cols, dtype, k, caps);
}

LogitsProblem rows_problem(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride,
                           float temperature, float* stats, argr_stream stream) {
    LogitsProblem pr = {};
    pr.x = x;
    pr.dtype = dtype;
    pr.rows = rows;
    pr.cols = static_cast<int>(cols);
    pr.row_stride = row_stride;
    pr.temperature = temperature;
    pr.inv_t = 1.0f / temperature;
    pr.stats = reinterpret_cast<float4*>(stats);
    pr.stream = reinterpret_cast<cudaStream_t>(stream);
    return pr;
}

#define ARGR_LOGITS_DISPATCH(fn, p, pr)                                   \
    ((pr).dtype == ARGR_F32   ? launched(fn##_f32((p), (pr)))             \
     : (pr).dtype == ARGR_F16 ? launched(fn##_f16((p), (pr)))             \
                              : launched(fn##_bf16((p), (pr))))

}  // namespace
}  // namespace argr

using namespace argr;

extern "C" {

argr_status argreduce_logprobs(const void* x, argr_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                               float temperature, const int64_t* tokens, int32_t top_k, float* logprob,
                               float* entropy, float* lse, int64_t* top_ids, float* top_logprobs, float* stats,
                               const argr_plan* plan, argr_stream stream) {
    argr_status s = check_rows(x, dtype, rows, cols, row_stride, temperature);
    if (s != ARGR_OK) return s;
    if (top_k < 0 || top_k > ARGR_LOGITS_MAX_TOP || top_k > cols) return ARGR_EINVAL;
    if (logprob && !tokens && rows > 0) return ARGR_EINVAL;
    if (misaligned(tokens, 8) || misaligned(top_ids, 8) || misaligned(logprob, 4) || misaligned(entropy, 4) ||
        misaligned(lse, 4) || misaligned(top_logprobs, 4) || misaligned(stats, 16))
        return ARGR_EINVAL;
    if (rows == 0) return ARGR_OK;
    if (!top_ids && !top_logprobs) top_k = 0;
    argr_plan p;
    if ((s = pick_plan(ARGR_LOGITS_LOGPROBS, plan, rows, cols, dtype, top_k, &p)) != ARGR_OK) return s;
    LogitsProblem pr = rows_problem(x, dtype, rows, cols, row_stride, temperature, stats, stream);
    pr.tokens = tokens;
    pr.top_k = top_k;
    pr.logprob = logprob;
    pr.entropy = entropy;
    pr.lse = lse;
    pr.top_ids = top_ids;
    pr.top_logprobs = top_logprobs;
    return ARGR_LOGITS_DISPATCH(launch_logprobs, p, pr);
}

argr_status argreduce_logprobs_backward(const void* x, argr_dtype dtype, int64_t rows, int64_t cols,
                                        int64_t row_stride, float temperature, const int64_t* tokens,
                                        const float* stats, const float* grad_logprob, const float* grad_entropy,
                                        const float* grad_lse, void* grad, int64_t grad_stride,
                                        const argr_plan* plan, argr_stream stream) {
    argr_status s = check_rows(x, dtype, rows, cols, row_stride, temperature);
    if (s != ARGR_OK) return s;
    if (misaligned(tokens, 8) || misaligned(stats, 16) || misaligned(grad_logprob, 4) ||
        misaligned(grad_entropy, 4) || misaligned(grad_lse, 4))
        return ARGR_EINVAL;
    if (rows == 0) return ARGR_OK;
    if (!stats || (grad_logprob && !tokens)) return ARGR_EINVAL;
    if ((s = check_grad(x, dtype, rows, cols, row_stride, grad, grad_stride)) != ARGR_OK) return s;
    argr_plan p;
    if ((s = pick_plan(ARGR_LOGITS_LOGPROBS_GRAD, plan, rows, cols, dtype, 0, &p)) != ARGR_OK) return s;
    LogitsProblem pr =
        rows_problem(x, dtype, rows, cols, row_stride, temperature, const_cast<float*>(stats), stream);
    pr.tokens = tokens;
    pr.grad_logprob = grad_logprob;
    pr.grad_entropy = grad_entropy;
    pr.grad_lse = grad_lse;
    pr.grad = grad;
    pr.grad_stride = grad_stride;
    return ARGR_LOGITS_DISPATCH(launch_logprobs_grad, p, pr);
}

argr_status argreduce_distill(const void* x, argr_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                              float temperature, const int64_t* ids, const float* teacher, int32_t slots, int tail,
                              float* loss, float* stats, const argr_plan* plan, argr_stream stream) {
    argr_status s = check_rows(x, dtype, rows, cols, row_stride, temperature);
    if (s != ARGR_OK || (s = check_slots(rows, ids, teacher, slots)) != ARGR_OK) return s;
    if (misaligned(loss, 4) || misaligned(stats, 16)) return ARGR_EINVAL;
    if (rows == 0) return ARGR_OK;
    argr_plan p;
    if ((s = pick_plan(ARGR_LOGITS_DISTILL, plan, rows, cols, dtype, slots, &p)) != ARGR_OK) return s;
    LogitsProblem pr = rows_problem(x, dtype, rows, cols, row_stride, temperature, stats, stream);
    pr.ids = ids;
    pr.teacher = teacher;
    pr.slots = slots;
    pr.tail = tail != 0;
    pr.loss = loss;
    return ARGR_LOGITS_DISPATCH(launch_distill, p, pr);
}

argr_status argreduce_distill_backward(const void* x, argr_dtype dtype, int64_t rows, int64_t cols,
                                       int64_t row_stride, float temperature, const int64_t* ids,
                                       const float* teacher, int32_t slots, int tail, const float* stats,
                                       const float* grad_loss, void* grad, int64_t grad_stride,
                                       const argr_plan* plan, argr_stream stream) {
    argr_status s = check_rows(x, dtype, rows, cols, row_stride, temperature);
    if (s != ARGR_OK || (s = check_slots(rows, ids, teacher, slots)) != ARGR_OK) return s;
    if (misaligned(stats, 16) || misaligned(grad_loss, 4)) return ARGR_EINVAL;
    if (rows == 0) return ARGR_OK;
    if (!stats || !grad_loss) return ARGR_EINVAL;
    if ((s = check_grad(x, dtype, rows, cols, row_stride, grad, grad_stride)) != ARGR_OK) return s;
    argr_plan p;
    if ((s = pick_plan(ARGR_LOGITS_DISTILL_GRAD, plan, rows, cols, dtype, slots, &p)) != ARGR_OK) return s;
    LogitsProblem pr =
        rows_problem(x, dtype, rows, cols, row_stride, temperature, const_cast<float*>(stats), stream);
    pr.ids = ids;
    pr.teacher = teacher;
    pr.slots = slots;
    pr.tail = tail != 0;
    pr.grad_logprob = grad_loss;
    pr.grad = grad;
    pr.grad_stride = grad_stride;
    return ARGR_LOGITS_DISPATCH(launch_distill_grad, p, pr);
}

argr_status argreduce_distill_step(const void* x, argr_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                                   float temperature, const int64_t* ids, const float* teacher, int32_t slots,
                                   int tail, const float* grad_loss, float* loss, float* stats, void* grad,
                                   int64_t grad_stride, const argr_plan* plan, argr_stream stream) {
    argr_status s = check_rows(x, dtype, rows, cols, row_stride, temperature);
    if (s != ARGR_OK || (s = check_slots(rows, ids, teacher, slots)) != ARGR_OK) return s;
    if (misaligned(loss, 4) || misaligned(stats, 16) || misaligned(grad_loss, 4)) return ARGR_EINVAL;
    if (rows == 0) return ARGR_OK;
    if (!stats || !grad_loss) return ARGR_EINVAL;
    if ((s = check_grad(x, dtype, rows, cols, row_stride, grad, grad_stride)) != ARGR_OK) return s;
    argr_plan p, g;
    if ((s = pick_plan(ARGR_LOGITS_DISTILL_STEP, plan, rows, cols, dtype, slots, &p)) != ARGR_OK) return s;
    LogitsProblem pr = rows_problem(x, dtype, rows, cols, row_stride, temperature, stats, stream);
    pr.ids = ids;
    pr.teacher = teacher;
    pr.slots = slots;
    pr.tail = tail != 0;
    pr.loss = loss;
    pr.grad_logprob = grad_loss;
    pr.grad = grad;
    pr.grad_stride = grad_stride;
    if (p.path == ARGR_PATH_LOGITS_STEP) return ARGR_LOGITS_DISPATCH(launch_distill_step, p, pr);
    // a row too long for the shared memory of a cluster: the two passes
    if ((s = pick_plan(ARGR_LOGITS_DISTILL_GRAD, nullptr, rows, cols, dtype, slots, &g)) != ARGR_OK) return s;
    if ((s = ARGR_LOGITS_DISPATCH(launch_distill, p, pr)) != ARGR_OK) return s;
    return ARGR_LOGITS_DISPATCH(launch_distill_grad, g, pr);
}

argr_status argreduce_logits_plan(argr_logits_op what, int64_t rows, int64_t cols, argr_dtype dtype, int32_t k,
                                  const argr_caps* caps, argr_plan* out) {
    if (!out) return ARGR_EINVAL;
    argr_caps c;
    if (caps) {
        c = *caps;
    } else {
        argr_status s = current_caps(&c);
        if (s != ARGR_OK) return s;
    }
    return make_logits_plan(what, rows, cols, dtype, k, c, out);
}

}  // extern "C"
