#include "fi_delta.h"
extern "C" fi_status fi_delta_backward(const fi_delta_desc *desc, const void *q, const void *k, const void *v, const float *decay,
                            const float *beta, const float *state, const int32_t *lengths, const void *saved,
                            const void *dy, const float *dfinal, void *dq, void *dk, void *dv, float *ddecay,
                            float *dbeta, float *dstate, void *workspace, void *stream) { return FI_EINVAL; }
