// The operators' shared host state: the calling thread's error message.
#include "fi_ops.h"

namespace fi {

char *op_error() {
    static thread_local char msg[kOpErrorBytes] = "";
    return msg;
}

}  // namespace fi

extern "C" const char *fi_op_last_error(void) { return fi::op_error(); }
