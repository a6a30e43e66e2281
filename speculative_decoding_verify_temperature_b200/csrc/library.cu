// library.cu -- the translation unit of the verify kernels (spec_verify.cu) and
// of the host-side services that the cache calls share with them: both report
// through spec_last_error_detail() and spec_launch_count().
#include "spec_verify.cu"

#include "internal.h"

namespace sv_host {

spec_status fail(spec_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_detail, sizeof g_detail, fmt, ap);
    va_end(ap);
    return st;
}
spec_status launched(const char* what) { return ::launched(what); }
int num_sms() { return ::num_sms(); }
unsigned wait_tries() { return g_wait_tries; }
void range_push(const char* name) { nvtxRangePushA(name); }
void range_pop() { nvtxRangePop(); }

}  // namespace sv_host
