// Attention of one new token over a cache of this type: see attend_device.h.
#include "attend_device.h"

namespace bd {
namespace attend {

void go_e2m1(const Args& p, bool q_fp32, hipStream_t s) { go_held<BD_E2M1, false>(p, q_fp32, s); }

}  // namespace attend
}  // namespace bd
