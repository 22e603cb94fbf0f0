// Attention of one new token with formed scores over a cache of this type: see attend_device.h.
#include "attend_device.h"

namespace bd {
namespace attend {

void go_bf16_formed(const Args& p, bool q_fp32, hipStream_t s) { go_held<BD_BF16, true>(p, q_fp32, s); }

}  // namespace attend
}  // namespace bd
