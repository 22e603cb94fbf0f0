// Attention of a prompt's tokens with formed scores over a cache of this type: see prompt_device.h.
#include "prompt_device.h"

namespace bd {
namespace prompt {

void go_e2m1_formed(const Args& p, unsigned groups, hipStream_t s) { go<BD_E2M1, true>(p, groups, s); }

}  // namespace prompt
}  // namespace bd
