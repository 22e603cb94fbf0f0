// Attention of a prompt's tokens with formed scores over a cache of this type: see prompt_device.h.
#include "prompt_device.h"

namespace bd {
namespace prompt {

void go_bf16_formed(const Args& p, unsigned groups, hipStream_t s) { go<BD_BF16, true>(p, groups, s); }

}  // namespace prompt
}  // namespace bd
