// Attention of a prompt's tokens over a cache of this type: see prompt_device.h.
#include "prompt_device.h"

namespace bd {
namespace prompt {

void go_bf16(const Args& p, unsigned groups, hipStream_t s) { go<BD_BF16, false>(p, groups, s); }

}  // namespace prompt
}  // namespace bd
