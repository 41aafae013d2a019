// Which kernel takes a grouped bf16 product.  Plain C++, so that the host's
// tests can ask for the choice that the launch makes.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {
namespace bf16 {

enum Mode { kPlain = 0, kGlu = 1, kDgrad = 2, kDgradGlu = 3, kWgrad = 4 };

}  // namespace bf16
}  // namespace moe
