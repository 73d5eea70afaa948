// The streaming kernel of the experts for 4-bit weight rows, a scale for every 32 inputs.
#include "mol_moe.cuh"

namespace mol {
MOL_MOE_FORMAT(32)
}  // namespace mol
