// The streaming kernel of the experts for bf16 weight rows.
#include "mol_moe.cuh"

namespace mol {
MOL_MOE_FORMAT(0)
}  // namespace mol
