// Slots and barriers of the code units that k_lora_tc copies ahead.  Two groups of weight warps take the
// units in turn (unit u: group u & 1), so neither sees every fill of a slot when their number is odd: a
// parity wait of a group that saw fill n of a slot's barrier, but not n + 1, returns at once while the
// barrier is still in phase n + 1, and copies may land out of order.  So every barrier belongs to one
// group: unit u lies in slot u % slots and is counted on barrier u % barriers, an even multiple.
#pragma once

namespace gptq {

constexpr int kLoraCodeSlotsForward = 3, kLoraCodeSlotsBackward = 6;
constexpr int lora_code_barriers(int slots) { return slots % 2 ? 2 * slots : slots; }

}  // namespace gptq
