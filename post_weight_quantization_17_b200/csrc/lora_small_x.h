// Which 16 bytes of its token's row a lane of k_lora_small loads ahead.
#pragma once

namespace gptq {

// A lane holds columns 32 t4 .. 32 t4 + 31 of each 128-column step and loads them 8 at a time: piece q
// of step s, counted on into the step after (q 4 and up), or into this one once more where the warp's
// last step is s1 - 1.  Returns the piece's distance, in 8 columns, from the lane's columns of step s, or
// -1 where the step that is read is the `ragged` one (the last of a row of d columns that is no multiple
// of 128; -1: none) and the piece lies behind column d: nothing is read there.
__host__ __device__ inline int small_x_piece(int d, int s, int q, int s1, int ragged, int t4) {
  const int next = q >= 4 && s + 1 < s1 ? 1 : 0;
  if (s + next == ragged && (s + next) * 128 + t4 * 32 + 8 * (q & 3) >= d) return -1;
  return next * 16 + (q & 3);
}

}  // namespace gptq
