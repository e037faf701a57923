// Where the forward pass of the balance loss leaves its sums of q (one value a token)
// and where the loss of a sequence finds them; plain functions, for host and device.
//
// A block's waves take `run` tokens each, a block ROW_WAVES times as many.  The sum over
// the tokens of a block that are in the sequence of its first token lies at that token.
// In the block that a sequence begins in behind the first token, every wave left a sum
// of its own, at the later of its own and the sequence's first token.
#pragma once

namespace qmoe {

constexpr int ROW_WAVES = 16;  // of a block of the forward pass

// Tokens of a wave: as many as make one round of waves (without tokens there are still
// sequences, whose sums are looked for).
constexpr int run_of(int T) { return T > 0 ? (T + 8191) / 8192 : 1; }

// The first block whose first token is not in front of token `first`.
constexpr int block_from(int first, int run) { return (first + ROW_WAVES * run - 1) / (ROW_WAVES * run); }

// The place of the sum that wave `wave` of the block before left for the tokens [first,
// end) of a sequence, or -1 (an empty sequence has none, at the last token neither).
constexpr int wave_place(int first, int end, int wave, int run) {
  const int block = block_from(first, run), at = (block - 1) * ROW_WAVES * run + wave * run;
  const bool any = first < end && first < block * ROW_WAVES * run && at + run > first && at < end;
  return !any ? -1 : at > first ? at : first;
}

}  // namespace qmoe
