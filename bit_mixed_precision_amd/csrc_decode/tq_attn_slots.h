// Slots through which the waves of an attention workgroup hand each other their
// parts of rows (tq_attn.hip): plain arithmetic, so that a host compiler can check it.
#pragma once

#ifdef __HIP__
#define TQ_SLOT_FN __host__ __device__ constexpr
#else
#define TQ_SLOT_FN constexpr
#endif

namespace tq {

constexpr int kAttnWaves = 4;
// A wave leaves two parts at most: the end of a row that began before its run
// (part 0; also its only part) and the start of one that goes on after it (part 1).
constexpr int kAttnParts = 2;
constexpr int kAttnSlots = kAttnParts * kAttnWaves;

// The slot of a wave's part.  No other wave writes to it before the workgroup's
// barrier, also not to mark it empty: between that mark and the part itself only
// the order within one wave holds.
TQ_SLOT_FN int attn_slot(int wave, int part) { return kAttnParts * wave + part; }

// Where a slot's sums lie in LDS, in units of one part.  A workgroup with one row
// (direct) has no second parts and no room for them: its slots of part 1 stay empty.
TQ_SLOT_FN int attn_sums_at(bool direct, int slot) { return direct ? slot / kAttnParts : slot; }

}  // namespace tq

#undef TQ_SLOT_FN
