// The rings of the block-scaled product on tcgen05 (block_fp8_tc.cu): stages of
// copied operands and accumulation buffers in tensor memory. Plain C++, so that
// the barrier schedule that follows from these numbers can be checked on a host.
//
// Block i of a CTA's contraction uses stage i mod stages and buffer i mod
// buffers, and issuing thread i mod kTcIssuers. A wait on a barrier by parity
// tells a phase only from its neighbours: it returns at once where the phase
// BEFORE the one meant is still open. So whoever waits has to have seen the
// phase before, which an issuing thread has only if every block of a stage (and
// of a buffer) is its own: stages and buffers are multiples of the issuers.
// (With 5 stages a stage's blocks go to the two threads in turn; where the copy
// of block 0 lands after those of blocks 1 and 3, the odd thread's wait for
// block 5 returns before block 0 has landed, and its product then reads a stage
// that does not hold block 5.)
#pragma once

namespace moe {

constexpr int kTcIssuers = 2;

// By tile width: the most that shared memory holds. (128 columns by one CTA a tile:
// 390 ns a block with four stages, 310 with six.)
constexpr int tc_stages(int bn) { return bn == 256 ? 4 : 6; }
constexpr int tc_buffers(int bn) { return 512 / bn < 4 ? 512 / bn : 4; }

}  // namespace moe
