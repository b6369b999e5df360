// The bits that kernels record in the device status words, and what gdn_device_status says of them.
// Plain C++, so that what is said can be tested without a device.
#pragma once

#include <string>

namespace gdn {

constexpr int kDevErrTimeout = 1;      // a wait for an asynchronous copy gave up
constexpr int kDevErrFlagTimeout = 2;  // a wait for another CTA's flag gave up (chunked prep hand-off)
constexpr int kDevErrNormTimeout = 4;  // a wait for another CTA's sums of squares gave up (fused sequential norm)
constexpr int kDevErrRingTimeout = 8;  // a chunk prep's wait for a free slot of the tile ring gave up
constexpr int kDevErrLayout = 16;      // the scan's shared memory did not start where the kernel needs it
constexpr int kDevErrBlockNorm = 32;   // the block norm's wait for a row's copies gave up
constexpr int kDevErrKv = 64;          // a wait of the paged cache's attention gave up
constexpr int kDevErrKvLayout = 128;   // its shared memory did not start where the kernel needs it

// Of the words of the recurrence, its entry point that allocates nothing, and the operators over
// packed rows; not all 0.
inline std::string status_message(int word, int na_word, int packed_word) {
    constexpr int kOthers = kDevErrBlockNorm | kDevErrKv | kDevErrKvLayout;
    std::string msg = "a kernel gave up a bounded wait (status word " + std::to_string(word | na_word | packed_word) + ")";
    if (na_word != 0) msg += " in gdn_recurrence_chunked_noalloc";
    if (packed_word & kDevErrBlockNorm) msg += " in gdn_block_norm";
    if (packed_word & (kDevErrKv | kDevErrKvLayout)) msg += " in gdn_kv_attention";
    if (packed_word & ~kOthers) msg += " in gdn_ssm_scan";
    if (packed_word & (kDevErrLayout | kDevErrKvLayout)) msg += " (its shared memory does not start where it has to)";
    if (word & kDevErrNormTimeout) msg += " (the fused sequential norm's exchange between CTAs)";
    if (word & kDevErrRingTimeout) msg += " (a chunk prep's wait for a free slot of the tile ring)";
    return msg;
}

}  // namespace gdn
