// What the attention kernels over 4-bit rows share: copies of 32 keys and their values
// from the pages into shared memory, by one warp for itself.
#pragma once

#include "paged_attention_wide.cuh"

namespace sv {

constexpr int kQ4Keys = 32;  // of a copy

__device__ __forceinline__ void q4_copy16(uint32_t to, const char *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// Pages that are whole parts of 32 keys, or hold whole ones, their tokens one behind
// another, are copied without a look at each key: of the 16-byte pieces a lane copies
// every 32nd, a page's within the 32 keys are `per_slot`, and slot_of says from which of
// their pages (5 bits each).
// A warp's copies are kStride tokens behind one another.
template <int kRow, int kStride = kQ4Keys>
struct Q4Copies {
  static constexpr int kPieces = kRow / 16;
  static constexpr int kBytes = 2 * kQ4Keys * kRow;  // of a copy: keys, then values
  int P, log2, slots, per_slot;
  uint32_t slot_of;
  bool even, pages_fine;
  const char *k_head, *v_head;
  // The pages of the copies from some place on, `slots` lanes each, of which `used` are
  // asked for, and of those behind them; places of the next copy and of those behind.
  int pages, used, pages_behind, next_at, behind_at;

  __device__ __forceinline__ Q4Copies(const AttnParams &p, int lane) {
    P = p.C.page_size;
    log2 = 31 - __clz(P);
    even = (P & (P - 1)) == 0 && (P == 1 || (p.C.k_token == kRow && p.C.v_token == kRow));
    slots = max(kQ4Keys >> log2, 1);
    per_slot = min(P, kQ4Keys) * kPieces;
    slot_of = 0;
#pragma unroll
    for (int x = 0; x < kPieces; ++x) slot_of |= static_cast<uint32_t>((x * 32 + lane) / per_slot) << (5 * x);
    pages = used = pages_behind = next_at = behind_at = 0;
    pages_fine = false;
    k_head = v_head = nullptr;
  }
  __device__ __forceinline__ int fetch(const AttnParams &p, const UnitWalk &u, int at, int lane) const {
    const int copy = lane >> max(5 - log2, 0);
    const uint32_t index = ((static_cast<uint32_t>(at) + copy * kStride) >> log2) + (lane - copy * slots);
    return index <= static_cast<uint32_t>((u.k.end - 1) >> log2) ? page_at(p.S, u.b, static_cast<int>(index)) : 0;
  }
  // A unit's pages from key `at` on, on their way.
  __device__ __forceinline__ void begin(const AttnParams &p, const UnitWalk &u, int at, int lane) {
    k_head = p.C.k + u.h * p.C.k_head;
    v_head = p.C.v + u.h * p.C.v_head;
    next_at = -1;
    pages_fine = false;
    behind_at = at;
    if (even && u.k.end > 0) pages_behind = fetch(p, u, at, lane);
  }
  // Asks for the keys from at0 on and their values, or for the values alone or the keys
  // alone (kBoth false); which of them there are.
  template <bool kBoth = true>
  __device__ __forceinline__ uint32_t ask(const AttnParams &p, const UnitWalk &u, int at0, uint32_t to,
                                          int lane, bool values = false) {
    const uint32_t k_to = to + lane * 16 + (values ? kQ4Keys * kRow : 0), v_to = k_to + kQ4Keys * kRow;
    const char *one = values ? v_head : k_head;
    const long long one_page = values ? p.C.v_page : p.C.k_page, one_token = values ? p.C.v_token : p.C.k_token;
    // without gaps
    const bool plain = even && at0 + kQ4Keys <= u.k.end && (at0 >= u.k.first || at0 + kQ4Keys <= p.sinks);
    if (plain && (at0 != next_at || used + slots > 32)) {
      // (those behind were asked for when these were)
      pages = at0 == behind_at ? pages_behind : fetch(p, u, at0, lane);
      pages_fine = __all_sync(0xFFFFFFFFu, page_ok(p.C, pages));
      used = 0;
      next_at = at0;
      behind_at = static_cast<int>(static_cast<uint32_t>(at0) + 32 / slots * kStride);
      pages_behind = fetch(p, u, behind_at, lane);
    }
    if (plain && pages_fine) {
      const int in_page = (at0 & (P - 1)) * kRow + lane * 16;
#pragma unroll
      for (int x = 0; x < kPieces; ++x) {
        const int slot = (slot_of >> (5 * x)) & 31;
        const int page = __shfl_sync(0xFFFFFFFFu, pages, used + slot);
        const int at = in_page + x * 512 - slot * per_slot * 16;
        q4_copy16(k_to + x * 512, one + page * one_page + at);
        if (kBoth) q4_copy16(v_to + x * 512, v_head + page * p.C.v_page + at);
      }
      if (kBoth || values) {  // the last that is asked for here
        next_at = at0 + kStride;
        used += slots;
      }
      return 0xFFFFFFFFu;
    }
    // a key a lane finds its place, then a piece a lane
    const int at = at0 + lane;
    int page = -1;
    long long ko = 0, vo = 0;
    // not behind the last key, nor between the sinks and the window
    if (at < u.k.end && (at < p.sinks || at >= u.k.first)) {
      const int in = at / P;
      page = page_at(p.S, u.b, in);
      ko = page * one_page + (at - in * P) * one_token;
      if (kBoth) vo = page * p.C.v_page + (at - in * P) * p.C.v_token;
    }
    const uint32_t there = __ballot_sync(0xFFFFFFFFu, page_ok(p.C, page));
#pragma unroll 1
    for (int x = 0; x < kPieces; ++x) {
      const int key = (x * 32 + lane) / kPieces, piece = x * 32 + lane - key * kPieces;
      const long long kr = __shfl_sync(0xFFFFFFFFu, ko, key), vr = kBoth ? __shfl_sync(0xFFFFFFFFu, vo, key) : 0;
      if ((there >> key) & 1u) {
        q4_copy16(k_to + x * 512, one + kr + piece * 16);
        if (kBoth) q4_copy16(v_to + x * 512, v_head + vr + piece * 16);
      }
    }
    return there;
  }
};

}  // namespace sv
