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
template <int kRow>
struct Q4Copies {
  static constexpr int kPieces = kRow / 16;
  static constexpr int kBytes = 2 * kQ4Keys * kRow;  // of a copy: keys, then values
  int P, log2, slots, per_slot;
  uint32_t slot_of;
  bool even, pages_fine;
  const char *k_head, *v_head;
  // The page table's entries from pages_from on, one per lane, and those behind them.
  int pages_from, pages, pages_behind;

  __device__ __forceinline__ Q4Copies(const AttnParams &p, int lane) {
    P = p.C.page_size;
    log2 = 31 - __clz(P);
    even = (P & (P - 1)) == 0 && (P == 1 || (p.C.k_token == kRow && p.C.v_token == kRow));
    slots = max(kQ4Keys >> log2, 1);
    per_slot = min(P, kQ4Keys) * kPieces;
    slot_of = 0;
#pragma unroll
    for (int x = 0; x < kPieces; ++x) slot_of |= static_cast<uint32_t>((x * 32 + lane) / per_slot) << (5 * x);
    pages_from = pages = pages_behind = 0;
    pages_fine = false;
    k_head = v_head = nullptr;
  }
  __device__ __forceinline__ int fetch(const AttnParams &p, const UnitWalk &u, int from, int lane) const {
    return from + lane <= (u.k.end - 1) >> log2 ? page_at(p.S, u.b, from + lane) : 0;
  }
  // A unit's pages from key `at` on, on their way.
  __device__ __forceinline__ void begin(const AttnParams &p, const UnitWalk &u, int at, int lane) {
    k_head = p.C.k + u.h * p.C.k_head;
    v_head = p.C.v + u.h * p.C.v_head;
    pages_from = (at >> log2) - 32;
    pages_fine = false;
    if (even && u.k.end > 0) pages_behind = fetch(p, u, pages_from + 32, lane);
  }
  // Asks for the keys from at0 on; which of them there are.
  __device__ __forceinline__ uint32_t ask(const AttnParams &p, const UnitWalk &u, int at0, uint32_t to,
                                          int lane) {
    const uint32_t k_to = to + lane * 16, v_to = k_to + kQ4Keys * kRow;
    // without gaps
    const bool plain = even && at0 + kQ4Keys <= u.k.end && (at0 >= u.k.first || at0 + kQ4Keys <= p.sinks);
    const int index = at0 >> log2;
    if (plain && (index < pages_from || index + slots > pages_from + 32)) {
      // (those behind were asked for when these were)
      pages = index == pages_from + 32 ? pages_behind : fetch(p, u, index, lane);
      pages_from = index;
      pages_fine = __all_sync(0xFFFFFFFFu, page_ok(p.C, pages));
      pages_behind = fetch(p, u, index + 32, lane);
    }
    if (plain && pages_fine) {
      const int in_page = (at0 & (P - 1)) * kRow + lane * 16;
#pragma unroll
      for (int x = 0; x < kPieces; ++x) {
        const int slot = (slot_of >> (5 * x)) & 31;
        const int page = __shfl_sync(0xFFFFFFFFu, pages, index - pages_from + slot);
        const int at = in_page + x * 512 - slot * per_slot * 16;
        q4_copy16(k_to + x * 512, k_head + page * p.C.k_page + at);
        q4_copy16(v_to + x * 512, v_head + page * p.C.v_page + at);
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
      ko = page * p.C.k_page + (at - in * P) * p.C.k_token;
      vo = page * p.C.v_page + (at - in * P) * p.C.v_token;
    }
    const uint32_t there = __ballot_sync(0xFFFFFFFFu, page_ok(p.C, page));
#pragma unroll 1
    for (int x = 0; x < kPieces; ++x) {
      const int key = (x * 32 + lane) / kPieces, piece = x * 32 + lane - key * kPieces;
      const long long kr = __shfl_sync(0xFFFFFFFFu, ko, key), vr = __shfl_sync(0xFFFFFFFFu, vo, key);
      if ((there >> key) & 1u) {
        q4_copy16(k_to + x * 512, k_head + kr + piece * 16);
        q4_copy16(v_to + x * 512, v_head + vr + piece * 16);
      }
    }
    return there;
  }
};

}  // namespace sv
