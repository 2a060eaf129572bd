// cache_tickets.h -- how the CTAs that share a unit of the cache attention find out who leaves its last piece.
//
// A unit's pieces (cache_index.h) are joined in groups, and then the groups, by whoever counts last.  The counters live
// in the caller's workspace, whose contents are unspecified before a launch, and a captured launch comes again with
// the number that it was captured with.  So a counter's upper 48 bits are the launch's number, and any other number
// counts as none; and a counter is 0 again after its last count.  That holds when waits of a CTA have run out, too: it
// counts its pieces all the same, marked as failed, so that the next launch of the same number finds no counts, and
// nobody joins pieces that were never left.
//
// Plain C++: `Memory` holds the operations on a counter, so host tests compile it by itself.
#pragma once

#include "cache_index.h"

namespace attn {

constexpr unsigned long long kTicketFailed = 0x8000;  // beside a count below it

// Pieces that one CTA joins: up to `most` all of them, else the square root, so that groups of pieces are joined side by
// side and then the groups: 128 rows of one key/value head over 131072 keys, 128 pieces, take 55 us instead of 143, and
// 8 rows 23 instead of 27; for fewer pieces the second round costs more than it saves (30 sequences of 12800 keys in
// about 10 pieces each: 30 us instead of 26).
ATTN_HD int cache_group(int pieces, int most) {
    if (pieces <= most) return pieces;
    int n = 2;
    while (n * n < pieces) ++n;
    return n;
}
// A group that a piece is in: its first piece and how many it has.
struct CacheGroup {
    int begin, n;
};
ATTN_HD CacheGroup cache_group_of(int pieces, int group, int piece) {
    const int begin = piece / group * group, rest = pieces - begin;
    return {begin, rest < group ? rest : group};
}

// What a count says: more are to come, this was the last, or it was the last and one of them has failed.
enum CacheLast : int { kMoreToCome = 0, kWasLast = 1, kWasLastFailed = 2 };

// Each CTA that shares a unit does this before it counts its piece: a counter that does not carry this launch's
// number becomes 0 pieces of this launch.  An exchange that fails met another CTA's, which did the same.
template <typename Memory>
ATTN_HD void ticket_open(unsigned long long* at, unsigned long long number) {
    const unsigned long long had = Memory::load(at);
    if ((had ^ number) >> 16) Memory::compare_exchange(at, had, number);
}
// Counts one of `of`.
template <typename Memory>
ATTN_HD CacheLast ticket_count(unsigned long long* at, int of, bool failed) {
    if (failed) Memory::set(at, kTicketFailed);
    const unsigned long long had = Memory::add(at, 1);
    if ((int)(had & (kTicketFailed - 1)) + 1 != of) return kMoreToCome;
    Memory::clear(at);
    return had & kTicketFailed ? kWasLastFailed : kWasLast;
}

// The counters of a launch of `ctas` CTAs: of the group that begins with a CTA's piece, and of the groups of the unit
// that begins in a CTA.  A group of one piece needs none, so no two units meet at one.
ATTN_HD unsigned long long* ticket_of_group(unsigned long long* tickets, int first, const CacheGroup& g) {
    return tickets + first + g.begin;
}
ATTN_HD unsigned long long* ticket_of_unit(unsigned long long* tickets, int ctas, int first) { return tickets + ctas + first; }

// Opens the counters that piece `piece` of a unit of `pieces` that begins in CTA `first` will count at.
template <typename Memory>
ATTN_HD void tickets_open(unsigned long long* tickets, int ctas, unsigned long long number, int first, int pieces, int piece, int most) {
    const int group = cache_group(pieces, most);
    ticket_open<Memory>(ticket_of_group(tickets, first, cache_group_of(pieces, group, piece)), number);
    if (group < pieces) ticket_open<Memory>(ticket_of_unit(tickets, ctas, first), number);
}
// Counts the piece as left, or failed, in its group.
template <typename Memory>
ATTN_HD CacheLast tickets_leave(unsigned long long* tickets, int first, int pieces, int piece, int most, bool failed) {
    const CacheGroup g = cache_group_of(pieces, cache_group(pieces, most), piece);
    if (g.n == 1) return failed ? kWasLastFailed : kWasLast;
    return ticket_count<Memory>(ticket_of_group(tickets, first, g), g.n, failed);
}
// Counts a group of several as joined, or failed, in its unit.
template <typename Memory>
ATTN_HD CacheLast tickets_joined(unsigned long long* tickets, int ctas, int first, int pieces, int most, bool failed) {
    const int group = cache_group(pieces, most);
    return ticket_count<Memory>(ticket_of_unit(tickets, ctas, first), (pieces + group - 1) / group, failed);
}

}  // namespace attn
