// seqs.cuh -- the sequences of a call, dense [N, T] or packed one behind the other, and the order in which
// their tiles are worked on.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace dr {
struct Seqs {
    const int32_t* cu;  // packed: device [N + 1], the first row of each sequence; null: dense
    int N, T;           // sequences; tokens of each (dense) or rows in all (packed)
};

// First row and length of sequence s.  Offsets outside 0 .. T are taken as the nearest of them and a
// sequence that would end before it starts is empty, so that nothing outside the tensors is touched.
__device__ __forceinline__ void seq_rows(const Seqs& q, int s, int& row0, int& len) {
    if (!q.cu) {
        row0 = s * q.T;
        len = q.T;
        return;
    }
    row0 = min(max(q.cu[s], 0), q.T);
    len = max(min(max(q.cu[s + 1], 0), q.T) - row0, 0);
}

// Tiles of R rows that the sequences can have in all (offsets in order): a grid size.
inline long long most_tiles(const Seqs& q, int R) {
    return q.cu ? (long long)q.T / R + q.N : (long long)q.N * ((q.T + R - 1) / R);
}

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Tile number `item` of all tiles of R rows in the order of the sequences, and for a sequence of several tiles how many
// tiles such sequences have before it (`slot`: a place for each of them); called by a whole warp.  A sequence without tokens
// counts as `least` tiles, 0 or 1.
__device__ __forceinline__ bool find_tile_in_order(const Seqs& q, int R, int least, long long item, int& seq, int& tile,
                                                   int& tiles, long long& slot) {
    const int lane = threadIdx.x & 31;
    if (!q.cu) {
        tiles = max((q.T + R - 1) / R, least);
        if (item >= (long long)tiles * q.N) return false;
        seq = (int)(item / tiles);
        tile = (int)(item % tiles);
        slot = (long long)seq * tiles;
        return true;
    }
    long long all = 0, split = 0;  // tiles before these 32 sequences; of those that are split
    for (int s0 = 0; s0 < q.N; s0 += 32) {
        int row0, len = 0;
        if (s0 + lane < q.N) seq_rows(q, s0 + lane, row0, len);
        const int m = s0 + lane >= q.N ? 0 : max((len + R - 1) / R, least);
        int a = m, b = m > 1 ? m : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
            if (lane >= o) a += x, b += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, all + a > item);
        if (hit) {
            const int l = __ffs(hit) - 1;
            seq = s0 + l;
            tiles = __shfl_sync(0xffffffffu, m, l);
            tile = (int)(item - all) - (__shfl_sync(0xffffffffu, a, l) - tiles);
            slot = split + __shfl_sync(0xffffffffu, b, l) - (tiles > 1 ? tiles : 0);
            return true;
        }
        all += __shfl_sync(0xffffffffu, a, 31);
        split += __shfl_sync(0xffffffffu, b, 31);
    }
    return false;
}
// Tile number `item` of all tiles of R rows, those with the largest index in their sequence first (under a
// causal mask the longest rows of work start first and the short ones fill the gaps); called by a whole warp.
// Returns false where there are fewer tiles.  With many sequences, whose tiles are few, in their order: a search is
// a pass over the offsets instead of one for each power of two of the tiles.  Attention, 8 heads of 64, longest first and
// in order: 512 sequences of 1 to 500 tokens forward 397 and 235 us, gradient 1134 and 760; 256 of them 151 and 117, 436 and
// 328; but 16 of 1 to 2500 (16 heads of 128), gradient 236 and 250.  A walk over the offsets for each tile is the square of
// the number of sequences in time: 4096 of 1 to 16 tokens 3.5 ms forward, 65536 for one head 0.14 s.
__device__ __forceinline__ bool find_tile(const Seqs& q, int R, long long item, int& seq, int& tile) {
    if (!q.cu) {
        const int n = (q.T + R - 1) / R;
        if (item >= (long long)n * q.N) return false;
        tile = n - 1 - (int)(item / q.N);
        seq = (int)(item % q.N);
        return true;
    }
    if (q.cu && q.N > 256) {
        int tiles;
        long long slot;
        return find_tile_in_order(q, R, 0, item, seq, tile, tiles, slot);
    }
    const int lane = threadIdx.x & 31;
    auto tiles = [&](int s) {
        if (s >= q.N) return 0;
        int row0, len;
        seq_rows(q, s, row0, len);
        return (len + R - 1) / R;
    };
    auto count = [&](int v) {  // tiles with index v or more
        long long c = 0;
        for (int s = lane; s < q.N; s += 32) c += max(0, tiles(s) - v);
        return warp_sum(c);
    };
    if (item >= count(0)) return false;
    int lo = 0, hi = (q.T + R - 1) / R;  // count(lo) > item >= count(hi)
    long long above = 0;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        const long long c = count(mid);
        if (c > item) lo = mid;
        else hi = mid, above = c;
    }
    tile = lo;
    int rest = (int)(item - above);  // among the sequences that have tile lo
    for (int s0 = 0; s0 < q.N; s0 += 32) {
        const unsigned has = __ballot_sync(0xffffffffu, tiles(s0 + lane) > lo);
        const int n = __popc(has);
        if (rest < n) {
            const bool mine = (has >> lane & 1) && __popc(has & ((1u << lane) - 1)) == rest;
            seq = s0 + __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
            return true;
        }
        rest -= n;
    }
    return false;
}

// find_tile_in_order's `slot` of a sequence that has several tiles; called by a whole warp.
__device__ __forceinline__ long long slots_before(const Seqs& q, int R, int seq) {
    if (!q.cu) return (long long)seq * ((q.T + R - 1) / R);
    long long c = 0;
    for (int s = threadIdx.x & 31; s < seq; s += 32) {
        int row0, len;
        seq_rows(q, s, row0, len);
        if (len > R) c += (len + R - 1) / R;
    }
    return warp_sum(c);
}
}  // namespace dr
