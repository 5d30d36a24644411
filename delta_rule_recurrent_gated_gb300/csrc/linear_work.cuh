// linear_work.cuh -- the division of a linear-attention scan into blocks.
#pragma once
#include "linear_attn.cuh"
#include "vec4.cuh"

namespace dr {
namespace {

// A block's chunks: all of a sequence or a segment of them.
struct Work {
    int seq, row0, len, c0, chunks;
    bool first, last;       // of the sequence's segments in the order of the scan
    const float* before;    // the state before a segment that is not the only one (first step: where its own goes)
    __device__ __forceinline__ int at(const ScanParams& p, int n) const { return (c0 + (p.reverse ? chunks - 1 - n : n)) * kScanChunk; }
    __device__ __forceinline__ int tokens(int at) const { return min(kScanChunk, len - at); }
};
__device__ __forceinline__ bool make_work(const ScanParams& p, int item, int head, Work& w) {
    const int span = p.span ? p.span : (1 << 30) / kScanChunk;
    int tile, tiles;
    long long slot;
    if (p.span) {
        if (!find_tile_in_order(p.s, span * kScanChunk, 1, item, w.seq, tile, tiles, slot)) return false;
    } else {  // an item for each sequence
        w.seq = item;
        tile = 0;
        tiles = 1;
        slot = 0;
    }
    seq_rows(p.s, w.seq, w.row0, w.len);
    w.c0 = tile * span;
    w.chunks = min(span, (w.len + kScanChunk - 1) / kScanChunk - w.c0);
    w.first = p.reverse ? tile == tiles - 1 : tile == 0;
    w.last = p.reverse ? tile == 0 : tile == tiles - 1;
    if (tiles > 1 && slot + tiles > p.slots) return false;  // offsets out of order: sequences that overlap
    w.before = tiles > 1 ? p.part + ((slot + tile) * p.H + head) * p.dk * p.dv : nullptr;
    return true;
}

// Items of a launch: segments of the sequences, a sequence without tokens as one.
long long scan_items(const ScanParams& p) {
    const long long R = (p.span ? p.span : (1 << 30) / kScanChunk) * (long long)kScanChunk;
    if (!p.span) return p.s.N;
    return p.s.cu ? p.s.T / R + p.s.N : p.s.N * (p.s.T > R ? (p.s.T + R - 1) / R : 1);
}

}  // namespace
}  // namespace dr
