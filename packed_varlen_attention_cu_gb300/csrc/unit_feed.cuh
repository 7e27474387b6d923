// unit_feed.cuh -- how a persistent CTA's roles learn which work unit comes next.
//
// One producer thread decides the CTA's next unit and publishes it in a small
// shared-memory ring (UnitRing): its index, -1 once the CTA has no more work, and
// what the other roles need of the worklist.  These read the slots in the same
// order and release each when they have done with it.  The producer decides
// either from a fixed list (static dispatch) or by claiming the next rank of a
// dispatch order from a global counter (dynamic dispatch: "数据并行负载均衡" §4.4's LPT rule with the
// least loaded worker being whichever CTA frees up first).
//
// A dispatch counter is a pair (next, done) in device memory that starts at
// (0, 0): CTAs claim ranks with atomicAdd on `next`, and at exit each CTA adds
// one to `done`; the last one puts both back to 0, so the next launch that
// uses the same counter starts from rank 0.  One launch at a time may use a
// counter (launches ordered on a stream are fine).
#pragma once

#include <stdint.h>

#include "ptx.cuh"
#include "wl_layout.cuh"

namespace pva {

// R slots of T.
template <int R, class T>
struct UnitRing {
    uint64_t full[R], empty[R];
    T slot[R];
};

// `readers` arrivals free a slot.
template <int R, class T>
__device__ __forceinline__ void uring_init(UnitRing<R, T>& r, uint32_t readers) {
    for (int s = 0; s < R; ++s) {
        mbar_init(&r.full[s], 1);
        mbar_init(&r.empty[s], readers);
    }
}

// Producer: slot n (the n-th unit of this CTA) is free once every reader has
// taken unit n - R.
template <int R, class T>
__device__ __forceinline__ bool uring_wait_free(UnitRing<R, T>& r, uint32_t n,
                                                volatile int* abort_flag, int* err_word, int site,
                                                uint64_t timeout_ns) {
    return mbar_wait(&r.empty[n % R], ((n / R) & 1) ^ 1, abort_flag, err_word, site, timeout_ns);
}

struct SubTile {
    int32_t q_row, nrows, q_pos, head;
};

struct Unit {
    int32_t nsub, kvh, run_begin, run_count, ntiles;
    SubTile st[2];
};

// A slot of the unit ring: the unit as the producer found it, with its first run and that run's
// slice.  Units of one key tile are bounded by the chain of the role that computes on their scores, in
// which four dependent reads of the worklist for every unit were 2 of 5.7 us (forward, 209 groups of
// short pairs, 16 heads).
struct UnitSlot {
    int32_t idx;  // -1: no more work
    int32_t slice, lo, hi;
    int32_t split;  // forward: both sub-tiles are the unit's one, with alternate key tiles each
    Unit u;
    WlSlice s;
};

__device__ __forceinline__ Unit decode_unit(const WlUnit& u, const WlSeg* segs) {
    const WlSeg g = segs[u.seg];
    Unit r;
    r.nsub = u.h1 >= 0 ? 2 : 1;
    r.kvh = u.kvh;
    r.run_begin = u.run_begin;
    r.run_count = u.run_count;
    r.ntiles = u.ntiles;
    const int32_t ts[2] = {u.t0, u.t1};
    const int32_t hs[2] = {u.h0, u.h1};
    for (int i = 0; i < 2; ++i) {
        const int32_t t = ts[i] >= 0 ? ts[i] : 0;
        r.st[i].q_row = g.q_row0 + t * 128;
        r.st[i].nrows = min(128, g.q_len - t * 128);
        r.st[i].q_pos = g.q_pos0 + t * 128;
        r.st[i].head = hs[i];
    }
    return r;
}

// The n-th unit's slot, once it is published: for a whole converged warp, and for one thread.  It
// stays as it is until released, once by each reader (warp or thread).
template <int R, class T>
__device__ __forceinline__ bool uring_wait_warp(UnitRing<R, T>& r, uint32_t n, volatile int* abort_flag,
                                                int* err_word, int site, uint64_t timeout_ns) {
    return mbar_wait_warp(&r.full[n % R], (n / R) & 1, abort_flag, err_word, site, timeout_ns);
}
template <int R, class T>
__device__ __forceinline__ void uring_release_warp(UnitRing<R, T>& r, uint32_t n) {
    __syncwarp();
    mbar_arrive_elect(&r.empty[n % R]);
}
template <int R, class T>
__device__ __forceinline__ bool uring_wait(UnitRing<R, T>& r, uint32_t n, volatile int* abort_flag,
                                           int* err_word, int site, uint64_t timeout_ns) {
    return mbar_wait(&r.full[n % R], (n / R) & 1, abort_flag, err_word, site, timeout_ns);
}
template <int R, class T>
__device__ __forceinline__ void uring_release(UnitRing<R, T>& r, uint32_t n) {
    mbar_arrive(&r.empty[n % R]);
}

// Dynamic dispatch: the next rank for this CTA.
__device__ __forceinline__ int32_t dispatch_claim(int32_t* next) { return atomicAdd(next, 1); }

// Called by one thread of every CTA after its last claim (all of its roles
// are done): the last CTA of the launch resets the counter.
__device__ __forceinline__ void dispatch_exit(int32_t* next, int32_t* done) {
    __threadfence();
    if (atomicAdd(done, 1) == (int)gridDim.x - 1) {
        atomicExch(next, 0);
        atomicExch(done, 0);
    }
}

}  // namespace pva
