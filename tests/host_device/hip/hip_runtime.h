// Runs device code on the host, one workgroup at a time, in a chosen order of
// its wavefronts: a kernel's source is compiled as plain C++ against this
// header in place of the HIP runtime's.
//
// Every thread is a fiber. It runs until an operation that needs others: a
// wavefront's exchange (shuffle, ballot) waits for the wavefront's live
// threads, __syncthreads for the workgroup's. Of the threads that can run, the
// first of the wavefront that comes first in `order` does, so that a
// wavefront goes as far ahead of those behind it as the barriers allow: what
// two wavefronts do to one LDS word between two barriers happens in both
// orders over the orders tried. A barrier that some threads wait at after
// others have returned is counted (`broken_barriers`), a workgroup in which
// nothing can go on any more ends the run (`stuck`).
//
// Limits: the exchanges of a wavefront must be reached by all of its live
// threads; memory is that of one thread (no stores in flight).
#pragma once

#include <float.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <functional>
#include <memory>
#include <type_traits>
#include <vector>

#include "hip_runtime_api.h"

namespace host_device {

constexpr int kLanes = 64;

struct Fiber {
    ucontext_t at;
    std::unique_ptr<char[]> stack;
    int tid;
    bool done;
    int waits;        // 0: can run, 1: for its wavefront, 2: for the workgroup
    uint32_t turn;    // exchanges of its wavefront so far
};

struct Wave {
    uint64_t slot[2][kLanes];
    uint64_t live[2];
    int here;         // threads that have arrived at the exchange
};

struct State {
    std::vector<Fiber> fibers;
    std::vector<Wave> waves;
    ucontext_t home;
    int now = 0;
    uint32_t block = 0, threads = 0, blocks = 0;
    std::function<void()> body;
    std::vector<int> order;        // of the wavefronts; those not named come last
    int64_t broken_barriers = 0, stuck = 0;
    bool dry = false;              // launches are only looked at
    uint64_t most_threads = 0;     // of any launch's grid
    std::function<void(const void *)> on_load;  // before an atomic load
};

inline State &state()
{
    static State s;
    return s;
}

inline void yield()
{
    State &s = state();
    swapcontext(&s.fibers[s.now].at, &s.home);
}

inline void enter()
{
    State &s = state();
    s.body();
    s.fibers[s.now].done = true;
    yield();
}

inline void run_block()
{
    State &s = state();
    const int n = (int)s.threads, waves = (n + kLanes - 1) / kLanes;
    constexpr size_t kStack = 128 << 10;
    if ((int)s.fibers.size() < n)
        s.fibers.resize(n);
    s.waves.assign(waves, Wave{});
    for (int i = 0; i < n; ++i) {
        Fiber &f = s.fibers[i];
        if (!f.stack)
            f.stack.reset(new char[kStack]);
        getcontext(&f.at);
        f.at.uc_stack.ss_sp = f.stack.get();
        f.at.uc_stack.ss_size = kStack;
        f.at.uc_link = nullptr;
        makecontext(&f.at, (void (*)())enter, 0);
        f.tid = i;
        f.done = false;
        f.waits = 0;
        f.turn = 0;
    }
    std::vector<int> seq;
    for (int w : s.order)
        if (w < waves)
            seq.push_back(w);
    for (int w = 0; w < waves; ++w)
        if (std::find(seq.begin(), seq.end(), w) == seq.end())
            seq.push_back(w);
    int left = n;
    while (left) {
        bool ran = false;
        for (int w : seq) {
            const int end = std::min(n, (w + 1) * kLanes);
            for (int i = w * kLanes; i < end; ++i) {
                Fiber &f = s.fibers[i];
                if (f.done || f.waits)
                    continue;
                s.now = i;
                swapcontext(&s.home, &f.at);
                left -= f.done;
                ran = true;
            }
            // an exchange all live threads have reached
            int live = 0, here = 0;
            for (int i = w * kLanes; i < end; ++i) {
                live += !s.fibers[i].done;
                here += !s.fibers[i].done && s.fibers[i].waits == 1;
            }
            if (live && here == live) {
                for (int i = w * kLanes; i < end; ++i)
                    s.fibers[i].waits = 0;
                s.waves[w].here = 0;
                ran = true;
            }
            if (ran)
                break;
        }
        if (ran || !left)
            continue;
        int here = 0;
        for (int i = 0; i < n; ++i)
            here += !s.fibers[i].done && s.fibers[i].waits == 2;
        if (here != left) {
            ++s.stuck;
            return;
        }
        s.broken_barriers += left < n;
        for (int i = 0; i < n; ++i)
            s.fibers[i].waits = 0;
    }
}

inline void launch(uint32_t blocks, uint32_t threads, std::function<void()> body)
{
    State &s = state();
    s.most_threads = std::max(s.most_threads, (uint64_t)blocks * threads);
    if (s.dry)
        return;
    s.body = std::move(body);
    s.threads = threads;
    s.blocks = blocks;
    for (s.block = 0; s.block < blocks && !s.stuck; ++s.block)
        run_block();
}

// The values that the wavefront's live threads hold, and which are live.
struct Seen {
    const uint64_t *slot;
    uint64_t live;
};

inline Seen exchange(uint64_t mine)
{
    State &s = state();
    Fiber &f = s.fibers[s.now];
    Wave &w = s.waves[f.tid / kLanes];
    const int half = f.turn++ & 1, lane = f.tid % kLanes;
    if (w.here == 0)
        w.live[half] = 0;
    w.slot[half][lane] = mine;
    w.live[half] |= 1ull << lane;
    ++w.here;
    f.waits = 1;
    yield();
    return Seen{w.slot[half], w.live[half]};
}

template <typename T>
inline T from_bits(uint64_t v)
{
    T x;
    memcpy(&x, &v, sizeof(T));
    return x;
}
template <typename T>
inline uint64_t to_bits(T x)
{
    static_assert(sizeof(T) <= 8, "");
    uint64_t v = 0;
    memcpy(&v, &x, sizeof(T));
    return v;
}
// (a thread that is not live gives back the asking thread's own value)
template <typename T>
inline T from_lane(T x, int lane)
{
    const Seen seen = exchange(to_bits(x));
    return (seen.live >> lane) & 1 ? from_bits<T>(seen.slot[lane]) : x;
}
inline int lane()
{
    State &s = state();
    return s.fibers[s.now].tid % kLanes;
}

struct Dim {
    uint32_t x, y, z;
};
inline Dim thread_idx()
{
    State &s = state();
    return Dim{(uint32_t)s.fibers[s.now].tid, 0, 0};
}
inline Dim block_idx() { return Dim{state().block, 0, 0}; }
inline Dim block_dim() { return Dim{state().threads, 1, 1}; }

inline void barrier()
{
    State &s = state();
    s.fibers[s.now].waits = 2;
    yield();
}

template <typename T>
inline T load(const T *p)
{
    if (state().on_load)
        state().on_load(p);
    return *p;
}

}  // namespace host_device

struct dim3 {
    uint32_t x, y, z;
    dim3(uint32_t a = 1, uint32_t b = 1, uint32_t c = 1) : x(a), y(b), z(c) {}
};

#define __device__
#define __host__
#define __global__
#define __forceinline__ inline
#define __launch_bounds__(...)
#ifndef __shared__
#define __shared__ static
#endif
#define threadIdx host_device::thread_idx()
#define blockIdx host_device::block_idx()
#define blockDim host_device::block_dim()
#define __syncthreads() host_device::barrier()
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...)                          \
    host_device::launch((grid).x, (block).x, [=] { (kernel)(__VA_ARGS__); })

// waits for memory: nothing is in flight here
#define asm
#define volatile(...) ((void)0)

#define __hip_atomic_load(p, order, scope) host_device::load(p)
#define __hip_atomic_store(p, v, order, scope) ((void)(*(p) = (v)))
#define __hip_atomic_fetch_add(p, v, order, scope) host_fetch_add(p, v)
#define __hip_atomic_fetch_min(p, v, order, scope) host_fetch_min(p, v)
#define __builtin_amdgcn_exp2f(x) exp2f(x)
#define __builtin_amdgcn_readfirstlane(x) host_first(x)
inline void sincospif(float x, float *s, float *c)
{
    *s = (float)sin(M_PI * (double)x);
    *c = (float)cos(M_PI * (double)x);
}
// (8-bit conversions: not run here)
#define __builtin_amdgcn_cvt_f32_fp8(x, i) (abort(), (float)(x))
#define __builtin_amdgcn_cvt_pk_fp8_f32(a, b, c, d) (abort(), (int)(a))

template <typename T> inline T host_fetch_add(T *p, T v) { const T x = *p; *p = x + v; return x; }
template <typename T> inline T host_fetch_min(T *p, T v)
{
    const T x = *p;
    *p = v < x ? v : x;
    return x;
}
template <typename T> inline T host_first(T x)
{
    const host_device::Seen s = host_device::exchange(host_device::to_bits(x));
    return host_device::from_bits<T>(s.slot[__builtin_ctzll(s.live)]);
}
template <typename T> inline T __shfl(T x, int from) { return host_device::from_lane(x, from & 63); }
template <typename T> inline T __shfl_xor(T x, int m)
{
    return host_device::from_lane(x, host_device::lane() ^ m);
}
template <typename T> inline T __shfl_up(T x, int n)
{
    const int at = host_device::lane();
    return host_device::from_lane(x, at < n ? at : at - n);
}
inline uint64_t __ballot(bool x)
{
    const host_device::Seen s = host_device::exchange(x);
    uint64_t v = 0;
    for (int i = 0; i < 64; ++i)
        v |= ((s.live >> i) & 1 & s.slot[i]) << i;
    return v;
}
inline bool __any(bool x) { return __ballot(x) != 0; }
inline unsigned int atomicOr(unsigned int *p, unsigned int v) { const unsigned int x = *p; *p |= v; return x; }
inline int atomicMin(int *p, int v) { return host_fetch_min(p, v); }
inline int atomicMax(int *p, int v) { const int x = *p; *p = v > x ? v : x; return x; }
inline float __uint_as_float(uint32_t v) { return host_device::from_bits<float>(v); }
inline uint32_t __float_as_uint(float x) { return (uint32_t)host_device::to_bits(x); }
