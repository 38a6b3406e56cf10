// Runs the pick's device functions (csrc/pick.cuh) on the host: the CTA's threads
// are contexts that take turns, switching at each barrier and warp exchange.
//
// stdin, whole numbers: cases, each
//   kind n_vis take lo hi need room total least most fill n  then n values
// kind 0: best_of over n / 2 keys, then their ids.  kind 1: scan_best over n
// scores as bits.  kind 2: scan_best, n / 2 scores for the passes that look for the
// limit, the others for the pass that writes.  room: ids the output has room for;
// fill: what the shared memory holds before the call.  kind 3: no call, but the
// areas of a CTA for n_vis blocks seen, `total` scored, `take` taken, by maxima if
// lo, by hi candidates if hi.
// stdout: a line per case: the output's room + n_vis words (-7: not written), or of
// the areas the places, the size, the rooms and the most a kernel is launched with.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <vector>

#define __device__
#define __host__
#define __forceinline__ inline
#define __noinline__
#pragma GCC diagnostic ignored "-Wunknown-pragmas"
using std::max;
using std::min;

struct Dim {
    int x;
};
static Dim threadIdx;
struct alignas(16) uint4 {
    uint32_t x, y, z, w;
};
static uint4 make_uint4(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return {x, y, z, w}; }

constexpr int CTA = 128, STACK = 1 << 16;
static ucontext_t g_main, g_ctx[CTA];
static bool g_done[CTA];

static void turn() {
    const int me = threadIdx.x;
    swapcontext(&g_ctx[me], &g_main);
    threadIdx.x = me;
}
struct Barrier {
    int n, here, round;
    void wait() {
        const int r = round;
        if (++here == n) {
            here = 0;
            ++round;
        }
        while (round == r) turn();
    }
};
static Barrier g_cta, g_warp[CTA / 32];
static uint32_t g_lane[CTA];

static void __syncthreads() { g_cta.wait(); }
// Every lane's v, to all lanes.
static void exchange(uint32_t v, uint32_t (&all)[32]) {
    const int w = threadIdx.x / 32;
    g_lane[threadIdx.x] = v;
    g_warp[w].wait();
    memcpy(all, g_lane + w * 32, sizeof all);
    g_warp[w].wait();
}
static int __shfl_up_sync(uint32_t, int v, int o) {
    uint32_t all[32];
    exchange((uint32_t)v, all);
    const int l = threadIdx.x % 32;
    return (int)all[l >= o ? l - o : l];
}
static uint32_t __reduce_max_sync(uint32_t, uint32_t v) {
    uint32_t all[32];
    exchange(v, all);
    return *std::max_element(all, all + 32);
}
static uint32_t __reduce_min_sync(uint32_t, uint32_t v) {
    uint32_t all[32];
    exchange(v, all);
    return *std::min_element(all, all + 32);
}
static int __reduce_add_sync(uint32_t, int v) {
    uint32_t all[32], sum = 0;
    exchange((uint32_t)v, all);
    for (uint32_t x : all) sum += x;
    return (int)sum;
}
static int atomicAdd(int* p, int v) {
    const int was = *p;
    *p = was + v;
    return was;
}
static uint32_t atomicOr(uint32_t* p, uint32_t v) {
    const uint32_t was = *p;
    *p = was | v;
    return was;
}
static int __popc(uint32_t x) { return __builtin_popcount(x); }
static int __ffs(uint32_t x) { return __builtin_ffs((int)x); }
static int __clz(int x) { return x ? __builtin_clz((unsigned)x) : 32; }
static float __uint_as_float(uint32_t u) {
    float f;
    memcpy(&f, &u, 4);
    return f;
}
static uint32_t __float_as_uint(float f) {
    uint32_t u;
    memcpy(&u, &f, 4);
    return u;
}

#include "../long_context_causal_gqa_gb300/csrc/pick.cuh"

using namespace gqa::select;

struct Case {
    int kind;
    RowRange R;
    int room, total;
    uint32_t least, most, fill;
    std::vector<uint32_t> v;
    std::vector<int32_t> out;
    std::vector<uint4> bits;
};
static Case* g_case;
static BestShared<CTA> g_shared;

static void thread_main() {
    Case& c = *g_case;
    if (c.kind == 0) {
        const int n = (int)c.v.size() / 2;
        best_of<CTA, false>(c.R, c.v.data(), (const int*)(c.v.data() + n), c.total, c.least,
                            c.most, c.out.data(), (uint32_t*)c.bits.data(), g_shared);
    } else {
        // Scores that another call changes: this thread's blocks of the four counting
        // passes, then others.
        long calls = 0;
        const int n = (int)c.v.size() / c.kind;
        long mine = 0;
        for (int b = c.R.lo + threadIdx.x; b < c.R.hi; b += CTA) ++mine;
        scan_best<CTA>(
            c.R,
            [&](int b) {
                const bool later = c.kind == 2 && calls++ >= 4 * mine;
                return __uint_as_float(c.v[b + (later ? n : 0)]);
            },
            c.out.data(), g_shared);
    }
    g_done[threadIdx.x] = true;
    swapcontext(&g_ctx[threadIdx.x], &g_main);
}

int main() {
    std::vector<char> stacks((size_t)CTA * STACK);
    Case c;
    long n, least, most, fill;
    while (scanf("%d %d %d %d %d %d %d %d %ld %ld %ld %ld", &c.kind, &c.R.n_vis, &c.R.take,
                 &c.R.lo, &c.R.hi, &c.R.need, &c.room, &c.total, &least, &most, &fill,
                 &n) == 12) {
        c.least = (uint32_t)least;
        c.most = (uint32_t)most;
        c.v.resize(n);
        for (auto& x : c.v) {
            long u;
            if (scanf("%ld", &u) != 1) return 2;
            x = (uint32_t)u;
        }
        if (c.kind == 3) {
            const PickAreas A = c.R.hi ? best_areas(c.R.n_vis, c.R.hi, c.R.take)
                                       : pick_areas(c.R.n_vis, c.total, c.R.take, c.R.lo);
            printf("%d %d %d %d %d %d %d %d %d %d\n", A.key(), A.id(), A.groups(), A.reach(),
                   A.bytes(), A.room, A.room_groups, A.room_reach,
                   c.R.hi ? BEST_MOST_BYTES : PICK_MOST_BYTES, (int)sizeof(BestShared<1024>));
            continue;
        }
        c.out.assign(c.room + c.R.n_vis, -7);
        c.bits.resize(bits_words(c.R.n_vis) / 4);
        memset(c.bits.data(), (int)fill, c.bits.size() * sizeof(uint4));
        memset(&g_shared, (int)fill, sizeof g_shared);
        g_case = &c;
        g_cta = {CTA, 0, 0};
        for (auto& w : g_warp) w = {32, 0, 0};
        for (int i = 0; i < CTA; ++i) {
            g_done[i] = false;
            getcontext(&g_ctx[i]);
            g_ctx[i].uc_stack.ss_sp = stacks.data() + (size_t)i * STACK;
            g_ctx[i].uc_stack.ss_size = STACK;
            g_ctx[i].uc_link = nullptr;
            makecontext(&g_ctx[i], thread_main, 0);
        }
        // Each turn runs to the next wait; far more turns than any call needs: stuck.
        bool some = true;
        for (long turns = 0; some; ++turns) {
            if (turns > 1000000) return 3;
            some = false;
            for (int i = 0; i < CTA; ++i) {
                if (g_done[i]) continue;
                some = true;
                threadIdx.x = i;
                swapcontext(&g_main, &g_ctx[i]);
            }
        }
        for (int32_t x : c.out) printf("%d ", x);
        printf("\n");
    }
    return 0;
}
