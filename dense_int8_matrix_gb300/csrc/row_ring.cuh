// Rows of up to three matrices on their way through rings in shared memory,
// and back for rows that are not aligned.
//
// A CTA is one team of warps or several.  A team takes a chunk of rows at a time
// from a ring of its own, which its first thread fills ahead (bulk copies).  What a
// row takes is mostly latency (two sums over the team, one after the other), so
// that a chunk is at least two rows, worked on together, and one team waits
// while another works.
#pragma once

#include <cstdint>
#include <initializer_list>

#include "f8_tc.cuh"

namespace gemm {

// A chunk is `per` neighbouring rows.  Dense rows (without gaps) are one run of
// bytes, others a run each.  A run is copied with the 16-byte words that hold its
// ends, to the same place modulo 16; of a chunk whose words could reach past the
// matrix (the first or the last, unless its ends are aligned) the words inside
// its runs are copied, and its team loads what is left.
struct ChunkRing {
    static constexpr int kSlots = 8;
    struct Array {
        const uint8_t* base;   // nullptr: none
        int64_t pitch;         // bytes from a row to the next
        uint32_t bytes;        // of a row
        uint32_t at, place;    // of its first run in a slot; from a run to the next
    };
    Array a[3];
    int64_t rows, chunks, by;  // by: chunks from one of this ring to its next
    int per, slots;
    bool dense;
    bool head, tail;           // whether the first and the last chunk are copied whole
    uint32_t ring, full0, slot_bytes;

    // Bytes of a run's place in a slot.
    __host__ __device__ static int64_t run_place(int64_t bytes) { return (bytes + 15) / 16 * 16 + 16; }
    // And of the `per` rows of an array.
    __host__ __device__ static int64_t place(int64_t row_bytes, int per, bool dense) {
        return dense ? run_place(row_bytes * per) : per * run_place(row_bytes);
    }

    __device__ __forceinline__ void init(int64_t rows_, int per_, bool dense_, int slots_, int64_t by_, uint32_t bars) {
        rows = rows_;
        per = per_;
        dense = dense_;
        chunks = (rows_ + per_ - 1) / per_;
        slots = slots_;
        by = by_;
        head = tail = true;
        full0 = bars;
        slot_bytes = 0;
    }
    // (rows of 16 bytes and more: only the first and the last row can reach past
    // the matrix)
    __device__ __forceinline__ void set(int i, const void* base, int64_t ld, int es, int64_t d) {
        a[i].base = static_cast<const uint8_t*>(base);
        a[i].pitch = ld * es;
        a[i].bytes = static_cast<uint32_t>(d * es);
        a[i].at = slot_bytes;
        a[i].place = static_cast<uint32_t>(run_place(d * es));
        if (!base) return;
        slot_bytes += static_cast<uint32_t>(place(d * es, per, dense));
        const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
        head = head && (lo & 15) == 0;
        tail = tail && ((lo + (rows - 1) * ld * es + d * es) & 15) == 0;
    }
    __device__ __forceinline__ int rows_of(int64_t c) const {
        return c + 1 < chunks ? per : static_cast<int>(rows - (chunks - 1) * per);
    }
    __device__ __forceinline__ bool whole(int64_t c) const { return (c > 0 || head) && (c + 1 < chunks || tail); }
    // One thread: chunk c (nothing past the last) into slot s.
    __device__ __forceinline__ void fill(int64_t c, int s) const {
        if (c >= chunks) return;
        const uint32_t bar = full0 + 8u * s, dst = ring + s * slot_bytes;
        const bool out = whole(c);   // words that hold an end, or words inside
        const int n = rows_of(c), runs = dense ? 1 : n;
        uint32_t all = 0;
        for (int r = 0; r < runs; ++r)
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                if (!a[i].base) continue;
                const uintptr_t from = reinterpret_cast<uintptr_t>(a[i].base) + (c * per + r) * a[i].pitch;
                const uint32_t low = static_cast<uint32_t>(from) & 15u, end = low + (dense ? n * a[i].bytes : a[i].bytes);
                const uint32_t lo = out ? 0u : (low + 15u) & ~15u, hi = out ? (end + 15u) & ~15u : end & ~15u;   // from the first word's start
                if (hi <= lo) continue;
                all += hi - lo;
                bulk_load(dst + a[i].at + r * a[i].place + lo, reinterpret_cast<const void*>((from & ~uintptr_t(15)) + lo), hi - lo, bar);
            }
        mbar_arrive_expect_tx(bar, all);
    }
    // Byte offset in the ring of row r of chunk c of array i, in slot s.
    __device__ __forceinline__ uint32_t row(int i, int s, int64_t c, int r) const {
        const uint32_t at = s * slot_bytes + a[i].at, low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(a[i].base));
        const uint32_t pitch = static_cast<uint32_t>(a[i].pitch), first = static_cast<uint32_t>(c) * static_cast<uint32_t>(per);
        return dense ? at + ((low + first * pitch) & 15u) + r * a[i].bytes : at + r * a[i].place + ((low + (first + r) * pitch) & 15u);
    }
    // The same for aligned rows that are not dense.
    __device__ __forceinline__ uint32_t aligned_row(int i, int s, int r) const { return s * slot_bytes + a[i].at + r * a[i].place; }
};

// Sixteen bytes and more go from shared memory to the same place modulo 16
// of a run of `bytes` bytes at dst: one thread moves the aligned middle ...
__device__ __forceinline__ void store_run(uintptr_t dst, uint32_t src, uint32_t bytes) {
    const uint32_t head = static_cast<uint32_t>(-static_cast<int64_t>(dst) & 15);
    if (bytes < head + 16) return;
    const uint32_t n = (bytes - head) & ~15u;
    bulk_store(reinterpret_cast<void*>(dst + head), src + head, n);
}
// ... and a warp its ends, by elements.
template <typename T>
__device__ __forceinline__ void store_ends(uintptr_t dst, const uint8_t* src, uint32_t bytes, int lane) {
    constexpr int ES = sizeof(T), kMost = 16 / ES - 1;   // elements at either end
    const uint32_t head = min(static_cast<uint32_t>(-static_cast<int64_t>(dst) & 15), bytes);
    const uint32_t tail = bytes < head + 16 ? bytes - head : (bytes - head) & 15u;   // (a short run has no middle)
    static_assert(kMost + 2 * kMost + 1 <= 32, "an element per lane");
    uint32_t at = ~0u;
    if (static_cast<uint32_t>(lane) * ES < head)
        at = lane * ES;
    else if (lane >= kMost && static_cast<uint32_t>(lane - kMost) * ES < tail)
        at = bytes - tail + (lane - kMost) * ES;
    if (at != ~0u) *reinterpret_cast<T*>(dst + at) = *reinterpret_cast<const T*>(src + at);
}

// A team: its place in the CTA, and its barrier.
constexpr int kMostTeams = 15;   // with more than one warp: barrier 0 is the CTA's
struct Team {
    int id, threads, thread, warp, warps;
    __device__ __forceinline__ Team(int threads_)
        : id(threadIdx.x / threads_), threads(threads_), thread(threadIdx.x - id * threads_), warp(thread >> 5), warps(threads_ >> 5) {}
    __device__ __forceinline__ void sync() const {
        if (warps == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
    }
    // Sums of N values over the team, in place; `red` (N floats for each of the
    // CTA's warps) is used by this call alone until the team's next sync.
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N], float* red) const {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
        if (warps == 1) return;
        const int lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[(threadIdx.x >> 5) * N + i] = v[i];
        sync();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? red[(id * warps + lane) * N + i] : 0.f);
    }
};

// Loads the ends of a chunk that was not copied whole (at most seven elements of
// two bytes at either end of a run).  The whole team.
__device__ __forceinline__ void load_ends(const ChunkRing& ring, uint8_t* slots, int s, int64_t c, const Team& team) {
    const int n = ring.rows_of(c), runs = ring.dense ? 1 : n;
    for (int k = team.thread; k < runs * 3 * 16; k += team.threads) {
        const int r = k / 48, i = k / 16 % 3, j = k % 16;
        if (!ring.a[i].base) continue;
        const uintptr_t from = reinterpret_cast<uintptr_t>(ring.a[i].base) + (c * ring.per + r) * ring.a[i].pitch;
        const uint32_t low = static_cast<uint32_t>(from) & 15u, end = low + (ring.dense ? n : 1) * ring.a[i].bytes;
        const uint32_t lo = (low + 15u) & ~15u, hi = max(end & ~15u, lo);   // (rows are longer than a word)
        const uint32_t at = j < 8 ? low + 2 * j : hi + 2 * (j - 8);
        if (j < 8 ? at < lo : at < end)
            *reinterpret_cast<uint16_t*>(slots + s * ring.slot_bytes + ring.a[i].at + r * ring.a[i].place + at) =
                *reinterpret_cast<const uint16_t*>((from & ~uintptr_t(15)) + at);
    }
    team.sync();
}

// ---- eight values as four pairs ------------------------------------------------
// (the packed instructions do two fp32 operations at once)
struct Pairs {
    uint64_t p[4];
};
__device__ __forceinline__ uint64_t both(float x) { return pair_of(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ float sum_of(uint64_t x) {
    float a, b;
    unpair(x, a, b);
    return a + b;
}
__device__ __forceinline__ Pairs pairs(const Vec8<__nv_bfloat16>& v) {
    const uint32_t w[4] = {v.u.x, v.u.y, v.u.z, v.u.w};
    Pairs r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = pair_of(w[i] << 16, w[i] & 0xffff0000u);
    return r;
}
__device__ __forceinline__ Pairs pairs(const Vec8<float>& v) {
    Pairs r;
    r.p[0] = pair_of(__float_as_uint(v.a.x), __float_as_uint(v.a.y));
    r.p[1] = pair_of(__float_as_uint(v.a.z), __float_as_uint(v.a.w));
    r.p[2] = pair_of(__float_as_uint(v.b.x), __float_as_uint(v.b.y));
    r.p[3] = pair_of(__float_as_uint(v.b.z), __float_as_uint(v.b.w));
    return r;
}
__device__ __forceinline__ Pairs pairs(const float* aligned) {
    Vec8<float> v;
    v.load(aligned);
    return pairs(v);
}
template <typename T>
__device__ __forceinline__ Vec8<T> vec(const Pairs& x) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair(x.p[i], f[2 * i], f[2 * i + 1]);
    Vec8<T> v;
    v.set(f);
    return v;
}

// The pair of values at x[0] and x[stride], zero where they are not `in` the row.
__device__ __forceinline__ uint32_t bits(const float* x) { return __float_as_uint(*x); }
__device__ __forceinline__ uint32_t bits(const __nv_bfloat16* x) {
    return static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(x)) << 16;
}
template <typename T>
__device__ __forceinline__ uint64_t pair_at(const T* x, int stride, bool in0, bool in1) {
    return pair_of(in0 ? bits(x) : 0u, in1 ? bits(x + stride) : 0u);
}
// And back.
template <typename T>
__device__ __forceinline__ void put_pair(uint64_t v, T* x, int stride, bool in0, bool in1) {
    float a, b;
    unpair(v, a, b);
    if (in0) from_f32(a, x);
    if (in1) from_f32(b, x + stride);
}
// Rounded to T as it is stored.
template <typename T>
__device__ __forceinline__ uint64_t rounded_pair(uint64_t v) {
    if constexpr (sizeof(T) == 4) return v;
    float a, b;
    unpair(v, a, b);
    const uint32_t w = bf16x2(a, b);
    return pair_of(w << 16, w & 0xffff0000u);
}

// ---- host: how a ring kernel is launched -----------------------------------------
struct RingShape {
    int each;            // vectors (aligned rows) or values of a row per thread
    int per;             // rows of a chunk
    int dense;
    int team, teams;     // threads of a team, teams of a CTA
    int slots;           // of a team's ring
    int64_t smem;
    int grid;
};
constexpr int kRingThreads = 512;   // of 128 registers
constexpr int kPair = 2;            // rows of a chunk of the kernels of aligned rows
// Rows that an unaligned kernel of J values per thread works on together
// (measured, 159783 x 105 bfloat16 forward: 71 us with two, 85 with four, 109
// with eight).
__host__ __device__ constexpr int rows_together(int values) { return values <= 12 ? 2 : 1; }
constexpr int64_t kRingSmem = 216 * 1024;
// The team and the number of units (vectors, values) per thread for a row of
// n: the choice that leaves the fewest of them idle, more per thread before
// more threads.
inline void team_of(RingShape* r, int64_t n, std::initializer_list<int> choices) {
    int64_t best = INT64_MAX;
    r->each = *choices.begin();
    r->team = kRingThreads;
    for (int each : choices) {   // the largest first
        const int64_t team = ((n + each - 1) / each + 31) / 32 * 32;
        if (team * each >= best || team > kRingThreads) continue;
        best = team * each;
        r->each = each;
        r->team = static_cast<int>(team);
    }
}
// Short rows that a warp takes at a time: about two KiB, as more leave room for
// fewer warps, and fewer are many small copies (measured, 8 M values of fp32:
// 401 wide 50 us with four rows, 36 with two, 32 with one; 299 wide 54, 38,
// 42; 16 M of bfloat16, 511 wide 62, 47, 50; 105 wide 72 with 2 KiB, 81 with
// one, 127 with four).
inline int rows_of_a_warp(int64_t bytes) {
    if (bytes > 1536) return 1;
    return bytes > 512 ? 2 : static_cast<int>(std::min<int64_t>(32, 2048 / bytes / 4 * 4));
}
// slot, out: bytes of a slot and of a team's staging buffers.  As many teams as
// leave each two slots.
inline bool fit_ring(RingShape* r, int64_t rows, int64_t slot, int64_t out, int num_sms) {
    const int64_t chunks = (rows + r->per - 1) / r->per;
    int teams = kRingThreads / r->team;
    if (r->team > 32 && teams > kMostTeams) teams = kMostTeams;
    if (teams < 1) return false;
    while (teams > 1 && kRingSmem / teams / 16 * 16 - out < 2 * slot) --teams;
    while (teams > 1 && chunks < static_cast<int64_t>(teams) * num_sms) --teams;   // no team without a chunk
    const int64_t fit = (kRingSmem / teams / 16 * 16 - out) / slot;
    if (fit < 2) return false;
    r->teams = teams;
    r->slots = static_cast<int>(fit < ChunkRing::kSlots ? fit : ChunkRing::kSlots);
    r->smem = teams * (r->slots * slot + out);
    const int64_t grid = (chunks + teams - 1) / teams;
    r->grid = static_cast<int>(grid < num_sms ? grid : num_sms);
    return true;
}
// What a kernel counts on, asked before every launch: chunks of `per` rows, a
// thread for each of a row's `units`, and room for its slots (of `slot` bytes as the
// kernel lays them out), its staging buffers (`out`) and, at the end, a team's `sums`.
// (A ring sized for chunks of one row, under a kernel that takes two, overruns
// shared memory.)
inline bool ring_holds(const RingShape& r, int per, int64_t units, int64_t slot, int64_t out, int64_t sums) {
    return r.per == per && r.team % 32 == 0 && static_cast<int64_t>(r.each) * r.team >= units && r.teams >= 1 &&
           r.team * r.teams <= kRingThreads && (r.team == 32 || r.teams <= kMostTeams) && r.slots >= 2 && r.slots <= ChunkRing::kSlots &&
           r.teams * (r.slots * slot + out) <= r.smem && r.teams * sums <= r.smem && r.smem <= kRingSmem && r.grid >= 1;
}

}  // namespace gemm
