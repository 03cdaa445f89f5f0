// kda_selective.h -- device code shared by the selective scan's kernels.
//
// A lane holds one channel with all its S state entries in registers, a wave 64 channels of
// one group, so B_t and C_t are the same for the whole wave: they come through the scalar
// cache and enter the products as scalar operands, and the sums over the state's entries stay
// in a lane.  An entry and token costs a multiply and an exponential for the decay, a
// multiply and a multiply-add for the state and a multiply-add for the output.  With 34 more a
// token for the step size, the gate, conversions and accesses these are 114 instructions at 16
// entries (counted), and they bound the kernels: 195 us at an instruction every four cycles and
// 229 with a second slot for the 20 exponentials, logarithms and quotients among them, which
// part of the time is another wave's, for 67.1M tokens and channels, where HBM would ask 105.
#pragma once
#include "kda_layer.h"

namespace kda {

constexpr float kLn2 = 0.693147181f;

// A row of B or C on its way (uniform), and as fp32.
template <typename T, int S> struct UniformRow {
    static constexpr int kWords = S * sizeof(T) / 4;
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    unsigned w[kWords];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const u32x4 x = uniform_load<u32x4>(reinterpret_cast<const unsigned*>(p) + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i + j] = x[j];
        }
    }
    __device__ __forceinline__ float operator[](int n) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[n]);
        else return __uint_as_float(n & 1 ? w[n >> 1] & 0xffff0000u : w[n >> 1] << 16);
    }
};

// Rows of B (or C) one after another from `p`, `step` elements apart; the last of `left` rows is not passed.  Rows that fit
// eight scalar registers are loaded one token ahead; longer ones would push others out.
template <typename T, int S> struct UniformRows {
    static constexpr bool kAhead = S * sizeof(T) <= 32;
    const T* p;
    int64_t step;
    UniformRow<T, S> row;
    __device__ __forceinline__ UniformRows(const T* first, int64_t step_) : p(first), step(step_) {
        if constexpr (kAhead) row.load(p);
    }
    __device__ __forceinline__ UniformRow<T, S> next(bool more) {
        UniformRow<T, S> now;
        if constexpr (kAhead) {
            now = row;
            if (more) p += step;
            row.load(p);
        } else {
            now.load(p);
            if (more) p += step;
        }
        return now;
    }
};

// A wave's channels: `c` of a lane is clamped to its group, `valid` says whether it is its own.
struct Channels {
    int group;
    unsigned c, two, four;    // the channel, and its offset in bytes in rows of 2- and 4-byte elements
    bool valid;
    __device__ __forceinline__ Channels(const SelectiveParams& p, int wave) {
        const int per = p.C / p.G, in = (wave % p.group_waves) * 64 + (int)(threadIdx.x & 63);
        group = wave / p.group_waves;
        valid = in < per;
        c = group * per + (valid ? in : per - 1);
        two = c * 2;
        four = c * 4;
    }
};
// A lane's place in a row at a uniform address: one scalar base and a 32-bit offset.  Both pass through registers by
// force at each use; the compiler else widens the offset once before the loop and adds it to every row in vectors.
template <typename T> __device__ __forceinline__ T* lane_bytes(T* row, unsigned bytes) {
    __attribute__((address_space(1))) T* global = (__attribute__((address_space(1))) T*)row;
    asm("" : "+s"(global), "+v"(bytes));
    return atb((T*)global, bytes);
}
template <typename T> __device__ __forceinline__ T* lane_of(T* row, const Channels& ch) {
    return lane_bytes(row, sizeof(T) == 2 ? ch.two : ch.four);
}
template <typename T> __device__ __forceinline__ T row_at(const T* row, const Channels& ch) { return *lane_of(row, ch); }
__device__ __forceinline__ void row_put(void* base, int64_t row_start, const Channels& ch, float x, bool as_bf16) {
    if (as_bf16) *lane_of((bf16*)base + row_start, ch) = (bf16)x;
    else *lane_of((float*)base + row_start, ch) = x;
}

template <int S> __device__ __forceinline__ void load_entries(float (&v)[S], const float* p) {
#pragma unroll
    for (int n = 0; n < S; n += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(p + n);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[n + j] = x[j];
    }
}
template <int S> __device__ __forceinline__ void store_entries(float* p, const float (&v)[S]) {
#pragma unroll
    for (int n = 0; n < S; n += 4) {
        const f32x4 x = {v[n], v[n + 1], v[n + 2], v[n + 3]};
        *reinterpret_cast<f32x4*>(p + n) = x;
    }
}
// States between launches lie four entries of all channels side by side, [S / 4][C][4], so that a wave moves whole lines.
template <int S> __device__ __forceinline__ void load_kept(float (&v)[S], const float* p, int64_t slot, int C, unsigned c) {
#pragma unroll
    for (int n = 0; n < S; n += 4) {
        const f32x4 x = *lane_bytes(reinterpret_cast<const f32x4*>(p + (slot * (S / 4) + n / 4) * C * 4), c * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[n + j] = x[j];
    }
}
template <int S> __device__ __forceinline__ void store_kept(float* p, int64_t slot, int C, unsigned c, const float (&v)[S]) {
#pragma unroll
    for (int n = 0; n < S; n += 4) {
        const f32x4 x = {v[n], v[n + 1], v[n + 2], v[n + 3]};
        *lane_bytes(reinterpret_cast<f32x4*>(p + (slot * (S / 4) + n / 4) * C * 4), c * 16) = x;
    }
}
// A in units of log 2, so that a decay is one multiply and one exponential.
template <int S> __device__ __forceinline__ void load_A(float (&A2)[S], const float* A) {
    load_entries<S>(A2, A);
#pragma unroll
    for (int n = 0; n < S; ++n) A2[n] *= kLog2e;
}

__device__ __forceinline__ float step_size(float raw, float bias, bool soft) {
    const float v = raw + bias;
    float s = softplus(v);
    asm("" : "+v"(s));                        // a select instead of a branch
    return soft ? s : v;
}

}  // namespace kda
