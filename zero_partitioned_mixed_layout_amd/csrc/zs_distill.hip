// zs_distill.hip -- distillation from a teacher's top logits for gfx950: the
// loss of every row and its gradient with respect to the student's logits,
// already multiplied by the device's loss scale.
//
// A row is read once: one workgroup keeps it in registers (up to 131,072
// 16-bit or 65,536 fp32 logits), takes the softmax's maximum and sum from
// there and writes the gradient from there, so a row moves 2 s V bytes and
// the kernel is bound by HBM.  Longer rows are read a second time.  The few
// positions the teacher or the label names are written after the others.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "zero_shard.h"
#include "zs_internal.h"
#include "zs_ops.h"

namespace {

using zs::f32x4;
using zs::u32x4;
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLowest = -3.402823466e38f; // -FLT_MAX
constexpr uint32_t kMaxTop = ZERO_DISTILL_MAX_TOP;

// c = log2(e), or log2(e) / temperature
__device__ __forceinline__ float exp_of(float x, float c) { return __builtin_amdgcn_exp2f(x * c); }

struct DistillArgs {
    const void *logits;
    void *grad;
    const void *idx;
    const void *top;
    const void *labels;
    const float *row_weight;
    const float *teacher_lse;
    const int32_t *log2_scale;
    float *loss;
    int32_t *flag;
    uint64_t rows, vocab, ld_logits, ld_grad, ld_idx, ld_top;
    uint32_t k;
    int idx_bytes, top_type, label_bytes;
    float tau, inv_tau, soft, hard;
    uint32_t splits; // workgroups per row
};

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// Elements of one 16-byte vector of T.
template <class T>
constexpr uint32_t kVec = 16 / sizeof(T);

// Vectors stay packed in registers and are unpacked where they are used.
// The row streams through once: nontemporal stores took 4096 x 50257 bfloat16
// rows from 188 to 175 us, nontemporal loads 4096 x 32000 from 114 to 110.
template <class T>
__device__ __forceinline__ u32x4 load_vec(const T *p) {
    if constexpr (sizeof(T) == 4)
        return __builtin_nontemporal_load((const u32x4_a4 *)p);
    else
        return __builtin_nontemporal_load((const u32x4_a2 *)p);
}
template <class T>
__device__ __forceinline__ void store_vec(T *p, const u32x4 &v) {
    if constexpr (sizeof(T) == 4)
        __builtin_nontemporal_store(v, (u32x4_a4 *)p);
    else
        __builtin_nontemporal_store(v, (u32x4_a2 *)p);
}
template <class T>
__device__ __forceinline__ void unpack(const u32x4 &v, float (&x)[kVec<T>]) {
    for (uint32_t i = 0; i < 4; i++) {
        if constexpr (sizeof(T) == 4) {
            x[i] = __uint_as_float(v[i]);
        } else {
            typedef T T2 __attribute__((ext_vector_type(2)));
            const T2 h = __builtin_bit_cast(T2, (uint32_t)v[i]);
            x[2 * i] = (float)h[0];
            x[2 * i + 1] = (float)h[1];
        }
    }
}
template <class T>
__device__ __forceinline__ u32x4 pack(const T (&x)[kVec<T>]) {
    u32x4 v;
    __builtin_memcpy(&v, x, 16);
    return v;
}

template <class T>
__device__ __forceinline__ int nonfinite(T g) {
    return !(fabsf((float)g) <= 3.402823466e38f);
}

// Softmax statistics of a set of values: their maximum (at least -FLT_MAX,
// so that a set of -inf alone gives sums of 0, never inf - inf), the sum of
// exp((z - max) / tau) and, where the label's term needs it too, the sum of
// exp(z - max).
struct Stats {
    float max, st, s1;
};

// Add N values: one rescaling of the sums where the maximum moved.
template <bool BOTH, uint32_t N>
__device__ __forceinline__ void add_values(Stats &s, const float (&x)[N], float ct) {
    float m = s.max;
    for (uint32_t e = 0; e < N; e++)
        m = fmaxf(m, x[e]);
    if (m > s.max) {
        s.st *= exp_of(s.max - m, ct);
        if (BOTH)
            s.s1 *= exp_of(s.max - m, kLog2e);
        s.max = m;
    }
    for (uint32_t e = 0; e < N; e++) {
        s.st += exp_of(x[e] - m, ct);
        if (BOTH)
            s.s1 += exp_of(x[e] - m, kLog2e);
    }
}

// The same over the 64 lanes of a wave.
template <bool BOTH>
__device__ __forceinline__ void join_wave(Stats &s, float ct) {
    float m = s.max;
    for (int d = 32; d > 0; d >>= 1)
        m = fmaxf(m, __shfl_xor(m, d));
    s.st *= exp_of(s.max - m, ct);
    if (BOTH)
        s.s1 *= exp_of(s.max - m, kLog2e);
    s.max = m;
    for (int d = 32; d > 0; d >>= 1) {
        s.st += __shfl_xor(s.st, d);
        if (BOTH)
            s.s1 += __shfl_xor(s.s1, d);
    }
}

__device__ __forceinline__ float sum_wave(float v) {
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// What a workgroup shares about its row.
struct Row {
    float wave_max[16], wave_st[16], wave_s1[16];
    float logp[kMaxTop]; // the teacher's log probability of entry j
    float zat[kMaxTop];  // the student's logit there
    int32_t at[kMaxTop]; // its position, or -1
    // whether an earlier entry, or a later one, names the same position
    uint8_t earlier[kMaxTop], later[kMaxTop];
    float mass, zlabel; // sum of the probabilities; the logit at the label
    int label_named;    // whether an entry names the label
};

// The first 64 of the teacher's entries, one a lane of one wave, and the
// row's own few values, as they lie in memory: asked for before the row's
// loads (loads return in order) and converted after those are under way.
struct Ahead {
    uint32_t idx_lo, idx_hi, top, label_lo, label_hi, lse;
};

__device__ __forceinline__ uint32_t raw_real(const void *p, int type, uint64_t i) {
    return type == ZERO_F32 ? ((const uint32_t *)p)[i] : ((const uint16_t *)p)[i];
}
__device__ __forceinline__ float real_of(uint32_t raw, int type) {
    if (type == ZERO_F32)
        return __uint_as_float(raw);
    if (type == ZERO_F16)
        return (float)__builtin_bit_cast(_Float16, (uint16_t)raw);
    return __uint_as_float(raw << 16);
}
__device__ __forceinline__ void raw_int(const void *p, int bytes, uint64_t i, uint32_t &lo,
                                        uint32_t &hi) {
    if (bytes == 8) {
        lo = ((const uint32_t *)p)[2 * i];
        hi = ((const uint32_t *)p)[2 * i + 1];
    } else {
        lo = ((const uint32_t *)p)[i];
        hi = 0;
    }
}
__device__ __forceinline__ int64_t int_of(uint32_t lo, uint32_t hi, int bytes) {
    return bytes == 8 ? (int64_t)((uint64_t)hi << 32 | lo) : (int64_t)(int32_t)lo;
}

__device__ __forceinline__ Ahead ask_ahead(const DistillArgs &a, uint64_t row, bool teacher) {
    Ahead r = {0, 0, 0, 0, 0, 0};
    const uint32_t lane = threadIdx.x & 63u;
    if (teacher && lane < a.k) {
        raw_int(a.idx, a.idx_bytes, row * a.ld_idx + lane, r.idx_lo, r.idx_hi);
        r.top = raw_real(a.top, a.top_type, row * a.ld_top + lane);
    }
    if (a.labels)
        raw_int(a.labels, a.label_bytes, row, r.label_lo, r.label_hi);
    if (a.teacher_lse)
        r.lse = __float_as_uint(a.teacher_lse[row]);
    return r;
}

// The row's label: -1 for none, kOutside for one past the vocabulary.
constexpr int32_t kOutside = INT32_MAX;
__device__ __forceinline__ int32_t label_of(const DistillArgs &a, const Ahead &r) {
    const int64_t l = a.labels ? int_of(r.label_lo, r.label_hi, a.label_bytes) : -1;
    return __builtin_amdgcn_readfirstlane(l < 0                     ? -1
                                          : l >= (int64_t)a.vocab ? kOutside
                                                                  : (int32_t)l);
}

// The teacher's entries of a row, by one wave on its own.
template <class T>
__device__ __forceinline__ void read_teacher(const DistillArgs &a, uint64_t row, const T *z,
                                             int32_t label, const Ahead &ahead, Row &sh) {
    const uint32_t lane = threadIdx.x & 63u;
    const int64_t V = (int64_t)a.vocab;
    const float zlabel = lane == 0 && label >= 0 && label != kOutside ? (float)z[label] : 0.0f;
    bool outside = false;
    float tmax = kLowest;
    for (uint32_t j = lane; j < a.k; j += 64) {
        uint32_t lo = ahead.idx_lo, hi = ahead.idx_hi, top = ahead.top;
        if (j >= 64) {
            raw_int(a.idx, a.idx_bytes, row * a.ld_idx + j, lo, hi);
            top = raw_real(a.top, a.top_type, row * a.ld_top + j);
        }
        const float t = real_of(top, a.top_type);
        int64_t p = int_of(lo, hi, a.idx_bytes);
        outside |= p >= V;
        if (p < 0 || p >= V || t == -INFINITY) // probability 0: as if absent
            p = -1;
        sh.at[j] = (int32_t)p;
        sh.earlier[j] = sh.later[j] = 0;
        sh.logp[j] = t;
        sh.zat[j] = p < 0 ? 0.0f : (float)z[p];
        if (p >= 0)
            tmax = fmaxf(tmax, t);
    }
    // log p = (t - base) / tau - lse, from the largest entry where the sum is
    // taken here: entries of the type's lowest value then stay finite
    float base = 0.0f, lse;
    if (a.teacher_lse) {
        lse = __uint_as_float(ahead.lse);
    } else {
        for (int d = 32; d > 0; d >>= 1)
            tmax = fmaxf(tmax, __shfl_xor(tmax, d));
        float sum = 0.0f;
        for (uint32_t j = lane; j < a.k; j += 64)
            if (sh.at[j] >= 0)
                sum += exp_of(sh.logp[j] - tmax, a.inv_tau * kLog2e);
        base = tmax;
        lse = logf(sum_wave(sum));
    }
    float mass = 0.0f;
    for (uint32_t j = lane; j < a.k; j += 64) {
        const float logp = sh.at[j] < 0 ? -INFINITY : (sh.logp[j] - base) * a.inv_tau - lse;
        mass += exp_of(logp, kLog2e);
        sh.logp[j] = logp;
    }
    mass = sum_wave(mass);
    if (__any(outside))
        mass = __builtin_nanf("");
    if (lane == 0) {
        sh.mass = mass;
        sh.zlabel = zlabel;
        sh.label_named = 0;
    }
}

// The row's gradient outside the named positions, ct exp((z - max) / tau) +
// c1 exp(z - max) (one exponential where both have the same temperature),
// and what the named ones need.
template <class T, bool BOTH>
struct Gradient {
    Stats s;
    float c_tau; // log2(e) / temperature
    float ct, c1;
    float unit, soft, hard, mass;
    // whether a value can overflow T (exponentials are at most 1), or is NaN
    bool check;

    __device__ __forceinline__ T at(float x) const {
        float g = ct * exp_of(x - s.max, c_tau);
        if (BOTH)
            g += c1 * exp_of(x - s.max, kLog2e);
        return (T)g;
    }
    // at a position with teacher probability p
    __device__ __forceinline__ T named(float x, float p, bool is_label) const {
        const float qt = exp_of(x - s.max, c_tau) / s.st;
        const float q1 = BOTH ? exp_of(x - s.max, kLog2e) / s.s1 : qt;
        return (T)(unit * (soft * (mass * qt - p) + hard * (q1 - (is_label ? 1.0f : 0.0f))));
    }
};

template <class T>
constexpr float kTypeMax = 3.3895313892515355e38f; // bfloat16 and fp32 (rounded down)
template <>
constexpr float kTypeMax<_Float16> = 65504.0f;

// Join the waves' statistics, after which every wave has the row's.
template <class T, bool BOTH>
__device__ __forceinline__ Gradient<T, BOTH> make_gradient(const DistillArgs &a, float weight,
                                                           int32_t label, Stats s, Row &sh) {
    const float c_tau = a.inv_tau * kLog2e;
    join_wave<BOTH>(s, c_tau);
    const uint32_t lane = threadIdx.x & 63u, waves = blockDim.x >> 6;
    if (lane == 0) {
        sh.wave_max[threadIdx.x >> 6] = s.max;
        sh.wave_st[threadIdx.x >> 6] = s.st;
        if (BOTH)
            sh.wave_s1[threadIdx.x >> 6] = s.s1;
    }
    const int k2 = a.log2_scale ? *a.log2_scale : 0;
    const int kc = k2 < -ZERO_LOG2_SCALE_MAX  ? -ZERO_LOG2_SCALE_MAX
                   : k2 > ZERO_LOG2_SCALE_MAX ? ZERO_LOG2_SCALE_MAX
                                              : k2;
    __syncthreads();
    s = {kLowest, 0.0f, 0.0f};
    if (lane < waves) {
        s.max = sh.wave_max[lane];
        s.st = sh.wave_st[lane];
        if (BOTH)
            s.s1 = sh.wave_s1[lane];
    }
    join_wave<BOTH>(s, c_tau);
    s = {uniform(s.max), uniform(s.st), uniform(BOTH ? s.s1 : s.st)};
    Gradient<T, BOTH> g;
    g.s = s;
    g.c_tau = c_tau;
    g.mass = uniform(sh.mass);
    g.hard = label < 0 ? 0.0f : label == kOutside ? __builtin_nanf("") : a.hard;
    g.unit = weight * __uint_as_float((uint32_t)(kc + 127) << 23);
    g.soft = a.soft * a.tau;
    const float c_soft = g.soft * g.mass / s.st, c_hard = g.hard / s.s1;
    g.ct = uniform(g.unit * (BOTH ? c_soft : c_soft + c_hard));
    g.c1 = uniform(g.unit * c_hard);
    g.check = !(fabsf(g.ct) + (BOTH ? fabsf(g.c1) : 0.0f) <= kTypeMax<T>);
    return g;
}

// The row's loss, by one wave.
template <class T, bool BOTH>
__device__ __forceinline__ void write_loss(const DistillArgs &a, const Gradient<T, BOTH> &g,
                                           const Row &sh, uint64_t row, float weight,
                                           int32_t label) {
    const uint32_t lane = threadIdx.x & 63u;
    const float log_st = logf(g.s.st);
    float kl = 0.0f;
    for (uint32_t j = lane; j < a.k; j += 64) {
        const float logp = sh.logp[j], p = exp_of(logp, kLog2e);
        if (p != 0.0f)
            kl += p * (logp - ((sh.zat[j] - g.s.max) * a.inv_tau - log_st));
    }
    kl = sum_wave(kl);
    // a NaN mass (an index outside) or hard weight (a label outside) stays
    float loss = a.soft * a.tau * a.tau * kl + g.mass * 0.0f;
    if (label >= 0)
        loss += g.hard * (logf(g.s.s1) - (sh.zlabel - g.s.max));
    if (lane == 0)
        a.loss[row] = loss * weight;
}

// Whether a non-finite value at i counts: one at a position that is written
// again does not.
__device__ __forceinline__ bool counts(const DistillArgs &a, const Row &sh, int32_t label,
                                       uint64_t i) {
    bool named = (int32_t)i == label;
#pragma unroll 1
    for (uint32_t j = 0; j < a.k; j++)
        named |= sh.at[j] == (int32_t)i;
    return !named;
}

// Which entries name the same position: every pair is looked at, the first
// entry by a lane and the second by a wave.
__device__ __forceinline__ void find_repeats(const DistillArgs &a, int32_t label, Row &sh) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint32_t j = threadIdx.x & 63u; j < a.k; j += 64) {
        const int32_t p = sh.at[j];
        if (p < 0)
            continue;
        if (p == label)
            sh.label_named = 1;
#pragma unroll 4
        for (uint32_t i = wave; i < a.k; i += blockDim.x >> 6)
            if (sh.at[i] == p) {
                if (i < j)
                    sh.earlier[j] = 1;
                else if (i > j)
                    sh.later[j] = 1;
            }
    }
}

// The named positions in [lo, hi), after the others: the first entry of a
// position writes the sum of all entries that name it.  Returns whether a
// value was not finite.
template <class T, bool BOTH>
__device__ __forceinline__ int write_named(const DistillArgs &a, const Gradient<T, BOTH> &g,
                                           const Row &sh, int32_t label, uint64_t lo, uint64_t hi,
                                           T *out) {
    int bad = 0;
    for (uint32_t j = threadIdx.x; j < a.k; j += blockDim.x) {
        const int32_t p = sh.at[j];
        if (p < 0 || (uint64_t)p < lo || (uint64_t)p >= hi || sh.earlier[j])
            continue;
        float pj = exp_of(sh.logp[j], kLog2e);
        if (sh.later[j])
#pragma unroll 1
            for (uint32_t i = j + 1; i < a.k; i++)
                pj += sh.at[i] == p ? exp_of(sh.logp[i], kLog2e) : 0.0f;
        const T v = g.named(sh.zat[j], pj, p == label);
        bad |= nonfinite(v);
        out[p] = v;
    }
    if (threadIdx.x == 64 && label >= 0 && !sh.label_named && (uint64_t)label >= lo &&
        (uint64_t)label < hi) {
        const T v = g.named(sh.zlabel, 0.0f, true);
        bad |= nonfinite(v);
        out[label] = v;
    }
    return bad;
}

template <class T>
__device__ __forceinline__ void write_zeros(T *out, uint64_t lo, uint64_t hi) {
    const u32x4 zero = {0, 0, 0, 0};
    for (uint64_t i = lo / kVec<T> + threadIdx.x; i < hi / kVec<T>; i += blockDim.x)
        store_vec(out + i * kVec<T>, zero);
    for (uint64_t i = hi / kVec<T> * kVec<T> + threadIdx.x; i < hi; i += blockDim.x)
        out[i] = (T)0.0f;
}

// NV > 0: the row in registers, NV vectors a thread (NT * NV hold it).
// NV = 0: rows of any length, read twice.
template <class T, bool BOTH, uint32_t NT, uint32_t NV>
__global__ __launch_bounds__(NT, NV <= 8 ? 8 : 4) void zs_distill_kernel(DistillArgs a) {
    constexpr uint32_t E = kVec<T>;
    __shared__ Row sh;
    const uint32_t tid = threadIdx.x;
    const uint64_t row = blockIdx.x / a.splits;
    const uint32_t part = blockIdx.x % a.splits;
    const uint64_t V = a.vocab;
    const T *z = (const T *)a.logits + row * a.ld_logits;
    T *out = (T *)a.grad + row * a.ld_grad;
    // this workgroup's columns, cut at whole vectors
    const uint64_t per = a.splits == 1 ? V : (V / a.splits + E) / E * E;
    const uint64_t lo = part * per < V ? part * per : V;
    const uint64_t hi = lo + per < V ? lo + per : V;
    // the first wave reads the teacher's part
    const bool teacher = tid < 64;
    float weight = a.row_weight ? a.row_weight[row] : 1.0f;
    const Ahead ahead = ask_ahead(a, row, teacher);
    auto masked = [&]() { // a masked row: nothing of it counts
        weight = uniform(weight);
        if (weight != 0.0f)
            return false;
        write_zeros(out, lo, hi);
        if (part == 0 && tid == 0)
            a.loss[row] = 0.0f;
        return true;
    };
    // with rows enough to fill the chip, masked ones are not read; with few,
    // what counts is that no load waits for another
    if (a.splits == 1 && masked())
        return;
    const uint32_t nv = (uint32_t)(V / E), rest = (uint32_t)(V % E);
    constexpr uint32_t kMinusInf =
        sizeof(T) == 4 ? 0xFF800000u : sizeof(T) == 2 && kTypeMax<T> < 1e5f ? 0xFC00FC00u : 0xFF80FF80u;
    u32x4 x[NV ? NV : 1];
    float f[E], last[1] = {-INFINITY}; // last: of the values after the last whole vector
    if constexpr (NV > 0) {
#pragma unroll
        for (uint32_t v = 0; v < NV; v++) {
            x[v] = u32x4{kMinusInf, kMinusInf, kMinusInf, kMinusInf};
            if (v * NT + tid < nv)
                x[v] = load_vec(z + (uint64_t)(v * NT + tid) * E);
        }
    }
    if (tid < rest)
        last[0] = (float)z[(uint64_t)nv * E + tid];
    if (a.splits != 1 && masked())
        return;
    const int32_t label = label_of(a, ahead);
    if (teacher)
        read_teacher(a, row, z, label, ahead, sh);
    Stats s = {kLowest, 0.0f, 0.0f};
    const float c_tau = a.inv_tau * kLog2e;
    if constexpr (NV > 0) {
#pragma unroll
        for (uint32_t v = 0; v < NV; v++) {
            unpack<T>(x[v], f);
            for (uint32_t e = 0; e < E; e++)
                s.max = fmaxf(s.max, f[e]);
        }
        s.max = fmaxf(s.max, last[0]);
#pragma unroll
        for (uint32_t v = 0; v < NV; v++) {
            asm volatile("" : "+v"(x[v])); // unpacked again, not kept unpacked
            unpack<T>(x[v], f);
            for (uint32_t e = 0; e < E; e++) {
                s.st += exp_of(f[e] - s.max, c_tau);
                if (BOTH)
                    s.s1 += exp_of(f[e] - s.max, kLog2e);
            }
        }
    } else {
        for (uint32_t i = tid; i < nv; i += NT) {
            unpack<T>(load_vec(z + (uint64_t)i * E), f);
            add_values<BOTH>(s, f, c_tau);
        }
    }
    add_values<BOTH>(s, last, c_tau);
    // every read of the row that another thread's write could meet (all but
    // the second reading of long rows, by the thread that writes there) lies
    // before the barrier in here
    const Gradient<T, BOTH> g = make_gradient<T, BOTH>(a, weight, label, s, sh);
    int bad = 0;
    auto write = [&](u32x4 z_in, uint64_t i) {
        T o[E];
        asm volatile("" : "+v"(z_in));
        unpack<T>(z_in, f);
        for (uint32_t e = 0; e < E; e++)
            o[e] = g.at(f[e]);
        store_vec(out + i * E, pack(o));
    };
    const uint32_t v0 = (uint32_t)(lo / E), v1 = (uint32_t)(hi / E);
    if constexpr (NV > 0) {
#pragma unroll
        for (uint32_t v = 0; v < NV; v++)
            if (v * NT + tid >= v0 && v * NT + tid < v1)
                write(x[v], v * NT + tid);
    } else {
        for (uint32_t i = v0 + tid; i < v1; i += NT)
            write(load_vec(z + (uint64_t)i * E), i);
    }
    if (hi == V && tid < rest) {
        out[(uint64_t)nv * E + tid] = g.at(last[0]);
    }
    if (g.check) { // rare: look through what this thread wrote, and nothing else:
                   // no barrier lies between.  From registers it wrote the vectors
                   // that are tid mod NT.
        static_assert((NT & (NT - 1)) == 0, "tid - v0 wraps");
        const uint32_t first = v0 + (NV > 0 ? (tid - v0) % NT : tid);
        for (uint32_t i = first; i < v1 && !bad; i += NT)
            for (uint32_t e = 0; e < E && !bad; e++)
                bad = nonfinite(out[(uint64_t)i * E + e]) &&
                      counts(a, sh, label, (uint64_t)i * E + e);
        if (hi == V && tid < rest && !bad)
            bad = nonfinite(out[(uint64_t)nv * E + tid]) &&
                  counts(a, sh, label, (uint64_t)nv * E + tid);
    }
    find_repeats(a, label, sh);
    __syncthreads();
    if (part == 0 && tid >= NT - 64) // the first waves write what is named
        write_loss(a, g, sh, row, weight, label);
    bad |= write_named(a, g, sh, label, lo, hi, out);
    zs::raise_flag(a.flag, bad);
}

// Workgroups per row: one from kFullRows rows on; below, as many as keep
// within that many workgroups (one round of the chip), each with at least
// kMinSplit elements of the row to write (every one of them reads the whole
// row for its statistics, from cache, which needs no second launch and no
// memory between the two).  60 rows of 131,072: 21 us, with 512 workgroups 38.
// In place a row stays with one workgroup, which has read all of it before it
// writes: 5 x 50257 fp16 12.5 us against 10.5 apart, 60 x 131072 21.1 and 19.4.
constexpr uint64_t kFullRows = 256;
constexpr uint64_t kMinSplit = 4096;

uint32_t splits_of(uint64_t rows, uint64_t vocab) {
    if (rows >= kFullRows)
        return 1;
    const uint64_t want = kFullRows / rows, most = vocab / kMinSplit;
    const uint64_t s = want < most ? want : most;
    return s < 1 ? 1 : (uint32_t)s;
}

template <class T, bool BOTH, uint32_t NT, uint32_t NV>
void launch(const DistillArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((zs_distill_kernel<T, BOTH, NT, NV>),
                       dim3((uint32_t)(a.rows * a.splits)), dim3(NT), 0, st, a);
}

// The kernel whose registers hold the row.  4096 x 50257 bfloat16, top 64: 1024
// threads of 7 vectors 143 us (5.8 TB/s, bound by HBM), 512 of 13 199, 768 of 9
// 197.  5 x 50257 fp16 takes 11.7, the latency of the teacher's list, the row,
// the statistics and the stores one after the other.
template <class T, bool BOTH>
void launch_for(const DistillArgs &a, hipStream_t st) {
    const uint64_t n = a.vocab / kVec<T>;
    if (n <= 256 * 2)
        launch<T, BOTH, 256, 2>(a, st);
    else if (n <= 256 * 8)
        launch<T, BOTH, 256, 8>(a, st);
    else if (n <= 256 * 16)
        launch<T, BOTH, 256, 16>(a, st);
    else if (n <= 1024 * 7)
        launch<T, BOTH, 1024, 7>(a, st);
    else if (n <= 1024 * 16)
        launch<T, BOTH, 1024, 16>(a, st);
    else
        launch<T, BOTH, 1024, 0>(a, st);
}

template <class T>
void launch_typed(const DistillArgs &a, bool both, hipStream_t st) {
    both ? launch_for<T, true>(a, st) : launch_for<T, false>(a, st);
}

bool half_or_float(int t) { return t == ZERO_F32 || t == ZERO_F16 || t == ZERO_BF16; }

// Byte range of a rows x cols array with a row pitch, elements of es bytes.
int range_of(const void *p, uint64_t es, uint64_t rows, uint64_t cols, uint64_t ld, bool written,
             zs::Range *r) {
    *r = {0, 0, written};
    if (ld < cols)
        return ZERO_EINVAL;
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if (!p || (uintptr_t)p % es)
        return ZERO_EINVAL;
    uint64_t b;
    if (__builtin_mul_overflow(rows - 1, ld, &b) || __builtin_add_overflow(b, cols, &b) ||
        __builtin_mul_overflow(b, es, &b) || (uintptr_t)p + b < (uintptr_t)p)
        return ZERO_EOVERFLOW;
    *r = {(uintptr_t)p, (uintptr_t)p + b, written};
    return ZERO_OK;
}

} // namespace

extern "C" int zero_distill_loss(const zero_distill *d, void *stream) {
    if (!d || !half_or_float(d->logits_type))
        return ZERO_EINVAL;
    // a weight of 0 leaves its term out, and its arrays unread
    const bool soft = d->soft_weight != 0.0 && d->top > 0;
    const bool hard = d->hard_weight != 0.0 && d->labels != nullptr;
    const uint64_t rows = d->rows, V = d->vocab;
    if (!(d->temperature > 0.0) || !(d->temperature <= 1e6) || !(d->temperature >= 1e-6) ||
        !__builtin_isfinite((float)d->soft_weight) || !__builtin_isfinite((float)d->hard_weight))
        return ZERO_EINVAL;
    // a workgroup a row, of up to 1024 threads (rows that are split are few)
    if (d->top > kMaxTop || rows > zs::kMaxWorkgroups1024 || V > 0x7FFFFFFFull)
        return ZERO_EOVERFLOW;
    const uint64_t es = d->logits_type == ZERO_F32 ? 4 : 2;
    zs::Range r[10];
    int rc, n = 0;
    if ((rc = range_of(d->grad, es, rows, V, d->ld_grad, true, &r[n++])) != ZERO_OK ||
        (rc = range_of(d->logits, es, rows, V, d->ld_logits, false, &r[n++])) != ZERO_OK)
        return rc;
    const bool in_place = d->grad == d->logits && d->ld_grad == d->ld_logits;
    if (in_place)
        n--; // each workgroup has read its row before it writes it
    if ((rc = range_of(d->loss, 4, rows, rows ? 1 : 0, 1, true, &r[n++])) != ZERO_OK)
        return rc;
    if (soft) {
        if ((d->idx_bytes != 4 && d->idx_bytes != 8) || !half_or_float(d->top_type))
            return ZERO_EINVAL;
        if ((rc = range_of(d->top_idx, d->idx_bytes, rows, d->top, d->ld_idx, false, &r[n++])) !=
                ZERO_OK ||
            (rc = range_of(d->top_logits, d->top_type == ZERO_F32 ? 4 : 2, rows, d->top,
                           d->ld_top, false, &r[n++])) != ZERO_OK)
            return rc;
        if (d->teacher_lse &&
            (rc = range_of(d->teacher_lse, 4, rows, 1, 1, false, &r[n++])) != ZERO_OK)
            return rc;
    }
    if (hard) {
        if (d->label_bytes != 4 && d->label_bytes != 8)
            return ZERO_EINVAL;
        if ((rc = range_of(d->labels, d->label_bytes, rows, 1, 1, false, &r[n++])) != ZERO_OK)
            return rc;
    }
    if (d->row_weight &&
        (rc = range_of(d->row_weight, 4, rows, 1, 1, false, &r[n++])) != ZERO_OK)
        return rc;
    if (d->scale) {
        if ((uintptr_t)d->scale % 4)
            return ZERO_EINVAL;
        r[n++] = {(uintptr_t)d->scale, (uintptr_t)d->scale + sizeof(zero_loss_scale), false};
    }
    if (d->nonfinite_flag) {
        if ((uintptr_t)d->nonfinite_flag % 4)
            return ZERO_EINVAL;
        r[n++] = {(uintptr_t)d->nonfinite_flag, (uintptr_t)d->nonfinite_flag + 4, true};
    }
    if (zs::writes_overlap(r, (size_t)n))
        return ZERO_EINVAL;
    if (rows == 0 || V == 0)
        return rows == 0 ? ZERO_OK : ZERO_EINVAL;
    DistillArgs a;
    a.logits = d->logits;
    a.grad = d->grad;
    a.idx = d->top_idx;
    a.top = d->top_logits;
    a.labels = hard ? d->labels : nullptr;
    a.row_weight = d->row_weight;
    a.teacher_lse = soft ? d->teacher_lse : nullptr;
    a.log2_scale = d->scale ? &d->scale->log2_scale : nullptr;
    a.loss = d->loss;
    a.flag = d->nonfinite_flag;
    a.rows = rows;
    a.vocab = V;
    a.ld_logits = d->ld_logits;
    a.ld_grad = d->ld_grad;
    a.ld_idx = d->ld_idx;
    a.ld_top = d->ld_top;
    a.k = soft ? d->top : 0;
    a.idx_bytes = d->idx_bytes;
    a.top_type = d->top_type;
    a.label_bytes = d->label_bytes;
    a.tau = (float)d->temperature;
    a.inv_tau = (float)(1.0 / d->temperature);
    a.soft = soft ? (float)d->soft_weight : 0.0f;
    a.hard = hard ? (float)d->hard_weight : 0.0f;
    a.splits = in_place ? 1 : splits_of(rows, V);
    const bool both = hard && d->temperature != 1.0;
    hipStream_t st = (hipStream_t)stream;
    if (d->logits_type == ZERO_F32)
        launch_typed<float>(a, both, st);
    else if (d->logits_type == ZERO_F16)
        launch_typed<_Float16>(a, both, st);
    else
        launch_typed<__bf16>(a, both, st);
    return hipGetLastError() == hipSuccess ? ZERO_OK : ZERO_EHIP;
}
