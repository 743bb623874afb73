// Gradient norm and clip of many adapters at once: tensors stacked by slot,
// [L][m]; slot i's norm runs over every tensor's row i.
//   norm[i] = sqrt(sum g^2);  out = round(g * min(1, max_norm[i] / (norm[i] + 1e-6)))
// Work-group = (tensor, chunk of kChunk elements of one slot's row).  Both
// passes stream their bytes once and are bound by HBM: 320 tensors, 453 MB, 83 us
// (5.4 TB/s) for the norm's and 160 us (5.7 TB/s) for the clip's.  Squares are summed in
// 64 bits (no overflow or underflow of a square, and no error that grows with
// the number of elements; the fp64 rate is far above what the bytes need), in
// a fixed order: partial sums [L][items], added by the slot's last work-group.
#include "linear.hpp"

#include "../../include/adapter_apply.h"

namespace aa {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;
constexpr int kMaxTensors = 96;       // per launch (kernel arguments)
constexpr int64_t kCountItems = 2048;
constexpr int32_t kMaxItems = 1 << 23; // per launch (grid times threads below 2^32)

typedef float floatx4_t __attribute__((ext_vector_type(4)));

struct GradArgs {
    const void *g[kMaxTensors];
    void *out[kMaxTensors];
    int64_t m[kMaxTensors];
    int32_t item[kMaxTensors + 1];    // first item (chunk) of each tensor
    int32_t n;
};

__device__ __forceinline__ int tensor_of(const GradArgs &a, int item) {
    int lo = 0, hi = a.n;             // a.item[lo] <= item < a.item[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.item[mid] <= item) lo = mid; else hi = mid;
    }
    return lo;
}

// 16 bytes of a row: 4 (fp32) or 8 (bf16) values.
template <bool BF16>
struct Vec {
    static constexpr int kN = BF16 ? 8 : 4;
    float v[kN];
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        if (BF16) {
            const uint4 u = ldg<uint4>(static_cast<const uint16_t *>(p) + i);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) { v[2 * k] = bf16_lo(w[k]); v[2 * k + 1] = bf16_hi(w[k]); }
        } else {
            const floatx4_t u = ldg<floatx4_t>(static_cast<const float *>(p) + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = u[k];
        }
    }
    __device__ __forceinline__ void store(void *p, int64_t i) const {
        if (BF16) {
            stg_nt(static_cast<uint16_t *>(p) + i,
                   make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
        } else {
            stg_nt(static_cast<float *>(p) + i,
                   make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                              __float_as_uint(v[3])));
        }
    }
};
template <bool BF16>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    return BF16 ? bf16_to_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store1(void *p, int64_t i, float v) {
    if (BF16) static_cast<uint16_t *>(p)[i] = (uint16_t)f32_to_bf16_rne(v);
    else static_cast<float *>(p)[i] = v;
}
template <bool BF16>
__device__ __forceinline__ bool aligned16(const void *p, int64_t i) {
    return ((reinterpret_cast<uintptr_t>(p) + i * (BF16 ? 2 : 4)) & 15) == 0;
}

// Sum over the work-group, the same order every time; valid on thread 0.
__device__ __forceinline__ double group_sum(double v, double *s) {
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    return s[0] + s[1] + s[2] + s[3];
}

// With count (few items): partial sums go to device-coherent memory (another
// XCD's work-group reads them), and the work-group that completes a slot's count
// adds them in order, writes the norm and leaves the count zero for the next
// call.  Without: k_grad_norm adds them.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void k_grad_sq(GradArgs a, double *part, int32_t *count, int64_t per_slot,
                                                      int64_t item0, float *norm) {
    constexpr int V = Vec<BF16>::kN, IT = kChunk / (kThreads * V);
    __shared__ double s_sum[kThreads / 64];
    const int t = tensor_of(a, blockIdx.x), slot = blockIdx.y, tid = threadIdx.x;
    const int64_t m = a.m[t], c0 = (int64_t)(blockIdx.x - a.item[t]) * kChunk;
    const int64_t base = slot * m + c0, len = min((int64_t)kChunk, m - c0);
    const void *g = a.g[t];
    double acc = 0.0;
    if (aligned16<BF16>(g, base)) {
        Vec<BF16> v[IT];
        if (len == kChunk) {
#pragma unroll
            for (int i = 0; i < IT; ++i) v[i].load(g, base + (int64_t)(i * kThreads + tid) * V);
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) acc += (double)v[i].v[k] * (double)v[i].v[k];
        } else {
            const int64_t whole = len / V;
            for (int64_t i = tid; i < whole; i += kThreads) {
                v[0].load(g, base + i * V);
#pragma unroll
                for (int k = 0; k < V; ++k) acc += (double)v[0].v[k] * (double)v[0].v[k];
            }
            for (int64_t i = whole * V + tid; i < len; i += kThreads) {
                const double x = load1<BF16>(g, base + i);
                acc += x * x;
            }
        }
    } else {
        for (int64_t i = tid; i < len; i += kThreads) {
            const double x = load1<BF16>(g, base + i);
            acc += x * x;
        }
    }
    const double sum = group_sum(acc, s_sum);
    __shared__ int s_last;
    double *p = part + slot * per_slot;
    if (!count) {
        if (tid == 0) p[item0 + blockIdx.x] = sum;
        return;
    }
    if (tid == 0) {
        __hip_atomic_store(p + item0 + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // stored before it is counted
        const int done = __hip_atomic_fetch_add(count + slot, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = done + 1 == per_slot;
    }
    __syncthreads();
    if (!s_last) return;
    acc = 0.0;
    for (int64_t i = tid; i < per_slot; i += kThreads)
        acc += __hip_atomic_load(p + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const double total = group_sum(acc, s_sum);
    if (tid == 0) {
        norm[slot] = (float)sqrt(total);
        __hip_atomic_store(count + slot, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

__global__ __launch_bounds__(kThreads) void k_grad_norm(const double *part, int64_t per_slot, float *norm) {
    __shared__ double s_sum[kThreads / 64];
    double acc = 0.0;
    const double *p = part + blockIdx.x * per_slot;
    for (int64_t i = threadIdx.x; i < per_slot; i += kThreads) acc += p[i];
    const double sum = group_sum(acc, s_sum);
    if (threadIdx.x == 0) norm[blockIdx.x] = (float)sqrt(sum);
}

// out may be the gradient itself; a factor of one then leaves it as it is.
// A NaN norm or limit gives a NaN factor.  Work-groups go backwards over the
// tensors, so that what the norm read last is still in the cache.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void k_grad_clip(GradArgs a, const float *norm, const float *max_norm) {
    constexpr int V = Vec<BF16>::kN, IT = kChunk / (kThreads * V);
    const int item = gridDim.x - 1 - blockIdx.x, slot = gridDim.y - 1 - blockIdx.y;
    const int t = tensor_of(a, item), tid = threadIdx.x;
    const int64_t m = a.m[t], c0 = (int64_t)(item - a.item[t]) * kChunk;
    const int64_t base = slot * m + c0, len = min((int64_t)kChunk, m - c0);
    const void *g = a.g[t];
    void *o = a.out[t];
    float c = max_norm[slot] / (norm[slot] + 1e-6f);
    if (c >= 1.f) c = 1.f;
    if (o == g && c == 1.f) return;
    if (aligned16<BF16>(g, base) && aligned16<BF16>(o, base)) {
        Vec<BF16> v[IT];
        if (len == kChunk) {
#pragma unroll
            for (int i = 0; i < IT; ++i) v[i].load(g, base + (int64_t)(i * kThreads + tid) * V);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
#pragma unroll
                for (int k = 0; k < V; ++k) v[i].v[k] *= c;
                v[i].store(o, base + (int64_t)(i * kThreads + tid) * V);
            }
        } else {
            const int64_t whole = len / V;
            for (int64_t i = tid; i < whole; i += kThreads) {
                v[0].load(g, base + i * V);
#pragma unroll
                for (int k = 0; k < V; ++k) v[0].v[k] *= c;
                v[0].store(o, base + i * V);
            }
            for (int64_t i = whole * V + tid; i < len; i += kThreads)
                store1<BF16>(o, base + i, load1<BF16>(g, base + i) * c);
        }
    } else {
        for (int64_t i = tid; i < len; i += kThreads)
            store1<BF16>(o, base + i, load1<BF16>(g, base + i) * c);
    }
}

inline int64_t chunks(int64_t m) { return (m + kChunk - 1) / kChunk; }

// Fills `a` with tensors [from, ...) that fit one launch; returns the next.
int32_t fill(GradArgs &a, void *const *out, const void *const *g, const int64_t *m, int32_t from, int32_t n) {
    a.n = 0;
    a.item[0] = 0;
    while (from < n && a.n < kMaxTensors) {
        const int64_t c = chunks(m[from]);
        if (a.item[a.n] + c > kMaxItems) break;
        if (c) {
            a.g[a.n] = g[from];
            a.out[a.n] = out ? out[from] : nullptr;
            a.m[a.n] = m[from];
            a.item[a.n + 1] = a.item[a.n] + (int32_t)c;
            ++a.n;
        }
        ++from;
    }
    return from;
}

}  // namespace

int64_t grad_items(const int64_t *m, int32_t n, int32_t L) {
    int64_t p = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (m[i] < 0 || m[i] > (int64_t)kMaxItems * kChunk) return -1;
        p += chunks(m[i]);
        if (p > INT32_MAX) return -1;             // counted in 32 bits
    }
    return p * L;
}

hipError_t launch_grad_norm(const void *const *g, const int64_t *m, int32_t n, int32_t L, int32_t dtype,
                            int32_t *count, double *part, float *norm, hipStream_t st) {
    const int64_t per_slot = grad_items(m, n, 1);
    // One launch fewer while the counting costs less than a launch: the counts
    // of a slot are adds to one address, one after the other (320 tensors, 13824
    // items: 4 x 50 us with counts, 4 x 21 and 5 us without).
    const bool joined = per_slot > 0 && per_slot * L <= kCountItems;
    if (!joined) count = nullptr;
    int64_t item0 = 0;
    for (int32_t i = 0; i < n;) {
        GradArgs a{};
        i = fill(a, nullptr, g, m, i, n);
        if (a.n == 0) continue;
        const dim3 grid((unsigned)a.item[a.n], (unsigned)L);
        if (dtype == LORA_DT_BF16)
            hipLaunchKernelGGL(k_grad_sq<true>, grid, dim3(kThreads), 0, st, a, part, count, per_slot, item0, norm);
        else
            hipLaunchKernelGGL(k_grad_sq<false>, grid, dim3(kThreads), 0, st, a, part, count, per_slot, item0, norm);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        item0 += a.item[a.n];
    }
    if (joined) return hipSuccess;
    hipLaunchKernelGGL(k_grad_norm, dim3((unsigned)L), dim3(kThreads), 0, st, part, per_slot, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(void *const *out, const void *const *g, const int64_t *m, int32_t n,
                            int32_t L, const float *norm, const float *max_norm, int32_t dtype,
                            hipStream_t st) {
    // the groups of tensors, last group first
    for (int32_t end = n; end > 0;) {
        GradArgs a{};
        int32_t from = end, items = 0, used = 0;
        while (from > 0) {
            const int64_t c = chunks(m[from - 1]);
            if (used + (c > 0) > kMaxTensors || items + c > kMaxItems) break;
            --from;
            items += (int32_t)c;
            used += c > 0;
        }
        fill(a, out, g, m, from, end);
        end = from;
        if (a.n == 0) continue;
        const dim3 grid((unsigned)a.item[a.n], (unsigned)L);
        if (dtype == LORA_DT_BF16) hipLaunchKernelGGL(k_grad_clip<true>, grid, dim3(kThreads), 0, st, a, norm, max_norm);
        else hipLaunchKernelGGL(k_grad_clip<false>, grid, dim3(kThreads), 0, st, a, norm, max_norm);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace aa
