// What the forward and the backward norm kernels share: row sums, loads and
// stores of a row's columns, gates, launch shapes.
#pragma once
#include <algorithm>
#include <atomic>

#include "elem.cuh"
#include "kernels.cuh"
#include "norm.cuh"

namespace moe {
namespace {

// Sums over the threads of one row (a warp, or the whole block): the warps'
// sums meet in shared memory, in one of two buffers by turns, so that one
// barrier does; every warp adds them in the same order.
// MAXW: the most warps of a block; entries of absent warps are zero throughout.
template <int MAXW>
struct RowSum {
  float* smem;  // [2][MAXW * 8]
  int threads_per_row, parity;

  __device__ __forceinline__ RowSum(float* s, int tpr) : smem(s), threads_per_row(tpr), parity(0) {
    if (tpr <= 32) return;
    for (int i = threadIdx.x; i < 2 * MAXW * 8; i += blockDim.x) s[i] = 0.f;
    __syncthreads();
  }

  __device__ __forceinline__ float one(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (threads_per_row <= 32) return v;
    float* s = smem + parity * (MAXW * 8);
    parity ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float4 f = *reinterpret_cast<const float4*>(s);
#pragma unroll
    for (int w = 4; w < MAXW; w += 4) {
      const float4 g = *reinterpret_cast<const float4*>(s + w);
      f.x += g.x;
      f.y += g.y;
      f.z += g.z;
      f.w += g.w;
    }
    return (f.x + f.y) + (f.z + f.w);
  }

  // Six sums: a lane hands half of its values to a partner until one is left
  // (9 shuffles instead of 30): value lane >> 2.
  __device__ __forceinline__ void six(float (&v)[6]) {
    const int lane = threadIdx.x & 31;
    float t[8] = {v[0], v[1], v[2], v[3], v[4], v[5], 0.f, 0.f};
#pragma unroll
    for (int half = 4; half >= 1; half >>= 1) {
      const int off = 4 * half;
      const bool upper = lane & off;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float give = upper ? t[i] : t[i + half];
        const float keep = upper ? t[i + half] : t[i];
        t[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
      }
    }
    float x = t[0];
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    // lane l now holds the warp's sum of value l >> 2
    if (threads_per_row > 32) {
      float* s = smem + parity * (MAXW * 8);
      parity ^= 1;
      if ((lane & 3) == 0) s[(threadIdx.x >> 5) * 8 + (lane >> 2)] = x;
      __syncthreads();
      s += (lane & 3) * 8 + (lane >> 2);
      x = s[0];
#pragma unroll
      for (int w = 4; w < MAXW; w += 4) x += s[w * 8];
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, x, 4 * i);
  }
};

// The elements of a row that one thread holds: with VEC, NPT / 8 runs of 8
// columns, run k at (k * threads + tid) * 8; else column j * threads + tid.
template <int NPT, bool VEC>
struct Cols {
  int tid, threads, d;
  __device__ __forceinline__ int at(int j) const {
    return VEC ? ((j >> 3) * threads + tid) * 8 + (j & 7) : j * threads + tid;
  }
  __device__ __forceinline__ bool in(int j) const { return at(j) < d; }
};

// This thread's elements of a row in global or (SMEM) shared memory.
template <typename T, bool SMEM = false, int NPT, bool VEC>
__device__ __forceinline__ void load_row(const Cols<NPT, VEC>& c, const T* p, float (&f)[NPT]) {
  if (VEC) {
    Raw8<T> raw[NPT / 8];
#pragma unroll
    for (int k = 0; k < NPT / 8; ++k) {
      if (SMEM)
        raw[k] = *reinterpret_cast<const Raw8<T>*>(p + c.at(8 * k));  // the ring holds zeros past the last column
      else
        raw[k] = c.in(8 * k) ? load_raw8<T>(p + c.at(8 * k)) : zero_raw8<T>();
    }
#pragma unroll
    for (int k = 0; k < NPT / 8; ++k) {
      float t[8];
      widen8(raw[k], t);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[8 * k + j] = t[j];
    }
  } else {
    T raw[NPT];
#pragma unroll
    for (int j = 0; j < NPT; ++j) raw[j] = c.in(j) ? p[c.at(j)] : from_f32<T>(0.f);
#pragma unroll
    for (int j = 0; j < NPT; ++j) f[j] = to_f32(raw[j]);
  }
}

// This thread's elements of a row, global to shared memory, asynchronously;
// zeros past the last column.
template <typename T, int NPT>
__device__ __forceinline__ void copy_row(const Cols<NPT, true>& c, T* dst, const T* src) {
#pragma unroll
  for (int k = 0; k < NPT / 8; ++k) {
    if (!c.in(8 * k)) {
      *reinterpret_cast<Raw8<T>*>(dst + c.at(8 * k)) = zero_raw8<T>();
      continue;
    }
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst + c.at(8 * k)));
    const T* from = src + c.at(8 * k);
#pragma unroll
    for (int b = 0; b < static_cast<int>(sizeof(T)) / 2; ++b)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16 * b),
                   "l"(reinterpret_cast<uint64_t>(from) + 16 * b)
                   : "memory");
  }
}

template <typename T, int NPT, bool VEC>
__device__ __forceinline__ void store_row(const Cols<NPT, VEC>& c, T* p, const float (&f)[NPT]) {
  if (VEC) {
#pragma unroll
    for (int k = 0; k < NPT / 8; ++k) {
      float t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = f[8 * k + j];
      if (c.in(8 * k)) store8(p + c.at(8 * k), t);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NPT; ++j)
      if (c.in(j)) p[c.at(j)] = from_f32<T>(f[j]);
  }
}

// Sum of a token's terms, ld elements apart.
template <typename A, bool SMEM, int NPT, bool VEC>
__device__ __forceinline__ void load_terms(const Cols<NPT, VEC>& c, const A* p, int ld, int terms, float (&z)[NPT]) {
  load_row<A, SMEM>(c, p, z);
#pragma unroll 4
  for (int m = 1; m < terms; ++m) {
    float f[NPT];
    load_row<A, SMEM>(c, p + static_cast<long long>(m) * ld, f);
#pragma unroll
    for (int j = 0; j < NPT; ++j) z[j] += f[j];
  }
}

// A gate, or the sigmoid of it (h: see sigmoid_approx).  FULL: by the full
// exponential, where a result has 32 bits and depends on the gate element by
// element; else by the approximate one, which 16-bit results do not show.  What
// w_post's gradient, a 32-bit sum over tokens, takes from 16-bit terms and gates
// is as exact as their part of it.
template <bool FULL>
__device__ __forceinline__ float gate_value(float x, int sigmoid, float& h) {
  h = x;
  return sigmoid ? (FULL ? sigmoid_full(x, h) : sigmoid_approx(x, h)) : x;
}

// Raw gates of the elements the thread holds.
template <typename A, bool SMEM, int NPT, bool VEC>
__device__ __forceinline__ void load_raw_gates(const Cols<NPT, VEC>& c, const void* p, int f32, float (&g)[NPT]) {
  if (f32)
    load_row<float, SMEM>(c, static_cast<const float*>(p), g);
  else
    load_row<A, SMEM>(c, static_cast<const A*>(p), g);
}
template <typename A, typename Args>
__device__ __forceinline__ float raw_token_gate(const Args& a, long long t) {
  return a.gate_f32 ? static_cast<const float*>(a.gate)[t] : to_f32(static_cast<const A*>(a.gate)[t]);
}

// Gate of every element the thread holds, from a row of gates.
template <typename A, bool SMEM, bool FULL, int NPT, bool VEC>
__device__ __forceinline__ void load_gates(const Cols<NPT, VEC>& c, const void* p, int f32, int sigmoid,
                                           float (&g)[NPT]) {
  load_raw_gates<A, SMEM>(c, p, f32, g);
  float h;
  if (sigmoid)
#pragma unroll
    for (int j = 0; j < NPT; ++j) g[j] = gate_value<FULL>(g[j], 1, h);
}

// The backward pass needs a sigmoid g, and g (1 - g), in which 1 - g taken from
// a rounded g near 1 has few digits left (7 % off at a gate of 14).  It holds
// gates folded, in one register, as the h of sigmoid_approx (without a sigmoid,
// the gate itself).
__device__ __forceinline__ float unfold_gate(float h, int sigmoid) {
  return sigmoid && __float_as_int(h) < 0 ? h + 1.0f : h;
}
__device__ __forceinline__ float fold_slope(float h) { return fabsf(h) - h * h; }  // g (1 - g)
// Folded gates h of the elements the thread holds, and the gates g.
template <typename A, bool SMEM, bool FULL, int NPT, bool VEC>
__device__ __forceinline__ void load_folded(const Cols<NPT, VEC>& c, const void* p, int f32, int sigmoid,
                                            float (&h)[NPT], float (&g)[NPT]) {
  load_raw_gates<A, SMEM>(c, p, f32, g);
  if (sigmoid) {
#pragma unroll
    for (int j = 0; j < NPT; ++j) g[j] = gate_value<FULL>(g[j], 1, h[j]);
  } else {
#pragma unroll
    for (int j = 0; j < NPT; ++j) h[j] = g[j];
  }
}
template <typename A, typename Args>
__device__ __forceinline__ const char* gate_row(const Args& a, long long t) {
  return static_cast<const char*>(a.gate) + t * a.d * (a.gate_f32 ? 4 : static_cast<int>(sizeof(A)));
}

// A kernel's kind of gate, compiled in: GateKind, or a gate for each element in 32
// bits where the block has 16 (its gradient has 32 too); -1: as the call says.
constexpr int kGateFull32 = 4;

// Rows of a block's ring in shared memory: stage s holds one row of every
// input that has one, at the byte offsets of `at`.
struct Ring {
  int stages, stage_bytes;
};
// Columns of a row in the ring: all that its threads could hold.
__host__ __device__ inline int ring_cols(int npt, int threads_per_row) { return npt * threads_per_row; }

// Threads that share a row, and rows of a block: 8 elements to a thread up to
// 4096 columns, else 16 (up to 512 threads, beyond 8192 columns up to 1024; rows
// that are not vector-aligned take the kernel compiled for 1024 from 4097 on);
// rows of at most 32 threads are one warp's each, four to a block.  Of blocks
// that stay, as many as fill an SM: forward 1024 threads of 8 elements (64
// registers) or 512 of 16 (110), backward 512 (128 at most).
struct Shape {
  int npt, max_threads, threads_per_row, rows_per_block, threads;
};
Shape shape_of(int d) {
  Shape s;
  s.npt = d <= 4096 ? 8 : 16;
  s.max_threads = d <= 8192 ? 512 : 1024;
  s.threads_per_row = ((d + s.npt - 1) / s.npt + 31) / 32 * 32;
  s.rows_per_block = s.threads_per_row <= 32 ? 4 : 1;
  s.threads = s.threads_per_row * s.rows_per_block;
  return s;
}
// Through the ring, rows of more than 2048 columns go 16 elements to a thread.
Shape pipe_shape_of(int d) {
  Shape s = shape_of(d);
  s.npt = d <= 2048 ? 8 : 16;
  s.threads_per_row = ((d + s.npt - 1) / s.npt + 31) / 32 * 32;
  s.rows_per_block = s.threads_per_row <= 32 ? 4 : 1;
  s.threads = s.threads_per_row * s.rows_per_block;
  return s;
}
constexpr int kFwdThreadsPerSm = 1024, kBwdThreadsPerSm = 512;
int blocks_per_sm(const Shape& s, int threads_per_sm) { return std::max(1, std::min(16, threads_per_sm / s.threads)); }

// Stages of a block's ring: up to three, as its share of shared memory holds;
// none (rows straight from global memory) when not one fits.
constexpr int kRingBytes = 208 * 1024;
Ring ring_of(long long row_bytes, const Shape& s, int per_sm) {
  const long long stage = row_bytes * s.rows_per_block;
  const long long fit = std::min<long long>(3, kRingBytes / per_sm / stage);
  return Ring{static_cast<int>(fit), static_cast<int>(row_bytes)};
}

// Launches KERNEL with a ring; its shared memory beyond what needs no opting in
// is asked for once per device.
template <auto KERNEL, typename Args>
cudaError_t launch_ring(int blocks, const Shape& s, const Ring& ring, const Args& a, cudaStream_t stream) {
  static std::atomic<unsigned long long> opted{0};  // a bit for each device
  const size_t smem = static_cast<size_t>(ring.stages) * ring.stage_bytes * s.rows_per_block;
  if (smem > 40 * 1024) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev > 63 || !(opted.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
      if (e != cudaSuccess) return e;
      opted.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  return launch_chain(KERNEL, dim3(blocks), dim3(s.threads), smem, stream, a, s.threads_per_row, ring);
}

// FN<S, A, NPT, MAXT, VEC>(...) for the types and the row length.
#define MOE_NORM_DISPATCH(FN, ...)                                                                           \
  [&]() -> cudaError_t {                                                                                     \
    const bool vec = a.vec;                                                                                  \
    auto by_shape = [&](auto st, auto bt) -> cudaError_t {                                                   \
      using S = decltype(st);                                                                                \
      using A = decltype(bt);                                                                                \
      if (s.npt == 8) return vec ? FN<S, A, 8, 512, true>(__VA_ARGS__) : FN<S, A, 8, 512, false>(__VA_ARGS__); \
      if (!vec) return FN<S, A, 16, 1024, false>(__VA_ARGS__);                                               \
      return s.max_threads == 512 ? FN<S, A, 16, 512, true>(__VA_ARGS__) : FN<S, A, 16, 1024, true>(__VA_ARGS__); \
    };                                                                                                       \
    if (stream_type == kBf16) return by_shape(bf16(), bf16());                                               \
    if (stream_type == kFp16) return by_shape(__half(), __half());                                           \
    if (block_type == kBf16) return by_shape(float(), bf16());                                               \
    if (block_type == kFp16) return by_shape(float(), __half());                                             \
    return by_shape(float(), float());                                                                       \
  }()

}  // namespace
}  // namespace moe
