// The norms at a block's borders, fused with the block's gate, the residual
// scale and the residual add:
//   z = sum_j y[t][j],  v = w_post * z * rsqrt(mean z^2 + eps)   (or v = z)
//   out = x + alpha * g * v,   g = gate or sigmoid(gate), or 1
//   n   = w_pre * out * rsqrt(mean out^2 + eps)
// and the gradients of out and n with respect to x, the terms, the gate and
// the two weights.
//
// Bound by memory: every row is read once and written once.  Up to 8192 columns
// that are vector-aligned a row lives in the registers of the threads that share
// it between the loads and the stores (8 elements each, beyond 2048 columns 16;
// 8192 rows of 4096 columns: 51 us, 0.96 of the copy rate).  Longer rows, and from
// 4097 columns on rows that are not aligned, go 16 elements to each of up to 1024
// threads of 64 registers and spill 260 to 1260 bytes a thread (2048 rows of 16384
// columns 161 us, 4096 unaligned ones of 5121: 240 us).  All sums and roundings but
// the last are fp32.  With more rows than fit the GPU at once the blocks stay and
// take row after row: each thread copies its own columns of the rows to come
// into shared memory asynchronously (no barrier: it alone reads them), so that
// loads stay in flight while a row's sums are formed.
//
// Backward, with r = rsqrt(mean out^2 + eps), q = rsqrt(mean z^2 + eps) worked
// out again from the stored out and the terms, h = d_n * w_pre:
//   D  = d_out + r h - out r^3/d S0,       S0 = sum h out        (= dx)
//   dz = q c - z q^3/d Q,  c = alpha g w_post D,  Q = sum c z
// Q needs D, but it is linear in it: with a = alpha g w_post z,
//   Q = sum a d_out + r sum a h - r^3/d S0 sum a out,
// so all six sums of a row come from one pass and one block-wide reduction.
// Column sums (the weights' gradients, a gate per feature) stay in registers
// over the rows of a persistent block; a second kernel adds the blocks' sums
// in a fixed order, so results do not change from run to run.  Up to 4096
// columns a row's inputs stay in registers too (8192 rows: 102 us, bound by issue,
// 602 instructions a warp and row).  Beyond, every row is read twice, from L2 the
// second time, without the ring, and the threads spill: 108 to 156 bytes up to 8192
// columns (4096 rows of 5120: 228 us, of 8192: 240), 1.3 KB beyond (2048 rows of
// 16384: 383), 4 KB and more where rows are not aligned (4096 of 5121: 1330).
#include "norm_rows.cuh"

namespace moe {
namespace {

// NPT elements to a thread, at most MAXT threads, PER_SM blocks to an SM.  VEC:
// 16-byte accesses.  PIPE: rows come through the ring.  GATE >= 0: compiled for
// that kind of gate with both norms and all gradients there; -1: any parts
// (the checks cost a third of the instructions of a row).
template <typename S, typename A, int NPT, int MAXT, int PER_SM, bool VEC, bool PIPE, int GATE>
__global__ void __launch_bounds__(MAXT, PER_SM) norm_kernel(const NormArgs a, int threads_per_row, Ring ring) {
  __shared__ __align__(16) float s_red[2 * (MAXT / 32) * 8];
  extern __shared__ __align__(16) char s_rows[];
  pdl_trigger();
  const int rows_per_block = blockDim.x / threads_per_row;
  const int rg = threads_per_row <= 32 ? threadIdx.x / 32 : 0;
  const Cols<NPT, VEC> c{static_cast<int>(threadIdx.x) - rg * threads_per_row, threads_per_row, a.d};
  RowSum<MAXT / 32> sum(s_red, threads_per_row);
  const long long step = static_cast<long long>(gridDim.x) * rows_per_block;
  const long long t0 = static_cast<long long>(blockIdx.x) * rows_per_block + rg;
  const bool branch = GATE >= 0 || a.y != nullptr, post = GATE >= 0 || a.w_post != nullptr,
             pre = GATE >= 0 || a.w_pre != nullptr;
  const int gate_kind = GATE >= 0 ? GATE : a.gate_kind;
  const bool full = gate_kind == kGateFull;
  const float inv_d = 1.0f / a.d;
  constexpr bool WIDE_OUT = sizeof(S) == 4;
  // a row group's part of a stage: x, the terms, the gates
  char* const mine = s_rows + rg * ring.stage_bytes * ring.stages;
  const int wide = ring_cols(NPT, threads_per_row);
  const int at_y = wide * static_cast<int>(sizeof(S)), at_g = at_y + a.terms * wide * static_cast<int>(sizeof(A));
  auto fetch = [&](long long t, int stage) {
    if constexpr (PIPE) {
      if (t < a.T) {
        char* st = mine + stage * ring.stage_bytes;
        copy_row<S>(c, reinterpret_cast<S*>(st), static_cast<const S*>(a.x) + t * a.d);
        if (branch)
          for (int m = 0; m < a.terms; ++m)
            copy_row<A>(c, reinterpret_cast<A*>(st + at_y) + m * wide,
                        static_cast<const A*>(a.y) + (t * a.terms + m) * a.d);
        if (full) {
          if (a.gate_f32)
            copy_row<float>(c, reinterpret_cast<float*>(st + at_g), static_cast<const float*>(a.gate) + t * a.d);
          else
            copy_row<A>(c, reinterpret_cast<A*>(st + at_g), static_cast<const A*>(a.gate) + t * a.d);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  pdl_wait();
  if constexpr (PIPE)
    for (int s = 0; s + 1 < ring.stages; ++s) fetch(t0 + s * step, s);
  // with 8 elements to a thread the columns' vectors stay in registers
  constexpr bool KEEP = PIPE || NPT == 8;
  float w_post[NPT], w_pre[NPT], g_col[NPT];
  auto load_columns = [&]() {
    if (post) load_row<float>(c, a.w_post, w_post);
    if (pre) load_row<float>(c, a.w_pre, w_pre);
    if (gate_kind == kGateFeature) load_gates<A, false, WIDE_OUT>(c, a.gate, a.gate_f32, a.sigmoid, g_col);
  };
  if (KEEP) load_columns();
  int stage = 0;
  // a block's warps leave the loop together when a row spans the block
  for (long long t = t0; t < a.T; t += step) {
    if (!KEEP) load_columns();
    const char* st = mine + stage * ring.stage_bytes;
    if constexpr (PIPE) {
      int ahead = stage + ring.stages - 1;
      if (ahead >= ring.stages) ahead -= ring.stages;
      fetch(t + (ring.stages - 1) * step, ahead);
      // every group but those of the rows to come has landed (a ring has two or three stages)
      if (ring.stages == 2)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 2;" ::: "memory");
      if (++stage == ring.stages) stage = 0;
    }
    float o[NPT];
    load_row<S, PIPE>(c, PIPE ? reinterpret_cast<const S*>(st) : static_cast<const S*>(a.x) + t * a.d, o);
    if (branch) {
      float z[NPT];
      load_terms<A, PIPE>(c, PIPE ? reinterpret_cast<const A*>(st + at_y) : static_cast<const A*>(a.y) + t * a.terms * a.d,
                          PIPE ? wide : a.d, a.terms, z);
      float k = a.alpha;
      float h;
      if (gate_kind == kGateToken) k *= gate_value<WIDE_OUT>(raw_token_gate<A>(a, t), a.sigmoid, h);
      if (post) {
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < NPT; ++j) q += z[j] * z[j];
        k *= rsqrtf(sum.one(q) * inv_d + a.eps);
#pragma unroll
        for (int j = 0; j < NPT; ++j) z[j] *= w_post[j];
      }
      if (full) {
        float g[NPT];
        load_gates<A, PIPE, WIDE_OUT>(c, PIPE ? st + at_g : gate_row<A>(a, t), a.gate_f32, a.sigmoid, g);
#pragma unroll
        for (int j = 0; j < NPT; ++j) z[j] *= g[j];
      } else if (gate_kind == kGateFeature) {
#pragma unroll
        for (int j = 0; j < NPT; ++j) z[j] *= g_col[j];
      }
#pragma unroll
      for (int j = 0; j < NPT; ++j) o[j] += k * z[j];
      store_row<S>(c, static_cast<S*>(a.out) + t * a.d, o);
    }
    if (pre) {
      float q = 0.f;
#pragma unroll
      for (int j = 0; j < NPT; ++j) q += o[j] * o[j];
      const float r = rsqrtf(sum.one(q) * inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < NPT; ++j) o[j] *= r * w_pre[j];
      store_row<A>(c, static_cast<A*>(a.n) + t * a.d, o);
    }
  }
}

// Forward through the ring.
template <typename S, typename A, int NPT>
cudaError_t launch_fwd_ring(const NormArgs& a, const Shape& s, int blocks, const Ring& ring, cudaStream_t stream) {
  if (a.y != nullptr && a.w_post != nullptr && a.w_pre != nullptr) {
    switch (a.gate_kind) {
      case kGateNone:
        return launch_ring<norm_kernel<S, A, NPT, 512, 16 / NPT, true, true, kGateNone>>(blocks, s, ring, a, stream);
      case kGateFeature:
        return launch_ring<norm_kernel<S, A, NPT, 512, 16 / NPT, true, true, kGateFeature>>(blocks, s, ring, a, stream);
      case kGateToken:
        return launch_ring<norm_kernel<S, A, NPT, 512, 16 / NPT, true, true, kGateToken>>(blocks, s, ring, a, stream);
      default:
        return launch_ring<norm_kernel<S, A, NPT, 512, 16 / NPT, true, true, kGateFull>>(blocks, s, ring, a, stream);
    }
  }
  return launch_ring<norm_kernel<S, A, NPT, 512, 16 / NPT, true, true, -1>>(blocks, s, ring, a, stream);
}

// Forward: rows through the ring where they outnumber the blocks that fit at
// once and are vector-aligned.
template <typename S, typename A, int NPT, int MAXT, bool VEC>
cudaError_t launch_fwd(const NormArgs& a, const Shape& s, int sms, cudaStream_t stream) {
  const int all = (a.T + s.rows_per_block - 1) / s.rows_per_block;
  if constexpr (VEC && MAXT == 512) {
    const Shape p = pipe_shape_of(a.d);
    const int per_sm = blocks_per_sm(p, kFwdThreadsPerSm * 8 / p.npt);
    const long long row = static_cast<long long>(ring_cols(p.npt, p.threads_per_row)) *
                          (sizeof(S) + (a.y != nullptr ? a.terms : 0) * sizeof(A) +
                           (a.gate_kind == kGateFull ? (a.gate_f32 ? 4 : sizeof(A)) : 0));
    const Ring ring = ring_of(row, p, per_sm);
    const int blocks = sms * per_sm;
    if ((a.T + p.rows_per_block - 1) / p.rows_per_block > blocks && ring.stages >= 2)
      return p.npt == 8 ? launch_fwd_ring<S, A, 8>(a, p, blocks, ring, stream)
                        : launch_fwd_ring<S, A, 16>(a, p, blocks, ring, stream);
    // few rows, in the same shape: a token's results have the same bits in a batch of any size
    if (p.npt == 16 && NPT == 8)
      return launch_chain(norm_kernel<S, A, 16, 512, 1, true, false, -1>,
                          dim3((a.T + p.rows_per_block - 1) / p.rows_per_block), dim3(p.threads), 0, stream, a,
                          p.threads_per_row, Ring{0, 0});
  }
  return launch_chain(norm_kernel<S, A, NPT, MAXT, 1, VEC, false, -1>, dim3(all), dim3(s.threads), 0, stream, a,
                      s.threads_per_row, Ring{0, 0});
}

}  // namespace

bool norm_types_ok(int stream_type, int block_type) {
  if (stream_type < kBf16 || stream_type > kFp32 || block_type < kBf16 || block_type > kFp32) return false;
  return stream_type == block_type || stream_type == kFp32;
}

cudaError_t launch_norm(int stream_type, int block_type, const NormArgs& a, int sms, cudaStream_t stream) {
  const Shape s = shape_of(a.d);
  return MOE_NORM_DISPATCH(launch_fwd, a, s, sms, stream);
}

}  // namespace moe
