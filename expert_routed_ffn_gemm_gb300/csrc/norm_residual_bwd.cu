// Gradients of the norms at a block's borders (the mathematics is in
// norm_residual.cu).
#include <type_traits>

#include "norm_rows.cuh"

namespace moe {
namespace {

__device__ __forceinline__ F2 pair(const float (&f)[8], int p) { return f2(f[2 * p], f[2 * p + 1]); }

template <typename S, typename A, int NPT, int MAXT, int PER_SM, bool VEC, bool PIPE, int GATE>
__global__ void __launch_bounds__(MAXT, PER_SM) norm_bwd_kernel(const NormBwdArgs a, int threads_per_row, Ring ring) {
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
             pre = GATE >= 0 || a.w_pre != nullptr, direct = GATE >= 0 || a.d_out != nullptr;
  const int gate_kind = GATE == kGateFull32 ? kGateFull : GATE >= 0 ? GATE : a.gate_kind;
  const bool full = gate_kind == kGateFull, feature = gate_kind == kGateFeature;
  // (with GATE a full gate has the block's type unless it says otherwise)
  const int gate_f32 = GATE == kGateFull32 || (GATE == kGateFull && sizeof(A) == 4) ? 1 : GATE == kGateFull ? 0 : a.gate_f32;
  // a row group's part of a stage: d_out, out, d_n, the terms, the gates
  char* const mine = s_rows + rg * ring.stage_bytes * ring.stages;
  const int wide = ring_cols(NPT, threads_per_row);
  const int row_s = wide * static_cast<int>(sizeof(S)), row_a = wide * static_cast<int>(sizeof(A));
  const int at_o = direct ? row_s : 0, at_h = at_o + (pre ? row_s : 0), at_y = at_h + (pre ? row_a : 0),
            at_g = at_y + a.terms * row_a;
  auto fetch = [&](long long t, int stage) {
    if constexpr (PIPE) {
      if (t < a.T) {
        char* st = mine + stage * ring.stage_bytes;
        if (direct) copy_row<S>(c, reinterpret_cast<S*>(st), static_cast<const S*>(a.d_out) + t * a.d);
        if (pre) {
          copy_row<S>(c, reinterpret_cast<S*>(st + at_o), static_cast<const S*>(a.out) + t * a.d);
          copy_row<A>(c, reinterpret_cast<A*>(st + at_h), static_cast<const A*>(a.d_n) + t * a.d);
        }
        if (branch)
          for (int m = 0; m < a.terms; ++m)
            copy_row<A>(c, reinterpret_cast<A*>(st + at_y) + m * wide,
                        static_cast<const A*>(a.y) + (t * a.terms + m) * a.d);
        if (full) {
          if (gate_f32)
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
  // A thread's elements in runs of 8.  One run: a row's inputs and the columns'
  // vectors stay in registers.  Two: they are read again once the sums are
  // there (from the ring, L1 or L2), and only the column sums stay.
  constexpr int RUNS = NPT / 8;
  constexpr bool AGAIN = RUNS > 1;
  using Run = Cols<8, VEC>;
  auto run_of = [&](int k) { return Run{c.tid + (VEC ? k : 8 * k) * threads_per_row, threads_per_row, a.d}; };
  float wp[8], wq[8], g_col[8];
  // two of the gates held folded (see fold_gate)
  auto gate_pair = [&](const float (&f)[8], int p) {
    return f2(unfold_gate(f[2 * p], a.sigmoid), unfold_gate(f[2 * p + 1], a.sigmoid));
  };
  auto load_columns = [&](const Run& r, auto full_exp) {
#pragma unroll
    for (int j = 0; j < 8; ++j) wp[j] = 0.f, wq[j] = 1.f;
    if (pre) load_row<float>(r, a.w_pre, wp);
    if (post) load_row<float>(r, a.w_post, wq);
    if (feature) {
      float g[8];
      load_folded<A, false, decltype(full_exp)::value>(r, a.gate, a.gate_f32, a.sigmoid, g_col, g);
    }
  };
  if (!AGAIN) load_columns(run_of(0), std::true_type());
  F2 acc_pre[NPT / 2], acc_post[NPT / 2], acc_gate[NPT / 2];
#pragma unroll
  for (int p = 0; p < NPT / 2; ++p) acc_pre[p] = acc_post[p] = acc_gate[p] = f2(0.f);
  const float inv_d = 1.0f / a.d;
  int stage = 0;
  for (long long t = t0; t < a.T; t += step) {
    const char* st = mine + stage * ring.stage_bytes;
    if constexpr (PIPE) {
      int ahead = stage + ring.stages - 1;
      if (ahead >= ring.stages) ahead -= ring.stages;
      fetch(t + (ring.stages - 1) * step, ahead);
      if (ring.stages == 2)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 2;" ::: "memory");
      if (++stage == ring.stages) stage = 0;
    }
    float D[8], o[8], h[8], z[8], g[8], g_plain[8];  // g: folded gates; plain ones live to the sums only
    auto load_run = [&](const Run& r, auto sums_only) {
#pragma unroll
      for (int j = 0; j < 8; ++j) D[j] = o[j] = h[j] = z[j] = 0.f, g[j] = g_plain[j] = 1.f;
      if (direct)
        load_row<S, PIPE>(r, PIPE ? reinterpret_cast<const S*>(st) : static_cast<const S*>(a.d_out) + t * a.d, D);
      if (pre) {
        load_row<S, PIPE>(r, PIPE ? reinterpret_cast<const S*>(st + at_o) : static_cast<const S*>(a.out) + t * a.d, o);
        load_row<A, PIPE>(r, PIPE ? reinterpret_cast<const A*>(st + at_h) : static_cast<const A*>(a.d_n) + t * a.d, h);
      }
      if (branch) {
        load_terms<A, PIPE>(r,
                            PIPE ? reinterpret_cast<const A*>(st + at_y) : static_cast<const A*>(a.y) + t * a.terms * a.d,
                            PIPE ? wide : a.d, a.terms, z);
        if (full) {
          const char* p = PIPE ? st + at_g : gate_row<A>(a, t);
          if (decltype(sums_only)::value)
            load_folded<A, PIPE, sizeof(A) == 4>(r, p, gate_f32, a.sigmoid, g, g_plain);
          else if (sizeof(A) == 4 || gate_f32)
            load_folded<float, PIPE, true>(r, p, 1, a.sigmoid, g, g_plain);
          else
            load_folded<A, PIPE, false>(r, p, 0, a.sigmoid, g, g_plain);
        } else if (feature) {
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = g_col[j], g_plain[j] = unfold_gate(g[j], a.sigmoid);
        }
      }
    };
    float g_row = 1.f, folded = 1.f;
    if (branch && gate_kind == kGateToken) g_row = gate_value<true>(raw_token_gate<A>(a, t), a.sigmoid, folded);
    // sums: h out, out^2, z^2, and a's products with d_out, h and out (a without
    // alpha and the token's gate; h times w_pre here), two columns at a time
    F2 s2[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) s2[i] = f2(0.f);
    F2 hw[4];
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      if (AGAIN) load_columns(run_of(k), std::bool_constant<sizeof(A) == 4>());  // the sums go into dy only
      load_run(run_of(k), std::bool_constant<AGAIN>());
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const F2 po = pair(o, p), pz = pair(z, p), pd = pair(D, p);
        const F2 az = mul2(mul2(VEC ? pair(g_plain, p) : gate_pair(g, p), pair(wq, p)), pz);
        hw[p] = mul2(pair(h, p), pair(wp, p));
        s2[0] = fma2(hw[p], po, s2[0]);
        s2[1] = fma2(po, po, s2[1]);
        s2[2] = fma2(pz, pz, s2[2]);
        s2[3] = fma2(az, pd, s2[3]);
        s2[4] = fma2(az, hw[p], s2[4]);
        s2[5] = fma2(az, po, s2[5]);
      }
    }
    float s[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] = sum2(s2[i]);
    sum.six(s);
    const float r = pre ? rsqrtf(s[1] * inv_d + a.eps) : 0.f;
    // D = d_out + r (h - out back); r^3 and q^2 in factors, since by themselves they
    // overflow for rows of almost nothing where eps is small
    const float back = r * (r * (inv_d * s[0]));
    const float q = post ? rsqrtf(s[2] * inv_d + a.eps) : 1.f;
    const float Q = a.alpha * (s[3] + r * (s[4] - back * s[5]));
    const float down = post ? q * (q * (inv_d * (g_row * Q))) : 0.f;
    const float alpha_row = a.alpha * g_row;
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const Run run = run_of(k);
      if (AGAIN) {
        load_columns(run, std::true_type());
        load_run(run, std::false_type());
      }
      F2 pD[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const F2 po = pair(o, p), ph = pair(h, p);
        if (AGAIN) hw[p] = mul2(ph, pair(wp, p));
        acc_pre[4 * k + p] = fma2(ph, mul2(po, f2(r)), acc_pre[4 * k + p]);
        pD[p] = fma2(fma2(po, f2(-back), hw[p]), f2(r), pair(D, p));
        split(pD[p], D[2 * p], D[2 * p + 1]);
      }
      store_row<S>(run, static_cast<S*>(a.dx) + t * a.d, D);
      if (!branch) continue;
      float dy[8];
      F2 wv[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const F2 v = mul2(pair(z, p), f2(q));
        pD[p] = mul2(pD[p], f2(alpha_row));  // from here on times alpha and the token's gate
        const F2 gD = mul2(gate_pair(g, p), pD[p]);
        acc_post[4 * k + p] = fma2(gD, v, acc_post[4 * k + p]);
        split(fma2(v, f2(-down), mul2(mul2(pair(wq, p), f2(q)), gD)), dy[2 * p], dy[2 * p + 1]);
        wv[p] = mul2(pair(wq, p), v);
      }
      store_row<A>(run, static_cast<A*>(a.dy) + t * a.d, dy);
      if (full || feature) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          F2 dg = mul2(wv[p], pD[p]);
          if (a.sigmoid) dg = mul2(dg, f2(fold_slope(g[2 * p]), fold_slope(g[2 * p + 1])));
          if (feature) acc_gate[4 * k + p] = fma2(dg, f2(1.f), acc_gate[4 * k + p]);
          split(dg, dy[2 * p], dy[2 * p + 1]);
        }
        if (full && gate_f32)
          store_row<float>(run, static_cast<float*>(a.d_gate) + t * a.d, dy);
        else if (full)
          store_row<A>(run, static_cast<A*>(a.d_gate) + t * a.d, dy);
      }
    }
    if (branch && gate_kind == kGateToken && c.tid == 0)
      static_cast<float*>(a.d_gate)[t] = q * Q * (a.sigmoid ? fold_slope(folded) : 1.f);
  }
  // this row group's column sums
  float* part = a.part + static_cast<size_t>(blockIdx.x * rows_per_block + rg) * 3 * a.d;
  auto store_sums = [&](float* to, const F2 (&sums)[NPT / 2]) {
    float f[NPT];
#pragma unroll
    for (int p = 0; p < NPT / 2; ++p) split(sums[p], f[2 * p], f[2 * p + 1]);
    store_row<float>(c, to, f);
  };
  if (pre) store_sums(part, acc_pre);
  if (branch && post) store_sums(part + a.d, acc_post);
  if (branch && feature) store_sums(part + 2 * static_cast<size_t>(a.d), acc_gate);
}

// Column sums over the parts: a block takes 32 columns, warp w the parts w,
// w + 32, ... (few enough that a warp's loads are in flight together), and the
// warps' sums are added in warp order.
constexpr int kColThreads = 1024;
__global__ void __launch_bounds__(kColThreads)
    norm_cols_kernel(const float* __restrict__ part, int parts, int d, float* d_w_pre, float* d_w_post, float* d_gate) {
  __shared__ float s[kColThreads / 32][32];
  pdl_trigger();
  float* out = blockIdx.y == 0 ? d_w_pre : (blockIdx.y == 1 ? d_w_post : d_gate);
  pdl_wait();
  if (out == nullptr) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (col < d) {
    const float* p = part + static_cast<size_t>(blockIdx.y) * d + col;
#pragma unroll 8
    for (int i = warp; i < parts; i += kColThreads / 32) sum += p[static_cast<size_t>(i) * 3 * d];
  }
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && col < d) {
#pragma unroll
    for (int w = 1; w < kColThreads / 32; ++w) sum += s[w][lane];
    out[col] = sum;
  }
}

int bwd_blocks(int T, const Shape& s, int sms) {
  return std::max(1, std::min((T + s.rows_per_block - 1) / s.rows_per_block,
                              sms * blocks_per_sm(s, kBwdThreadsPerSm)));
}

template <typename S, typename A>
cudaError_t launch_bwd_ring(const NormBwdArgs& a, const Shape& s, int blocks, const Ring& ring, cudaStream_t stream) {
  if (a.y != nullptr && a.w_post != nullptr && a.w_pre != nullptr && a.d_out != nullptr) {
    switch (a.gate_kind) {
      case kGateNone:
        return launch_ring<norm_bwd_kernel<S, A, 8, 512, 1, true, true, kGateNone>>(blocks, s, ring, a, stream);
      case kGateFeature:
        return launch_ring<norm_bwd_kernel<S, A, 8, 512, 1, true, true, kGateFeature>>(blocks, s, ring, a, stream);
      case kGateToken:
        return launch_ring<norm_bwd_kernel<S, A, 8, 512, 1, true, true, kGateToken>>(blocks, s, ring, a, stream);
      default:
        if constexpr (sizeof(A) == 2)
          if (a.gate_f32)
            return launch_ring<norm_bwd_kernel<S, A, 8, 512, 1, true, true, kGateFull32>>(blocks, s, ring, a, stream);
        return launch_ring<norm_bwd_kernel<S, A, 8, 512, 1, true, true, kGateFull>>(blocks, s, ring, a, stream);
    }
  }
  return launch_ring<norm_bwd_kernel<S, A, 8, 512, 1, true, true, -1>>(blocks, s, ring, a, stream);
}

// Column sums: which shape a call runs in.
struct BwdPlan {
  Shape shape;
  Ring ring;
  int blocks;
};
BwdPlan bwd_plan(int T, int d, bool vec, long long row_bytes, int sms) {
  BwdPlan p;
  p.shape = shape_of(d);
  p.blocks = bwd_blocks(T, p.shape, sms);
  p.ring = d <= 4096 && vec ? ring_of(row_bytes, p.shape, blocks_per_sm(p.shape, kBwdThreadsPerSm))
                                   : Ring{0, 0};
  if (p.ring.stages < 2) p.ring = Ring{0, 0};
  return p;
}

template <typename S, typename A, int NPT, int MAXT, bool VEC>
cudaError_t launch_bwd(const NormBwdArgs& a, const Shape& s, int sms, int* parts, cudaStream_t stream) {
  const long long row = static_cast<long long>(ring_cols(shape_of(a.d).npt, shape_of(a.d).threads_per_row)) *
                        ((a.d_out != nullptr ? sizeof(S) : 0) + (a.w_pre != nullptr ? sizeof(S) + sizeof(A) : 0) +
                         (a.y != nullptr ? a.terms : 0) * sizeof(A) +
                         (a.gate_kind == kGateFull ? (a.gate_f32 ? 4 : sizeof(A)) : 0));
  const BwdPlan p = bwd_plan(a.T, a.d, a.vec, row, sms);
  *parts = p.blocks * p.shape.rows_per_block;
  if constexpr (VEC && NPT == 8) {
    if (p.ring.stages > 0) return launch_bwd_ring<S, A>(a, p.shape, p.blocks, p.ring, stream);
  }
  return launch_chain(norm_bwd_kernel<S, A, NPT, MAXT, 1, VEC, false, -1>, dim3(p.blocks), dim3(s.threads), 0, stream,
                      a, s.threads_per_row, Ring{0, 0});
}

}  // namespace

int norm_bwd_parts(int T, int d, int sms) {
  const Shape s = shape_of(d);
  return bwd_blocks(T, s, sms) * s.rows_per_block;
}

cudaError_t launch_norm_bwd(int stream_type, int block_type, const NormBwdArgs& a, int sms, cudaStream_t stream) {
  const Shape s = shape_of(a.d);
  int parts = 0;
  const cudaError_t e = MOE_NORM_DISPATCH(launch_bwd, a, s, sms, &parts, stream);
  if (e != cudaSuccess) return e;
  float* gate = a.y != nullptr && a.gate_kind == kGateFeature ? static_cast<float*>(a.d_gate) : nullptr;
  float* post = a.y != nullptr && a.w_post != nullptr ? a.d_w_post : nullptr;
  float* pre = a.w_pre != nullptr ? a.d_w_pre : nullptr;
  if (pre == nullptr && post == nullptr && gate == nullptr) return cudaSuccess;
  return launch_chain(norm_cols_kernel, dim3((a.d + 31) / 32, 3), dim3(kColThreads), 0, stream,
                      static_cast<const float*>(a.part), parts, a.d, pre, post, gate);
}

}  // namespace moe
