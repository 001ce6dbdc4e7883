// C entry points of the MX 4-bit operators and of the norms at a block's
// borders (declared in include/moe.h): argument checks, the handle of a set
// of 4-bit expert weights, and the launches.
#include <algorithm>
#include <climits>
#include <initializer_list>
#include <new>

#include "../../include/moe.h"
#include "elem.cuh"
#include "gemm_common.cuh"
#include "host_common.cuh"
#include "kernels.cuh"
#include "mx4.cuh"
#include "norm.cuh"

using namespace moe;

static_assert(MOE_BF16 == kBf16 && MOE_FP16 == kFp16 && MOE_FP32 == kFp32, "moe_dtype and ElemType are the same codes");
static_assert(MOE_GATE_NONE == kGateNone && MOE_GATE_FEATURE == kGateFeature && MOE_GATE_TOKEN == kGateToken &&
                  MOE_GATE_FULL == kGateFull,
              "moe_gate_kind and GateKind are the same codes");

struct moe_mx4_handle {
  uint32_t magic;
  moe_mx4_config cfg;
  int device, num_sms;
  int m_tiles, m_stride, k_steps;
  int gated_boxes;
  unsigned long long wait_limit_ns;
  void* ws;               // one allocation: error word, part counts, parts, scale tiles
  uint32_t* err;
  int* ksplit_cnt;
  float* ksplit_part;
  uint8_t* scale_tiles;
  CUtensorMap map_w, map_s;
};

namespace {

constexpr uint32_t kMx4Magic = 0x4d583401u;
constexpr unsigned long long kDefaultWaitNs = 2000000000ull;
constexpr int kMaxTokenRows = 1 << 30;

bool valid_handle(const moe_mx4_handle* h) { return h != nullptr && h->magic == kMx4Magic; }

// Bytes of an element: what a row operator's pointers are aligned to at least
// (with 16-byte aligned rows it uses 16-byte accesses).
uintptr_t elem_bytes(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

bool valid_dtype(int t) { return t == MOE_BF16 || t == MOE_FP16 || t == MOE_FP32; }

bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 16)) return false;
  return true;
}

// Compute capability 10.3 and the SM count of a device.
int check_device(int dev, int* sms) {
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_NO_DEVICE;
  }
  return major == 10 && minor == 3 ? MOE_OK : MOE_ERR_NO_DEVICE;
}

// Codes of `rows` matrix rows in each of `groups` groups: boxes of 128 bytes x
// box_rows, 128-byte swizzle, zeros past a group's last row.
bool encode_codes(CUtensorMap* map, const void* base, uint64_t groups, uint64_t rows, uint64_t row_bytes,
                  uint32_t box_rows) {
  const int rank = groups > 0 ? 3 : 2;
  cuuint64_t dims[3] = {row_bytes, rows, groups};
  cuuint64_t strides[2] = {row_bytes, row_bytes * rows};
  cuuint32_t box[3] = {128, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return tensor_map_encode()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box,
                             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Gated weight codes where F is a multiple of 16: one box holds the 128 rows
// of a tile (4 blocks of 16 gate and the 16 up rows) and 128 bytes of each.
bool encode_gated(CUtensorMap* map, const void* base, uint64_t groups, uint64_t F, uint64_t row_bytes) {
  cuuint64_t dims[5] = {row_bytes, 16, 2, F / 16, groups};
  cuuint64_t strides[4] = {row_bytes, row_bytes * F, row_bytes * 16, row_bytes * 2 * F};
  cuuint32_t box[5] = {128, 16, 2, 4, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return tensor_map_encode()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(base), dims, strides, box, estr,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles: rows of 1 KB (one K step of one weight tile), a row to a box.
bool encode_scale_tiles(CUtensorMap* map, const void* base, uint64_t rows) {
  cuuint64_t dims[2] = {256, rows};
  cuuint64_t strides[1] = {2 * kMx4ScaleTile};
  cuuint32_t box[2] = {256, 1};
  cuuint32_t estr[2] = {1, 1};
  return tensor_map_encode()(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Work items of a call with tiles of `tile` rows, at most: a tile for a row of
// each group, and one more for every `tile` of the other rows, each times the
// weight tiles (pairs of CTAs: two at a time).
long long items_of(const moe_mx4_handle* h, int tile, long long rows) {
  const long long first = std::min<long long>(h->cfg.groups, rows);
  return (first + (rows - first) / tile) * (tile == kMx4PairTile ? h->m_stride / 2 : h->m_tiles);
}

// Token-tile width: the smallest that holds the mean rows of a group with some
// slack (the MMAs' N follows each tile's rows, so a wider tile costs ring depth
// only; flash shape's down product, 2048 tokens, 65 rows a group with the slack:
// 96 rows 170.8 us, 128 184.3, 64 180.4), but
//   - not below 64, the first that two groups of epilogue warps share, where a CTA
//     has many items of four K steps or more: gate/up, 128 tokens, 16 or 32 rows
//     235.1 us, 64 227.2; 512: 257.6 and 245.9; down, 256: 139.8 and 134.6. Few
//     items or short ones are the other way about: gate/up, 4 tokens, 34.8 and
//     37.1; 33 tokens to 5 of 74 experts, 3085 x 390: 24.0 and 28.0;
//   - narrower as long as the items of a narrower one still run all at once, one
//     to an SM (705 tokens to 4 of 15 experts, 48 x 567: 14.4 us without this,
//     9.6 so; 367 tokens to 1 of 3, 886 x 108: 11.6 and 7.5).
int choose_tile(const moe_mx4_handle* h, long long rows) {
  const double mean = 1.15 * static_cast<double>(rows) / h->cfg.groups;
  constexpr int kTwoGroupTile = 2;
  int i = 0;
  while (i + 1 < kMx4NumTileN && mean > kMx4TileN[i]) ++i;
  if (i < kTwoGroupTile && h->k_steps >= 4 && items_of(h, kMx4TileN[i], rows) > 8LL * h->num_sms) i = kTwoGroupTile;
  while (i > 0 && items_of(h, kMx4TileN[i - 1], rows) <= h->num_sms) --i;
  return kMx4TileN[i];
}

// Few items: the K steps of all items dealt out in equal contiguous ranges, one
// to a CTA, in place of whole items.  That saves what the last wave leaves idle,
// (SMs - its items) x K steps, and costs two to three microseconds for the parts
// (stored, counted and added up), and reads the token rows of an item in several
// places.  Measured over 8 to 64 steps and 22 to 1080 items (us, whole and balanced):
//   - two to four waves, the last at most half full and over 8 steps of every SM
//     idle: 16 steps, 160 items 14.0 and 12.9, 180: 17.0 and 16.0, 320: 20.2 and 18.5;
//     48 steps, 200: 34.8 and 29.6.  Not: 8 steps, 160: 9.2 and 10.6; 16 steps, 228: 15.0
//     and 15.7, 260: 15.4 and 16.4; five waves of 16 steps, 660: 35.4 and 36.7;
//   - one wave of at most a third of the SMs, which whole items leave the rest of
//     without work, from 24 steps on (an item has four parts at most): 24 items, 24
//     steps 10.3 and 9.6, 48: 16.2 and 11.8.  Not: 16 steps, 24 items 8.2 and 10.5; 24
//     steps, 88 items 11.0 and 12.7, 128: 12.3 and 15.0.
int choose_balanced(const moe_mx4_handle* h, int tile, long long rows) {
  if (tile > 32) return 0;
  const long long items = items_of(h, tile, rows), sms = h->num_sms;
  if (items <= sms) return 3 * items <= sms && h->k_steps >= 24;
  const long long last = items % sms;
  return items < 4 * sms && last > 0 && 2 * last <= sms && (sms - last) * h->k_steps > 8 * sms;
}

int check_norm_config(int T, int d, const moe_norm_config* c) {
  if (c == nullptr || T < 0 || d <= 0) return MOE_ERR_INVALID_ARG;
  if (!norm_types_ok(c->stream_dtype, c->block_dtype)) {
    return valid_dtype(c->stream_dtype) && valid_dtype(c->block_dtype) ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  }
  if (c->gate_kind < MOE_GATE_NONE || c->gate_kind > MOE_GATE_FULL || (c->sigmoid != 0 && c->sigmoid != 1))
    return MOE_ERR_INVALID_ARG;
  if (!(c->eps > 0.f) || !(c->eps < 1e30f) || !(c->alpha > -1e30f && c->alpha < 1e30f)) return MOE_ERR_INVALID_ARG;
  if (c->gate_kind != MOE_GATE_NONE && c->gate_dtype != c->block_dtype && c->gate_dtype != MOE_FP32)
    return valid_dtype(c->gate_dtype) ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  return d > kNormMaxCols ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Which of the operator's parts are there: a branch (y) or not, its norm, its gate, the norm after it.
int check_norm_parts(int terms, const moe_norm_config* c, const void* y, const void* w_post, const void* gate,
                     const void* w_pre) {
  if (y == nullptr && (w_post != nullptr || c->gate_kind != MOE_GATE_NONE || w_pre == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (y != nullptr && terms <= 0) return MOE_ERR_INVALID_ARG;
  if ((c->gate_kind != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
  return terms > kNormMaxTerms ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace

extern "C" {

int moe_mx4_quantize(const void* x, int dtype, long long n_src, int cols, const int* src, int src_div, long long rows,
                     void* codes, void* scales, void* values, void* stream) {
  if (!valid_dtype(dtype) || n_src < 0 || rows < 0 || cols <= 0 || src_div <= 0 || rows > kMaxTokenRows * 8ll ||
      cols > (1 << 24) || (src == nullptr && rows > 0 && rows != n_src))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if ((codes == nullptr) != (scales == nullptr) || (codes == nullptr && values == nullptr)) return MOE_ERR_INVALID_ARG;
  const uintptr_t elem = elem_bytes(dtype);
  CallBuffers b;
  if ((n_src > 0 && !b.need(x, elem)) || !b.maybe(codes) || !b.maybe(scales, 4) || !b.maybe(values, elem) ||
      !b.maybe(src, 4))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard device_guard(b.device());
  Mx4QuantizeArgs a{};
  a.x = x;
  a.src = src;
  a.n_src = n_src;
  a.src_div = src_div;
  a.rows = rows;
  a.cols = cols;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  a.values = values;
  a.vec = cols % 8 == 0 && aligned(x, 16) && aligned(values, 16);
  MOE_CUDA(launch_mx4_quantize(dtype, a, static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

int moe_mx4_gather(const void* codes, const void* scales, long long n_src, int cols, const int* src, int src_div,
                   long long rows, void* out_codes, void* out_scales, void* stream) {
  if (n_src < 0 || rows < 0 || cols <= 0 || src_div <= 0 || rows > kMaxTokenRows * 8ll || cols > (1 << 24))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  CallBuffers b;
  if ((n_src > 0 && (!b.need(codes) || !b.need(scales, 4))) || !b.need(src, 4) || !b.need(out_codes) ||
      !b.need(out_scales, 4))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard device_guard(b.device());
  Mx4GatherArgs a{};
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = static_cast<const uint8_t*>(scales);
  a.src = src;
  a.n_src = n_src;
  a.src_div = src_div;
  a.rows = rows;
  a.code_bytes = mx4_code_bytes(cols);
  a.scale_ld = mx4_scale_bytes(cols);
  a.out_codes = static_cast<uint8_t*>(out_codes);
  a.out_scales = static_cast<uint8_t*>(out_scales);
  MOE_CUDA(launch_mx4_gather(a, static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

int moe_mx4_init(const moe_mx4_config* cfg, const void* codes, const void* scales, moe_mx4_handle** out) {
  if (out == nullptr) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (cfg == nullptr || codes == nullptr || scales == nullptr || !aligned(codes, 16) || !aligned(scales, 4))
    return MOE_ERR_INVALID_ARG;
  const moe_mx4_config c = *cfg;
  if (c.groups <= 0 || c.rows <= 0 || c.cols <= 0 || (c.gated != 0 && c.gated != 1) || (c.gated && c.rows % 2 != 0))
    return MOE_ERR_INVALID_ARG;
  if (c.groups > gemm::kMaxGroups || c.rows > (1 << 20) || c.cols > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_NO_DEVICE;
  }
  int rc = check_device(dev, &sms);
  if (rc != MOE_OK) return rc;
  CallBuffers b(dev);
  if (!b.need(codes) || !b.need(scales, 4)) return MOE_ERR_INVALID_ARG;
  if (!load_encode() || mx4_gemm_prepare() != cudaSuccess) return MOE_ERR_CUDA;

  moe_mx4_handle* h = new (std::nothrow) moe_mx4_handle();
  if (h == nullptr) return MOE_ERR_CUDA;
  h->cfg = c;
  h->device = dev;
  h->num_sms = sms;
  h->wait_limit_ns = kDefaultWaitNs;
  h->m_tiles = c.gated ? (c.rows / 2 + 63) / 64 : (c.rows + 127) / 128;
  h->m_stride = h->m_tiles + (h->m_tiles & 1);
  h->k_steps = (c.cols + kMx4KStep - 1) / kMx4KStep;
  const size_t slots = 2 * static_cast<size_t>(sms);
  const size_t o_cnt = 256, o_part = o_cnt + (slots * 4 + 255) / 256 * 256,
               o_tiles = o_part + slots * kBlockM * 32 * 4,
               bytes = o_tiles + static_cast<size_t>(c.groups) * h->m_stride * h->k_steps * 2 * kMx4ScaleTile;
  if (cudaMalloc(&h->ws, bytes) != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return MOE_ERR_CUDA;
  }
  char* ws = static_cast<char*>(h->ws);
  h->err = reinterpret_cast<uint32_t*>(ws);
  h->ksplit_cnt = reinterpret_cast<int*>(ws + o_cnt);
  h->ksplit_part = reinterpret_cast<float*>(ws + o_part);
  h->scale_tiles = reinterpret_cast<uint8_t*>(ws + o_tiles);
  // the caller's weights may still be in flight on one of its streams
  bool ok = cudaDeviceSynchronize() == cudaSuccess;
  ok = ok && cudaMemset(h->ws, 0, o_part) == cudaSuccess;
  ok = ok && launch_mx4_tile_scales(static_cast<const uint8_t*>(scales), c.groups, c.rows, c.gated != 0, h->m_stride,
                                    h->k_steps, (c.cols + kMx4Block - 1) / kMx4Block, mx4_scale_bytes(c.cols),
                                    h->scale_tiles, nullptr) == cudaSuccess;
  // otherwise a tile's last block would run past the weights: boxes of 16 rows
  h->gated_boxes = c.gated && c.rows % 32 == 0 ? 1 : 8;
  ok = ok && (h->gated_boxes == 1
                  ? encode_gated(&h->map_w, codes, c.groups, c.rows / 2, mx4_code_bytes(c.cols))
                  : encode_codes(&h->map_w, codes, c.groups, c.rows, mx4_code_bytes(c.cols), c.gated ? 16 : 128));
  ok = ok && encode_scale_tiles(&h->map_s, h->scale_tiles, static_cast<uint64_t>(c.groups) * h->m_stride * h->k_steps);
  ok = ok && cudaDeviceSynchronize() == cudaSuccess;
  if (!ok) {
    cudaGetLastError();
    cudaFree(h->ws);
    delete h;
    return MOE_ERR_CUDA;
  }
  h->magic = kMx4Magic;
  *out = h;
  return MOE_OK;
}

int moe_mx4_matmul(moe_mx4_handle* h, const void* codes, const void* scales, long long rows, const int* offsets,
                   const int* out_rows, const float* row_scale, void* out, int out_dtype, long long n_out,
                   void* stream) {
  if (!valid_handle(h) || rows < 0 || n_out < 0 || !valid_dtype(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxTokenRows || n_out > kMaxTokenRows) return MOE_ERR_UNSUPPORTED;
  if (out_rows == nullptr && n_out != rows) return MOE_ERR_INVALID_ARG;
  if (rows == 0 || n_out == 0) return MOE_OK;
  DeviceGuard device_guard(h->device);
  CallBuffers b(h->device);
  if (!b.need(codes) || !b.need(scales, 4) || !b.need(offsets, 4) || !b.need(out, elem_bytes(out_dtype)) ||
      !b.maybe(out_rows, 4) || !b.maybe(row_scale, 4))
    return MOE_ERR_INVALID_ARG;
  const moe_mx4_config& c = h->cfg;
  const int tile = choose_tile(h, rows);
  if (items_of(h, tile, rows) > INT_MAX) return MOE_ERR_UNSUPPORTED;  // the kernel's item numbers
  CUtensorMap map_x;
  if (!encode_codes(&map_x, codes, 0, static_cast<uint64_t>(rows), mx4_code_bytes(c.cols), mx4_box_rows(tile)))
    return MOE_ERR_CUDA;
  Mx4GemmArgs a{};
  a.offsets = offsets;
  a.scales = static_cast<const uint8_t*>(scales);
  a.out_rows = out_rows;
  a.row_scale = row_scale;
  a.out = out;
  a.err = h->err;
  a.ksplit_part = h->ksplit_part;
  a.ksplit_cnt = h->ksplit_cnt;
  a.wait_limit_ns = h->wait_limit_ns;
  a.G = c.groups;
  a.rows = static_cast<int>(rows);
  a.n_out = static_cast<int>(n_out);
  a.out_cols = c.gated ? c.rows / 2 : c.rows;
  a.out_type = out_dtype;
  a.N = c.rows;
  a.m_tiles = h->m_tiles;
  a.m_stride = h->m_stride;
  a.blocks = (c.cols + kMx4Block - 1) / kMx4Block;
  a.k_steps = h->k_steps;
  a.scale_ld = mx4_scale_bytes(c.cols);
  a.scales_wide = a.scale_ld % 16 == 0 && aligned(scales, 16);
  a.out_wide = a.out_cols % (16 / static_cast<int>(elem_bytes(out_dtype))) == 0 && aligned(out, 16);
  a.gated_boxes = h->gated_boxes;
  a.balanced = choose_balanced(h, tile, rows);
  MOE_CUDA(launch_mx4_gemm(c.gated != 0, tile, &h->map_w, &h->map_s, &map_x, a, h->num_sms, static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

int moe_mx4_check(moe_mx4_handle* h, void* stream) {
  if (!valid_handle(h)) return MOE_ERR_INVALID_ARG;
  DeviceGuard device_guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
  uint32_t e = 0;
  MOE_CUDA(cudaMemcpyAsync(&e, h->err, sizeof e, cudaMemcpyDeviceToHost, s));
  MOE_CUDA(cudaMemsetAsync(h->err, 0, sizeof e, s));
  // a product that gave up may have left part counts behind
  MOE_CUDA(cudaMemsetAsync(h->ksplit_cnt, 0, sizeof(int) * 2 * static_cast<size_t>(h->num_sms), s));
  MOE_CUDA(cudaStreamSynchronize(s));
  return e ? MOE_ERR_DEVICE : MOE_OK;
}

int moe_mx4_set_wait_limit(moe_mx4_handle* h, unsigned long long ns) {
  if (!valid_handle(h)) return MOE_ERR_INVALID_ARG;
  h->wait_limit_ns = ns ? ns : kDefaultWaitNs;
  return MOE_OK;
}

int moe_mx4_free(moe_mx4_handle* h) {
  if (!valid_handle(h)) return MOE_ERR_INVALID_ARG;
  DeviceGuard device_guard(h->device);
  h->magic = 0;
  const bool ok = cudaDeviceSynchronize() == cudaSuccess;
  const bool freed = cudaFree(h->ws) == cudaSuccess;
  delete h;
  return ok && freed ? MOE_OK : MOE_ERR_CUDA;
}

int moe_norm_residual(const moe_norm_config* cfg, int T, int d, const void* x, const void* y, int terms,
                      const float* w_post, const void* gate, const float* w_pre, void* out, void* n, void* stream) {
  int rc = check_norm_config(T, d, cfg);
  if (rc != MOE_OK || T == 0) return rc;
  if ((rc = check_norm_parts(terms, cfg, y, w_post, gate, w_pre)) != MOE_OK) return rc;
  if ((y != nullptr) != (out != nullptr) || (w_pre != nullptr) != (n != nullptr)) return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const uintptr_t es = elem_bytes(cfg->stream_dtype), eb = elem_bytes(cfg->block_dtype),
                  eg = elem_bytes(cfg->gate_dtype);
  CallBuffers b;
  if (!b.need(x, es) || !b.maybe(y, eb) || !b.maybe(w_post, 4) || !b.maybe(gate, eg) || !b.maybe(w_pre, 4) ||
      !b.maybe(out, es) || !b.maybe(n, eb))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard device_guard(b.device());
  MOE_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, b.device()));
  NormArgs a{};
  a.vec = d % 8 == 0 && all_aligned({x, y, w_post, gate, w_pre, out, n});
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.out = out;
  a.n = n;
  a.alpha = cfg->alpha;
  a.eps = cfg->eps;
  a.T = T;
  a.d = d;
  a.terms = terms;
  a.gate_kind = cfg->gate_kind;
  a.gate_f32 = cfg->gate_dtype == MOE_FP32;
  a.sigmoid = cfg->sigmoid;
  MOE_CUDA(launch_norm(cfg->stream_dtype, cfg->block_dtype, a, sms, static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

long long moe_norm_residual_workspace(int T, int d) {
  if (T < 0 || d <= 0 || d > kNormMaxCols) return -1;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return static_cast<long long>(norm_bwd_parts(T, d, sms)) * 3 * d * 4;
}

int moe_norm_residual_backward(const moe_norm_config* cfg, int T, int d, const void* d_out, const void* d_n,
                               const void* out, const void* y, int terms, const float* w_post, const void* gate,
                               const float* w_pre, void* dx, void* dy, float* d_w_post, void* d_gate, float* d_w_pre,
                               void* workspace, long long workspace_bytes, void* stream) {
  int rc = check_norm_config(T, d, cfg);
  if (rc != MOE_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CallBuffers b;
  if (T == 0) {  // no rows: the sums over them are zero
    void* sums[] = {d_w_post, cfg->gate_kind == MOE_GATE_FEATURE ? d_gate : nullptr, d_w_pre};
    for (void* p : sums)
      if (!b.maybe(p, 4)) return MOE_ERR_INVALID_ARG;
    DeviceGuard device_guard(b.device());
    for (void* p : sums)
      if (p != nullptr) MOE_CUDA(cudaMemsetAsync(p, 0, sizeof(float) * static_cast<size_t>(d), s));
    return MOE_OK;
  }
  int sms = 0;
  if ((rc = check_norm_parts(terms, cfg, y, w_post, gate, w_pre)) != MOE_OK) return rc;
  const bool pre = w_pre != nullptr;
  if (dx == nullptr || (d_n != nullptr) != pre || (pre && out == nullptr) || (d_w_pre != nullptr) != pre ||
      (!pre && d_out == nullptr) || (y != nullptr) != (dy != nullptr) || (w_post != nullptr) != (d_w_post != nullptr) ||
      (gate != nullptr) != (d_gate != nullptr))
    return MOE_ERR_INVALID_ARG;
  const uintptr_t es = elem_bytes(cfg->stream_dtype), eb = elem_bytes(cfg->block_dtype),
                  eg = elem_bytes(cfg->gate_dtype);
  const uintptr_t edg = cfg->gate_kind == MOE_GATE_FULL ? eg : 4;
  if (!b.need(dx, es) || !b.maybe(d_out, es) || !b.maybe(d_n, eb) || !b.maybe(out, es) || !b.maybe(y, eb) ||
      !b.maybe(w_post, 4) || !b.maybe(gate, eg) || !b.maybe(w_pre, 4) || !b.maybe(dy, eb) || !b.maybe(d_w_post, 4) ||
      !b.maybe(d_gate, edg) || !b.maybe(d_w_pre, 4) || !b.need(workspace))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard device_guard(b.device());
  MOE_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, b.device()));
  const long long need = static_cast<long long>(norm_bwd_parts(T, d, sms)) * 3 * d * 4;
  if (workspace_bytes < need) return MOE_ERR_INVALID_ARG;
  NormBwdArgs a{};
  a.vec = d % 8 == 0 && all_aligned({d_out, d_n, out, y, w_post, gate, w_pre, dx, dy,
                                     cfg->gate_kind == MOE_GATE_FULL ? d_gate : nullptr});
  a.d_out = d_out;
  a.d_n = d_n;
  a.out = out;
  a.y = y;
  a.gate = gate;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.dx = dx;
  a.dy = dy;
  a.d_gate = d_gate;
  a.d_w_post = d_w_post;
  a.d_w_pre = d_w_pre;
  a.part = static_cast<float*>(workspace);
  a.alpha = cfg->alpha;
  a.eps = cfg->eps;
  a.T = T;
  a.d = d;
  a.terms = terms;
  a.gate_kind = cfg->gate_kind;
  a.gate_f32 = cfg->gate_dtype == MOE_FP32;
  a.sigmoid = cfg->sigmoid;
  MOE_CUDA(launch_norm_bwd(cfg->stream_dtype, cfg->block_dtype, a, sms, s));
  return MOE_OK;
}

}  // extern "C"
