// gemm_tc.cu -- host side of the base GEMM on the tensor cores (the kernel: gemm_tc.cuh): tensor
// maps, tile plans and launches.
#include "gemm_tc.cuh"

namespace lora {

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

cudaError_t encode_tmap_bf16(CUtensorMap* map, const void* base, int rows, int K, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBK), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_tmap_delta(CUtensorMap* map, const float* base, int rows, int N) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  if (N % 4 != 0 || rows < 1) return cudaErrorInvalidValue;  // rows start on 16-byte boundaries
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * 4};
  const cuuint32_t box[2] = {32, static_cast<cuuint32_t>(kBM)};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_tmap_u8(CUtensorMap* map, const void* base, int rows, int K, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  if (K % 16 != 0) return cudaErrorInvalidValue;  // rows start on 16-byte boundaries
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(2 * kBK), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// CTAs of this GEMM that can be resident at once in clusters of `csize` CTAs (every variant
// holds one CTA per SM; a cluster must fit in one GPC, whose sizes differ).  Queried once
// per device.
int gemm_tc_resident_ctas(int csize, int num_sms) {
  static int cache_all[kAttrDevices][9] = {};
  static int scratch[9] = {};
  if (csize < 1 || csize > 8) return 0;
  const int dev = attr_device();
  int* cache = dev >= 0 ? cache_all[dev] : scratch;
  {
    std::lock_guard<std::mutex> lock(attr_mutex());
    if (cache[csize] != 0) return cache[csize];
  }
  {
    const int smem = 200 * 1024;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = csize;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(csize * 64);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0, v = 0;
    if (raise_smem_limit<256, false, true>(smem) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, gemm_tc_kernel<256, false, true>, &cfg) ==
            cudaSuccess &&
        n > 0) {
      v = std::min(num_sms, n * csize);
    } else {
      cudaGetLastError();
      v = csize == 1 ? num_sms : 8 * (num_sms / 8 / csize) * csize;
    }
    std::lock_guard<std::mutex> lock(attr_mutex());
    cache[csize] = v;
    return v;
  }
}

// Tile shape, K split and CTA pairs, by least estimated time (cycles).  Measured on this
// kernel: a 64-wide K block costs its 4 MMA instructions (~124 cycles each below N = 256,
// 128 at N = 256) plus ~50 cycles of barrier hand-off, or its operand delivery at ~75 B
// per cycle per SM when that is slower (a 128 x 256 tile's 48 KB per block; a CTA pair
// halves the W rows each CTA loads, which made 256 x 256 pair tiles ~15% faster per block
// than 128 x 256 single-CTA tiles).  Each wave adds ~3k cycles of prologue, pipeline fill
// and epilogue; a split K adds the exchange of fp32 partials through L2 (written and read
// at ~50 B per cycle per SM).  Large problems (no split allowed) weigh the same costs
// without the split; their expand blocks (one per distinct slot of a tile) are not in
// the estimate, but a pair runs the expand blocks of all its 256 rows on both CTAs, which
// doubles them where slots change every few rows: pairs are taken there only when the
// batch averages at least 128 rows per slot (`slots` = the layer's slot count, 0 = none).
// With the e4m3 base in v mode single CTAs at N = 256 measured faster than pairs on every
// shape tried but one (8-18% at K = 4096; pairs 4% ahead at K = 14336, N = 4096), so the
// caller turns pairs off there.
GemmPlan gemm_tc_plan(int M, int N, int K, int num_sms, bool allow_split, int slots,
                      bool allow_pair) {
  const int mt = (M + kBM - 1) / kBM;
  const int nkb = (K + kBK - 1) / kBK;
  // every one of the cs K ranges of ceil(nkb / cs) blocks must be non-empty
  auto ranges_ok = [nkb](int c) { return (c - 1) * ((nkb + c - 1) / c) < nkb; };
  GemmPlan p{64, 1, 0};
  double best = 1e30;
  const int cand[3] = {256, 128, 64};
  // single CTAs first: a pair is taken only where it is estimated faster
  for (int pair = 0; pair <= 1; ++pair) {
    if (pair && (mt < 2 || !allow_pair)) continue;  // (one row tile: a pair leaves a CTA idle)
    if (pair && !allow_split && slots > 0 && (long long)M < 128LL * slots) continue;
    for (int i = 0; i < 3; ++i) {
      const int bn = cand[i];
      if (pair && bn < 128) continue;
      const double bytes = kABytes + (double)(pair ? bn / 2 : bn) * kBK * 2;
      const double per_kb = std::max(bytes / 75.0, 4.0 * std::max(124.0, 0.5 * bn)) + 50.0;
      const int ctas_m = pair ? 2 * ((mt + 1) / 2) : mt;
      const int tiles = ctas_m * ((N + bn - 1) / bn);
      // each CTA finishes bn / cs >= 32 columns (its epilogue and the split-K exchange work
      // in 32-column chunks)
      for (int cs = 1; cs <= (allow_split ? 4 : 1) && bn / cs >= 32; cs *= 2) {
        if (cs > 1 && !ranges_ok(cs)) break;
        const int conc = gemm_tc_resident_ctas((pair ? 2 : 1) * cs, num_sms);
        if (conc < 1) continue;
        const int waves = (tiles * cs + conc - 1) / conc;
        const int kb = (nkb + cs - 1) / cs;
        const double exch = cs > 1 ? 2.0 * (cs - 1) * kBM * (bn / cs) * 4.0 / 50.0 : 0.0;
        const double cost = waves * (kb * per_kb + 3000.0 + exch);
        if (cost < best * 0.999) {
          best = cost;
          p.block_n = bn;
          p.ksplit = cs;
          p.pair = pair;
        }
      }
    }
  }
  return p;
}

// Split-K scratch of a plan: per output block (one per CTA of a K range) cs x cs blocks of
// 128 rows x BN / cs columns.
size_t gemm_tc_plan_exchange_floats(const GemmPlan& p, int M, int N) {
  if (p.ksplit <= 1) return 0;
  const int mt = (M + kBM - 1) / kBM;
  const size_t gx = p.pair ? 2 * ((mt + 1) / 2) : mt;
  const size_t gy = (N + p.block_n - 1) / p.block_n;
  return gx * gy * p.ksplit * p.block_n * kBM;
}

// A delta-mode batch whose no-split plan leaves a last round of tiles at most half full
// runs as two launches: the column tiles of the whole rounds without a K split, then the
// remaining column tiles with a 2-way K split (their 2 x csize-CTA clusters fit in one
// round), so the last round takes half the time.  Returns the column tiles of the first
// launch, or 0 for no split.
static int delta_split_tiles(const GemmPlan& p, int M, int N, int nkb, int num_sms) {
  if (p.ksplit != 1 || nkb < 2) return 0;
  const int csize = p.pair ? 2 : 1;
  const int mt = (M + kBM - 1) / kBM, mtp = p.pair ? (mt + 1) / 2 : mt;
  const int nt = (N + p.block_n - 1) / p.block_n, units = mtp * nt;
  const int G = gemm_tc_resident_ctas(csize, num_sms) / csize;
  if (G < 1 || units <= G || units % G == 0 || 2 * (units % G) > G) return 0;
  const int ntA = (units / G) * G / mtp, ntB = nt - ntA;
  if (ntA < 1 || ntB < 1 || 2 * csize * mtp * ntB > gemm_tc_resident_ctas(2 * csize, num_sms)) return 0;
  if (p.block_n / 2 < 32) return 0;
  return ntA;
}

size_t gemm_tc_exchange_floats(int M, int N, int K, int num_sms) {
  const GemmPlan p = gemm_tc_plan(M, N, K, num_sms, true, 0);
  const int ntA = delta_split_tiles(p, M, N, (K + kBK - 1) / kBK, num_sms);
  if (ntA > 0)  // the second launch: the remaining columns with a 2-way split
    return gemm_tc_plan_exchange_floats(GemmPlan{p.block_n, 2, p.pair}, M, N - ntA * p.block_n);
  return gemm_tc_plan_exchange_floats(p, M, N);
}

int gemm_tc_tile_index(int BN) { return BN == 256 ? 0 : (BN == 128 ? 1 : 2); }

static cudaError_t launch_one(const GemmArgs& a, const GemmPlan& plan,
                              const CUtensorMap* tmap_w3, const CUtensorMap* tmap_bx3,
                              cudaStream_t stream);

cudaError_t launch_gemm_tc(const GemmArgs& a, const CUtensorMap* tmap_w3,
                           const CUtensorMap* tmap_bx3, cudaStream_t stream, int* launches) {
  if (a.ex.mode == kExpandV && !tmap_bx3) return cudaErrorInvalidValue;
  if (a.fp8 && (!a.tmap_xq || !a.sx || !a.sw || a.K % 16 != 0)) return cudaErrorInvalidValue;
  // the plan counts K blocks of 128 bytes: an e4m3 row of K elements is K / 2 bf16 wide
  const int k_bytes2 = a.fp8 ? (a.K + 1) / 2 : a.K;
  GemmPlan plan = gemm_tc_plan(a.M, a.N, k_bytes2, a.num_sms, a.ex.mode != kExpandV,
                               a.ex.mode == kExpandV ? a.ex.S : 0,
                               !(a.fp8 && a.ex.mode == kExpandV));
  if (a.force_bn != 0) {
    // v mode never splits K: its expand blocks run after the base ones in one accumulator
    plan = GemmPlan{a.force_bn, a.ex.mode == kExpandV ? 1 : a.force_cs, a.force_pair};
    const int nkb = (k_bytes2 + kBK - 1) / kBK, c = plan.ksplit;
    if (c > 1 && (c - 1) * ((nkb + c - 1) / c) >= nkb) return cudaErrorInvalidConfiguration;
  }
  GemmArgs whole = a;
  whole.n_begin = 0;
  whole.n_end = a.N;
  whole.trigger_next = false;
  whole.q_reset = true;  // the last launch of the batch resets the e4m3 row count
  // a last round at most half full: two launches (see delta_split_tiles)
  const int ntA = a.ex.mode == kExpandDelta && a.force_bn == 0
                      ? delta_split_tiles(plan, a.M, a.N, (k_bytes2 + kBK - 1) / kBK, a.num_sms)
                      : 0;
  if (ntA > 0) {
    GemmArgs first = whole, second = whole;
    first.n_end = ntA * plan.block_n;
    first.trigger_next = true;
    first.q_reset = false;
    second.n_begin = first.n_end;
    const GemmPlan plan2{plan.block_n, 2, plan.pair};
    cudaError_t e = launch_one(first, plan, tmap_w3, tmap_bx3, stream);
    if (e != cudaSuccess) return e;
    if (launches) ++*launches;
    e = launch_one(second, plan2, tmap_w3, tmap_bx3, stream);
    if (e == cudaSuccess && launches) ++*launches;
    return e;
  }
  const cudaError_t e = launch_one(whole, plan, tmap_w3, tmap_bx3, stream);
  if (e == cudaSuccess && launches) ++*launches;
  return e;
}

// One launch of the tcgen05 GEMM with the given plan (columns a.n_begin .. a.n_end).
static cudaError_t launch_one(const GemmArgs& a, const GemmPlan& plan, const CUtensorMap* tmap_w3,
                              const CUtensorMap* tmap_bx3, cudaStream_t stream) {
  CUtensorMap tmap_x;
  if (a.fp8) {
    tmap_x = *a.tmap_xq;
  } else {
    const cudaError_t e = encode_tmap_bf16(&tmap_x, a.x, a.M, a.K, kBM);
    if (e != cudaSuccess) return e;
  }
  // a CTA of a pair loads half of the N tile's rows: the map with boxes of block_n / 2 rows
  const int ti = gemm_tc_tile_index(plan.pair ? plan.block_n / 2 : plan.block_n);
  const CUtensorMap& tw = tmap_w3[ti];
  const CUtensorMap& tb = tmap_bx3 ? tmap_bx3[ti] : tw;  // unused in delta mode
  if (!a.ep.on) return launch_planned<kNoEpilogue>(a, plan, tmap_x, tw, tb, stream);
  switch (a.ep.act) {
    case LORA_ACT_NONE: return launch_planned_fused<LORA_ACT_NONE>(a, plan, tmap_x, tw, tb, stream);
    case LORA_ACT_RELU: return launch_planned_fused<LORA_ACT_RELU>(a, plan, tmap_x, tw, tb, stream);
    case LORA_ACT_GELU: return launch_planned_fused<LORA_ACT_GELU>(a, plan, tmap_x, tw, tb, stream);
    case LORA_ACT_GELU_TANH: return launch_planned_fused<LORA_ACT_GELU_TANH>(a, plan, tmap_x, tw, tb, stream);
    case LORA_ACT_SILU: return launch_planned_fused<LORA_ACT_SILU>(a, plan, tmap_x, tw, tb, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace lora
