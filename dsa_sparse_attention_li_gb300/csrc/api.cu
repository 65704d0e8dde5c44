// api.cu -- the C ABI (include/dsa.h): host-side validation, status codes, per-thread error
// text, TMA descriptor encoding and device-property caching.  No entry point allocates memory,
// synchronises, or keeps a pointer after it returns.
#include <cudaTypedefs.h>

#include <mutex>
#include <string>
#include <unordered_set>
#include <vector>

#include "dsa_internal.h"

namespace {

thread_local std::string g_last_error;

dsa_status fail(dsa_status s, const std::string& why) {
  g_last_error = why;
  return s;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

namespace dsa {

#ifdef DSA_TEST_HOOKS
int g_test_stall = 0;
#endif

void set_last_error(const std::string& why) { g_last_error = why; }

bool device_info(DeviceInfo& info, std::string& err) {
  static std::mutex mu;
  static std::vector<DeviceInfo> cache(64);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) {
    err = std::string("cudaGetDevice: ") + cudaGetErrorString(e);
    return false;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < (int)cache.size() && cache[dev].device == dev) {
    info = cache[dev];
    return true;
  }
  DeviceInfo d;
  d.device = dev;
  e = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&d.smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e != cudaSuccess) {
    err = std::string("cudaDeviceGetAttribute: ") + cudaGetErrorString(e);
    return false;
  }
  if (dev >= 0 && dev < (int)cache.size()) cache[dev] = d;
  info = d;
  return true;
}

static bool encode_tmap(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, uint32_t rank,
                        const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                        CUtensorMapSwizzle swizzle, std::string& err) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (!fn) {
    err = "cuTensorMapEncodeTiled is not available from the driver";
    return false;
  }
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, dtype, rank, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    err = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r);
    return false;
  }
  return true;
}

bool encode_tmap_2d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, uint64_t inner,
                    uint64_t outer, uint64_t row_stride_bytes, uint32_t box_inner,
                    uint32_t box_outer, CUtensorMapSwizzle swizzle, std::string& err) {
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {row_stride_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  return encode_tmap(map, dtype, base, 2, dims, strides, box, swizzle, err);
}

bool encode_tmap_3d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, const uint64_t dims[3],
                    const uint64_t strides[2], const uint32_t box[3], CUtensorMapSwizzle swizzle,
                    std::string& err) {
  cuuint64_t d[3] = {dims[0], dims[1], dims[2]};
  cuuint64_t s[2] = {strides[0], strides[1]};
  cuuint32_t b[3] = {box[0], box[1], box[2]};
  return encode_tmap(map, dtype, base, 3, d, s, b, swizzle, err);
}

}  // namespace dsa

extern "C" {

const char* dsa_status_string(dsa_status s) {
  switch (s) {
    case DSA_OK: return "DSA_OK";
    case DSA_ERR_INVALID_ARG: return "DSA_ERR_INVALID_ARG";
    case DSA_ERR_UNSUPPORTED: return "DSA_ERR_UNSUPPORTED";
    case DSA_ERR_CUDA: return "DSA_ERR_CUDA";
    case DSA_ERR_DEVICE_CHECK: return "DSA_ERR_DEVICE_CHECK";
    case DSA_ERR_TIMEOUT: return "DSA_ERR_TIMEOUT";
  }
  return "DSA_ERR_UNKNOWN";
}

const char* dsa_last_error(void) { return g_last_error.c_str(); }

int dsa_abi_version(void) { return DSA_ABI_VERSION; }

size_t dsa_page_bytes(dsa_dtype dtype, int rows, int dim) {
  if (rows < 0 || dim < 0) return 0;
  const size_t elt = dtype == DSA_BF16 ? 2 : ((dtype == DSA_FP8_E4M3 || dtype == DSA_MXFP8_E4M3) ? 1 : 0);
  return elt * (size_t)rows * (size_t)dim;
}

dsa_status dsa_page_table_validate(const int32_t* pt, int B, int max_pages, const int32_t* seq_lens,
                                   int page_size, int num_pages, int require_unique) {
  g_last_error.clear();
  if (!pt || !seq_lens || B <= 0 || max_pages <= 0 || page_size <= 0 || num_pages <= 0)
    return fail(DSA_ERR_INVALID_ARG, "page_table_validate: null pointer or non-positive size");
  std::vector<uint8_t> used(require_unique ? (size_t)num_pages : 0, 0);
  for (int b = 0; b < B; ++b) {
    const long long L = seq_lens[b];
    if (L < 0) return fail(DSA_ERR_INVALID_ARG, "seq_lens[" + std::to_string(b) + "] < 0");
    const long long np = (L + page_size - 1) / page_size;
    if (np > max_pages)
      return fail(DSA_ERR_INVALID_ARG, "sequence " + std::to_string(b) + " needs " +
                                           std::to_string(np) + " pages > max_pages");
    for (long long p = 0; p < np; ++p) {
      const int id = pt[(size_t)b * max_pages + p];
      if (id < 0 || id >= num_pages)
        return fail(DSA_ERR_INVALID_ARG, "page_table[" + std::to_string(b) + "][" +
                                             std::to_string(p) + "] = " + std::to_string(id) +
                                             " out of [0, num_pages)");
      if (require_unique) {
        if (used[id])
          return fail(DSA_ERR_INVALID_ARG, "page " + std::to_string(id) + " used twice");
        used[id] = 1;
      }
    }
  }
  return DSA_OK;
}

dsa_status dsa_li_topk(const dsa_li_args* a, dsa_stream_t stream) {
  g_last_error.clear();
  if (!a) return fail(DSA_ERR_INVALID_ARG, "li_topk: args is NULL");
  if (a->B <= 0 || a->n_q < 0 || a->K <= 0 || a->max_pages <= 0 || a->num_pages <= 0 ||
      a->H_I <= 0 || a->d_I <= 0)
    return fail(DSA_ERR_INVALID_ARG, "li_topk: non-positive size");
  if (a->dtype != DSA_BF16 && a->dtype != DSA_FP8_E4M3 && a->dtype != DSA_MXFP8_E4M3)
    return fail(DSA_ERR_INVALID_ARG, "li_topk: unknown dtype");
  if (a->n_q == 0) return DSA_OK;
  if (!a->q || !a->w || !a->k_pool || !a->page_table || !a->seq_lens || !a->q_start || !a->out_idx)
    return fail(DSA_ERR_INVALID_ARG, "li_topk: null device pointer");
  if (a->dtype == DSA_FP8_E4M3 && (!a->q_scale || !a->k_scale))
    return fail(DSA_ERR_INVALID_ARG, "li_topk: FP8 needs q_scale and k_scale");
  if (a->dtype == DSA_MXFP8_E4M3 &&
      (!a->q_sf || !a->k_sf || ((reinterpret_cast<uintptr_t>(a->q_sf) | reinterpret_cast<uintptr_t>(a->k_sf)) & 3u) != 0))
    return fail(DSA_ERR_INVALID_ARG, "li_topk: MXFP8 needs 4-byte aligned q_sf and k_sf");
  if (a->max_seq_len <= 0 || a->max_q_per_seq <= 0 || a->max_q_per_seq > a->n_q)
    return fail(DSA_ERR_INVALID_ARG, "li_topk: max_seq_len / max_q_per_seq out of range");
  if ((long long)a->max_seq_len > (long long)a->max_pages * a->page_size)
    return fail(DSA_ERR_INVALID_ARG, "li_topk: max_seq_len exceeds max_pages * page_size");
  if (!aligned16(a->q) || !aligned16(a->k_pool))
    return fail(DSA_ERR_INVALID_ARG, "li_topk: q and k_pool must be 16-byte aligned");
  if (a->page_size != 64) return fail(DSA_ERR_UNSUPPORTED, "li_topk: page_size must be 64");
  if (a->K > 2048) return fail(DSA_ERR_UNSUPPORTED, "li_topk: K > 2048");
  if (a->max_seq_len > 131072) return fail(DSA_ERR_UNSUPPORTED, "li_topk: max_seq_len > 131072");
  if (a->workspace != nullptr && (reinterpret_cast<uintptr_t>(a->workspace) & 255u) != 0)
    return fail(DSA_ERR_INVALID_ARG, "li_topk: workspace must be 256-byte aligned");
  std::string err;
  const dsa_status s = dsa::launch_li_topk(*a, reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

size_t dsa_li_workspace_bytes(const dsa_li_args* a) {
  if (!a || a->B <= 0 || a->K <= 0 || a->max_seq_len <= 0 || a->max_q_per_seq <= 0) return 0;
  return dsa::li_workspace_bytes(*a);
}

static dsa_status sfa_common(const dsa_sfa_args* a, bool prefill, dsa_stream_t stream) {
  g_last_error.clear();
  const char* name = prefill ? "sfa_prefill" : "sfa_decode";
  if (!a) return fail(DSA_ERR_INVALID_ARG, std::string(name) + ": args is NULL");
  if (a->B <= 0 || a->n_q < 0 || a->H <= 0 || a->K <= 0 || a->max_pages <= 0 || a->num_pages <= 0)
    return fail(DSA_ERR_INVALID_ARG, std::string(name) + ": non-positive size");
  if (!(a->softmax_scale > 0.f) || a->softmax_scale != a->softmax_scale)
    return fail(DSA_ERR_INVALID_ARG, std::string(name) + ": softmax_scale must be positive");
  if (a->n_q == 0) return DSA_OK;
  if (!a->q || !a->kv_pool || !a->page_table || !a->seq_lens || !a->q_start || !a->idx || !a->out)
    return fail(DSA_ERR_INVALID_ARG, std::string(name) + ": null device pointer");
  if (!aligned16(a->q) || !aligned16(a->kv_pool) || !aligned16(a->out))
    return fail(DSA_ERR_INVALID_ARG, std::string(name) + ": q, kv_pool, out must be 16-byte aligned");
  if (a->d_qk != 576 || a->d_v != 512)
    return fail(DSA_ERR_UNSUPPORTED, std::string(name) + ": d_qk must be 576 and d_v 512");
  if (a->page_size != 64) return fail(DSA_ERR_UNSUPPORTED, std::string(name) + ": page_size must be 64");
  if (a->kv_dtype != DSA_BF16 && a->kv_dtype != DSA_FP8_E4M3)
    return fail(DSA_ERR_UNSUPPORTED, std::string(name) + ": kv_dtype must be BF16 or FP8_E4M3");
  if (a->H > 128) return fail(DSA_ERR_UNSUPPORTED, std::string(name) + ": H > 128");
  if (a->K > 2048) return fail(DSA_ERR_UNSUPPORTED, std::string(name) + ": K > 2048");
  std::string err;
  const dsa_status s = dsa::launch_sfa(*a, prefill, reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

size_t dsa_sfa_workspace_bytes(const dsa_sfa_args* a) {
  if (!a || a->n_q <= 0 || a->K <= 0) return 0;
  return dsa::sfa_workspace_bytes(*a);
}

dsa_status dsa_sfa_decode(const dsa_sfa_args* a, dsa_stream_t stream) {
  return sfa_common(a, false, stream);
}

dsa_status dsa_sfa_prefill(const dsa_sfa_args* a, dsa_stream_t stream) {
  return sfa_common(a, true, stream);
}

// A softmax scale and its product with log2(e) are positive and finite.
static bool scale_ok(float s) { return s > 0.f && s <= 2.0e38f; }

static dsa_status mla_decode_check(const dsa_mla_decode_args* a) {
  if (!a) return fail(DSA_ERR_INVALID_ARG, "mla_decode: args is NULL");
  if (a->B <= 0 || a->n_q < 0 || a->H <= 0 || a->max_pages <= 0 || a->num_pages <= 0 || a->max_q_per_seq <= 0)
    return fail(DSA_ERR_INVALID_ARG, "mla_decode: non-positive size");
  if (a->H > 128) return fail(DSA_ERR_UNSUPPORTED, "mla_decode: H > 128");
  if (!scale_ok(a->softmax_scale))
    return fail(DSA_ERR_INVALID_ARG, "mla_decode: softmax_scale must be positive and finite");
  if (a->d_qk != 576 || a->d_v != 512) return fail(DSA_ERR_UNSUPPORTED, "mla_decode: d_qk must be 576 and d_v 512");
  if (a->page_size != 64) return fail(DSA_ERR_UNSUPPORTED, "mla_decode: page_size must be 64");
  if (a->kv_dtype != DSA_BF16 && a->kv_dtype != DSA_FP8_E4M3)
    return fail(DSA_ERR_UNSUPPORTED, "mla_decode: kv_dtype must be BF16 or FP8_E4M3");
  if ((long long)a->max_pages * 64 > 0x7ffffe00LL || (long long)a->num_pages * 64 > 0x7fffffffLL ||
      (long long)a->n_q * a->H > 0x7fffffffLL)
    return fail(DSA_ERR_UNSUPPORTED, "mla_decode: positions, cache rows and query rows must number below 2^31");
  if (a->n_q == 0) return DSA_OK;
  if (!a->q || !a->kv_pool || !a->page_table || !a->seq_lens || !a->q_start || !a->out)
    return fail(DSA_ERR_INVALID_ARG, "mla_decode: null device pointer");
  if (!aligned16(a->q) || !aligned16(a->kv_pool) || (reinterpret_cast<uintptr_t>(a->out) & 31u))
    return fail(DSA_ERR_INVALID_ARG, "mla_decode: q and kv_pool must be 16-byte aligned, out 32-byte aligned");
  if (a->workspace != nullptr && (reinterpret_cast<uintptr_t>(a->workspace) & 255u) != 0)
    return fail(DSA_ERR_INVALID_ARG, "mla_decode: workspace must be 256-byte aligned");
  const size_t need = dsa::mla_decode_workspace_bytes(*a);
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need))
    return fail(DSA_ERR_INVALID_ARG, "mla_decode: workspace of " + std::to_string(need) + " bytes required (got " +
                                         std::to_string(a->workspace ? a->workspace_bytes : 0) + ")");
  return DSA_OK;
}

size_t dsa_mla_decode_workspace_bytes(const dsa_mla_decode_args* a) {
  if (!a || a->n_q <= 0 || a->H <= 0 || a->H > 128 || a->max_q_per_seq <= 0) return 0;
  return dsa::mla_decode_workspace_bytes(*a);
}

dsa_status dsa_mla_decode(const dsa_mla_decode_args* a, dsa_stream_t stream) {
  g_last_error.clear();
  const dsa_status c = mla_decode_check(a);
  if (c != DSA_OK || a->n_q == 0) return c;
  std::string err;
  const dsa_status s = dsa::launch_mla_decode(*a, reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

dsa_status dsa_mla_prefill(const dsa_mla_prefill_args* a, dsa_stream_t stream) {
  g_last_error.clear();
  if (!a) return fail(DSA_ERR_INVALID_ARG, "mla_prefill: args is NULL");
  if (a->B <= 0 || a->n_q < 0 || a->n_kv < 0 || a->H <= 0 || a->max_q_per_seq <= 0)
    return fail(DSA_ERR_INVALID_ARG, "mla_prefill: non-positive size");
  if (!scale_ok(a->softmax_scale))
    return fail(DSA_ERR_INVALID_ARG, "mla_prefill: softmax_scale must be positive and finite");
  if (a->d_nope != 128 || a->d_rope != 64 || a->d_v != 128)
    return fail(DSA_ERR_UNSUPPORTED, "mla_prefill: d_nope must be 128, d_rope 64 and d_v 128");
  if (a->H > 1024) return fail(DSA_ERR_UNSUPPORTED, "mla_prefill: H > 1024");
  if (a->k_rope_stride < a->d_rope) return fail(DSA_ERR_INVALID_ARG, "mla_prefill: k_rope_stride below d_rope");
  if (a->k_rope_stride % 8) return fail(DSA_ERR_UNSUPPORTED, "mla_prefill: k_rope rows must start 16-byte aligned");
  if (a->n_q == 0) return DSA_OK;
  if (!a->q || (a->n_kv > 0 && (!a->kv || !a->k_rope)) || !a->q_start || !a->kv_start || !a->out)
    return fail(DSA_ERR_INVALID_ARG, "mla_prefill: null device pointer");
  if (!aligned16(a->q) || !aligned16(a->kv) || !aligned16(a->k_rope) || (reinterpret_cast<uintptr_t>(a->out) & 31u))
    return fail(DSA_ERR_INVALID_ARG, "mla_prefill: q, kv, k_rope must be 16-byte aligned, out 32-byte aligned");
  std::string err;
  const dsa_status s = dsa::launch_mla_prefill(*a, reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

static bool elem_ok(dsa_elem e) { return e == DSA_ELEM_BF16 || e == DSA_ELEM_FP16 || e == DSA_ELEM_FP32; }

// Rows of `dim` elements (of 2 or 4 bytes) that lie `stride` elements apart start on 16 bytes; one row has no stride.
static const char* rows_wrong(const void* p, long long stride, int rows, int dim, dsa_elem e) {
  if (!aligned16(p)) return "must be 16-byte aligned";
  if (rows <= 1) return nullptr;
  if (stride < dim || stride > (1LL << 40)) return "has a row stride below dim, or beyond 2^40";
  return stride % (e == DSA_ELEM_FP32 ? 4 : 8) ? "has rows that do not start 16-byte aligned" : nullptr;
}

// The 8-bit rows that a call writes.
static const char* rows8_wrong(const void* codes, long long codes_stride, const float* scale, long long scale_stride,
                               int rows, int dim) {
  if ((reinterpret_cast<uintptr_t>(codes) & 7u) || (rows > 1 && codes_stride % 8)) return "codes must have rows that start 8-byte aligned";
  if (reinterpret_cast<uintptr_t>(scale) & 3u) return "scale must be 4-byte aligned";
  if (rows > 1 && (codes_stride < dim || codes_stride > (1LL << 40))) return "codes has a row stride below dim, or beyond 2^40";
  if (rows > 1 && (scale_stride < (dim + 127) / 128 || scale_stride > (1LL << 40))) return "scale has a row stride below its columns, or beyond 2^40";
  return nullptr;
}

dsa_status dsa_rms_norm_quant(const dsa_rms_norm_quant_args* a, dsa_stream_t stream) {
  g_last_error.clear();
  const std::string name = "rms_norm_quant: ";
  if (!a) return fail(DSA_ERR_INVALID_ARG, name + "args is NULL");
  if (a->n_rows < 0 || a->dim <= 0) return fail(DSA_ERR_INVALID_ARG, name + "non-positive size");
  if (!elem_ok(a->elem) || !elem_ok(a->weight_elem)) return fail(DSA_ERR_INVALID_ARG, name + "unknown element type");
  if (a->weight_elem != a->elem && a->weight_elem != DSA_ELEM_FP32)
    return fail(DSA_ERR_UNSUPPORTED, name + "weight must have the type of x, or fp32");
  if (a->dim % 8 || a->dim > 32768) return fail(DSA_ERR_UNSUPPORTED, name + "dim must be a multiple of 8, up to 32768");
  if (!(a->eps >= 0.f && a->eps <= 3.0e38f)) return fail(DSA_ERR_INVALID_ARG, name + "eps must be finite and not negative");
  if (a->n_rows == 0) return DSA_OK;
  if (!a->x || !a->weight || !a->codes || !a->scale) return fail(DSA_ERR_INVALID_ARG, name + "null device pointer");
  if ((a->residual == nullptr) != (a->sum == nullptr))
    return fail(DSA_ERR_INVALID_ARG, name + "residual and sum go together");
  if (!aligned16(a->weight)) return fail(DSA_ERR_INVALID_ARG, name + "weight must be 16-byte aligned");
  const struct { const char* what; const void* p; long long stride; } rows[] = {
      {"x ", a->x, a->x_stride}, {"residual ", a->residual, a->residual_stride}, {"sum ", a->sum, a->sum_stride},
      {"y ", a->y, a->y_stride}};
  for (const auto& r : rows) {
    const char* why = r.p ? rows_wrong(r.p, r.stride, a->n_rows, a->dim, a->elem) : nullptr;
    if (why) return fail(DSA_ERR_INVALID_ARG, name + r.what + why);
  }
  if (const char* why = rows8_wrong(a->codes, a->codes_stride, a->scale, a->scale_stride, a->n_rows, a->dim))
    return fail(DSA_ERR_INVALID_ARG, name + why);
  std::string err;
  const dsa_status s = dsa::launch_rms_norm_quant(*a, reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

dsa_status dsa_quant_rows(const dsa_quant_rows_args* a, dsa_stream_t stream) {
  g_last_error.clear();
  const std::string name = "quant_rows: ";
  if (!a) return fail(DSA_ERR_INVALID_ARG, name + "args is NULL");
  if (a->n_rows < 0 || a->dim <= 0) return fail(DSA_ERR_INVALID_ARG, name + "non-positive size");
  if (!elem_ok(a->elem)) return fail(DSA_ERR_INVALID_ARG, name + "unknown element type");
  if (a->dim % 8 || a->dim > 0x40000000) return fail(DSA_ERR_UNSUPPORTED, name + "dim must be a multiple of 8, up to 2^30");
  if (a->n_rows == 0) return DSA_OK;
  if (!a->x || !a->codes || !a->scale) return fail(DSA_ERR_INVALID_ARG, name + "null device pointer");
  if (const char* why = rows_wrong(a->x, a->x_stride, a->n_rows, a->dim, a->elem))
    return fail(DSA_ERR_INVALID_ARG, name + "x " + why);
  if (const char* why = rows8_wrong(a->codes, a->codes_stride, a->scale, a->scale_stride, a->n_rows, a->dim))
    return fail(DSA_ERR_INVALID_ARG, name + why);
  std::string err;
  const dsa_status s = dsa::launch_quant_rows(*a, reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

dsa_status dsa_matmul_fp8(const dsa_matmul_fp8_args* a, dsa_stream_t stream) {
  g_last_error.clear();
  const std::string name = "matmul_fp8: ";
  if (!a) return fail(DSA_ERR_INVALID_ARG, name + "args is NULL");
  if (a->M < 0 || a->N <= 0 || a->K <= 0) return fail(DSA_ERR_INVALID_ARG, name + "non-positive size");
  if (!elem_ok(a->elem)) return fail(DSA_ERR_INVALID_ARG, name + "unknown element type");
  if (a->K % 16) return fail(DSA_ERR_UNSUPPORTED, name + "K must be a multiple of 16");
  if (a->M > 0x7fffff00 || a->N > 0x7fffff00 || a->K > 0x7fffff00)
    return fail(DSA_ERR_UNSUPPORTED, name + "M, N and K must be at most 2^31 - 256");
  if (a->M == 0) return DSA_OK;
  if (!a->a || !a->a_scale || !a->b || !a->b_scale || !a->out)
    return fail(DSA_ERR_INVALID_ARG, name + "null device pointer");
  const long long blocks = ((long long)a->K + 127) / 128, n_blocks = ((long long)a->N + 127) / 128;
  const struct { const char* what; const void* p; long long stride, rows, least, align; } parts[] = {
      {"a ", a->a, a->a_stride, a->M, a->K, 16}, {"b ", a->b, a->b_stride, a->N, a->K, 16},
      {"a_scale ", a->a_scale, a->a_scale_stride * 4, a->M, blocks * 4, 4},
      {"b_scale ", a->b_scale, a->b_scale_stride * 4, n_blocks, blocks * 4, 4},
      {"out ", a->out, a->out_stride * (a->elem == DSA_ELEM_FP32 ? 4 : 2), a->M,
       (long long)a->N * (a->elem == DSA_ELEM_FP32 ? 4 : 2), a->elem == DSA_ELEM_FP32 ? 4 : 2}};
  for (const auto& r : parts) {
    if (reinterpret_cast<uintptr_t>(r.p) % r.align || (r.rows > 1 && r.stride % r.align))
      return fail(DSA_ERR_INVALID_ARG, name + r.what + "must have rows that start " + std::to_string(r.align) + "-byte aligned");
    if (r.rows > 1 && (r.stride < r.least || r.stride >= (1LL << 40)))
      return fail(DSA_ERR_INVALID_ARG, name + r.what + "has a row stride below its columns, or of 2^40 bytes");
  }
  std::string err;
  const dsa_status s = dsa::launch_matmul_fp8(*a, reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

dsa_status dsa_topk_merge(const dsa_topk_merge_args* a, dsa_stream_t stream) {
  g_last_error.clear();
  if (!a) return fail(DSA_ERR_INVALID_ARG, "topk_merge: null args");
  if (a->S <= 0 || a->n_q < 0 || a->K_in <= 0 || a->K <= 0)
    return fail(DSA_ERR_INVALID_ARG, "topk_merge: non-positive size");
  if ((long long)a->S * a->K_in > 16384 || a->K > 16384)
    return fail(DSA_ERR_UNSUPPORTED, "topk_merge: S * K_in and K must be at most 16384");
  if (a->n_q > 0 && (!a->cand_idx || !a->cand_score || !a->shard_offset || !a->out_idx))
    return fail(DSA_ERR_INVALID_ARG, "topk_merge: null device pointer");
  std::string err;
  const dsa_status s = dsa::launch_topk_merge(*a, reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

static dsa_status prolog_check(const dsa_prolog_args* a, bool pointers) {
  if (!a) return fail(DSA_ERR_INVALID_ARG, "indexer_prolog: null args");
  if (a->n_q < 0 || a->B <= 0 || a->d_q <= 0 || a->d_model <= 0 || a->max_pages <= 0 ||
      a->num_pages <= 0)
    return fail(DSA_ERR_INVALID_ARG, "indexer_prolog: non-positive size");
  if (a->H_I != 64 || a->d_I != 128 || a->page_size != 64)
    return fail(DSA_ERR_UNSUPPORTED, "indexer_prolog: needs H_I 64, d_I 128, page_size 64");
  if (a->dtype != DSA_MXFP8_E4M3 && a->dtype != DSA_BF16)
    return fail(DSA_ERR_UNSUPPORTED, "indexer_prolog: dtype must be MXFP8_E4M3 or BF16");
  if (a->d_q % 8 || a->d_model % 8)
    return fail(DSA_ERR_UNSUPPORTED, "indexer_prolog: d_q and d_model must be multiples of 8");
  if (!pointers) return DSA_OK;  // sizes only (workspace query)
  if (!a->xq || !a->x || !a->w_q || !a->w_k || !a->w_w || !a->ln_gamma || !a->ln_beta ||
      !a->page_table || !a->seq_lens || !a->q_start || !a->q_out || !a->w_out || !a->k_pool ||
      (a->dtype == DSA_MXFP8_E4M3 && (!a->q_sf || !a->k_sf)))
    return fail(DSA_ERR_INVALID_ARG, "indexer_prolog: null device pointer");
  if (!aligned16(a->xq) || !aligned16(a->x) || !aligned16(a->w_q) || !aligned16(a->w_k) ||
      !aligned16(a->w_w))
    return fail(DSA_ERR_INVALID_ARG, "indexer_prolog: inputs and weights must be 16-byte aligned");
  return DSA_OK;
}

size_t dsa_prolog_workspace_bytes(const dsa_prolog_args* a) {
  if (prolog_check(a, false) != DSA_OK) return 0;
  return dsa::prolog_workspace_bytes(*a);
}

dsa_status dsa_indexer_prolog(const dsa_prolog_args* a, dsa_stream_t stream) {
  g_last_error.clear();
  const dsa_status c = prolog_check(a, true);
  if (c != DSA_OK) return c;
  std::string err;
  const dsa_status s = dsa::launch_prolog(*a, reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

dsa_status dsa_cache_write(void* pool, float* scale_pool, int num_pages, int page_size, int dim,
                           int elem_bytes, const int32_t* page_table, int max_pages, int B,
                           const int32_t* seq, const int32_t* pos, const void* rows,
                           const float* row_scales, int n_rows, int32_t* status,
                           dsa_stream_t stream) {
  g_last_error.clear();
  if (n_rows < 0 || num_pages <= 0 || page_size <= 0 || dim <= 0 || max_pages <= 0 || B <= 0)
    return fail(DSA_ERR_INVALID_ARG, "cache_write: non-positive size");
  if (elem_bytes != 1 && elem_bytes != 2)
    return fail(DSA_ERR_INVALID_ARG, "cache_write: elem_bytes must be 1 or 2");
  if ((dim * elem_bytes) % 16 != 0)
    return fail(DSA_ERR_UNSUPPORTED, "cache_write: row bytes must be a multiple of 16");
  if (n_rows == 0) return DSA_OK;
  if (!pool || !page_table || !seq || !pos || !rows)
    return fail(DSA_ERR_INVALID_ARG, "cache_write: null device pointer");
  if (!aligned16(pool) || !aligned16(rows))
    return fail(DSA_ERR_INVALID_ARG, "cache_write: pool and rows must be 16-byte aligned");
  if ((scale_pool == nullptr) != (row_scales == nullptr))
    return fail(DSA_ERR_INVALID_ARG, "cache_write: scale_pool and row_scales go together");
  std::string err;
  const dsa_status s = dsa::launch_cache_write(pool, scale_pool, num_pages, page_size, dim,
                                               elem_bytes, page_table, max_pages, B, seq, pos,
                                               rows, row_scales, n_rows, status,
                                               reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

static dsa_status cache_rows(const dsa_cache_rows_args* a, bool write, dsa_stream_t stream) {
  g_last_error.clear();
  const std::string name = write ? "cache_write_quant" : "cache_read";
  if (!a) return fail(DSA_ERR_INVALID_ARG, name + ": args is NULL");
  if (a->n_rows < 0 || a->dim <= 0 || a->B <= 0 || a->page_size <= 0 || a->max_pages <= 0 ||
      a->num_pages <= 0)
    return fail(DSA_ERR_INVALID_ARG, name + ": non-positive size");
  if (a->elem != DSA_ELEM_BF16 && a->elem != DSA_ELEM_FP16 && a->elem != DSA_ELEM_FP32)
    return fail(DSA_ERR_INVALID_ARG, name + ": unknown element type of rows");
  switch (a->format) {
    case DSA_ROW_BF16:
      if (write) return fail(DSA_ERR_UNSUPPORTED, name + ": a bf16 cache is written by dsa_cache_write");
      if (a->dim % 8) return fail(DSA_ERR_UNSUPPORTED, name + ": dim must be a multiple of 8");
      break;
    case DSA_ROW_FP8:
    case DSA_ROW_MXFP8:
      if (a->dim != 32 && a->dim != 64 && a->dim != 128 && a->dim != 256)
        return fail(DSA_ERR_UNSUPPORTED, name + ": dim must be 32, 64, 128 or 256");
      break;
    case DSA_ROW_LATENT_FP8:
      if (a->dim != 576) return fail(DSA_ERR_UNSUPPORTED, name + ": latent rows have 576 columns");
      break;
    default:
      return fail(DSA_ERR_INVALID_ARG, name + ": unknown cache format");
  }
  if (a->row_stride < a->dim) return fail(DSA_ERR_INVALID_ARG, name + ": row_stride below dim");
  if (a->row_stride % (a->elem == DSA_ELEM_FP32 ? 4 : 8))
    return fail(DSA_ERR_UNSUPPORTED, name + ": rows must start 16-byte aligned");
  if (a->row_stride > 0x7fffffffLL || (long long)a->num_pages * a->page_size > 0x7fffffffLL)
    return fail(DSA_ERR_UNSUPPORTED, name + ": row_stride and the cache's rows must be below 2^31");
  if (a->n_rows == 0) return DSA_OK;
  if (!a->rows || !a->pool || !a->page_table || !a->seq || !a->pos)
    return fail(DSA_ERR_INVALID_ARG, name + ": null device pointer");
  if ((a->format == DSA_ROW_FP8 && !a->scale_pool) || (a->format == DSA_ROW_MXFP8 && !a->sf_pool))
    return fail(DSA_ERR_INVALID_ARG, name + ": FP8 needs scale_pool, MXFP8 needs sf_pool");
  if (!aligned16(a->rows) || !aligned16(a->pool))
    return fail(DSA_ERR_INVALID_ARG, name + ": rows and pool must be 16-byte aligned");
  std::string err;
  const dsa_status s = dsa::launch_cache_rows(*a, write, reinterpret_cast<cudaStream_t>(stream), err);
  if (s != DSA_OK) g_last_error = err;
  return s;
}

dsa_status dsa_cache_write_quant(const dsa_cache_rows_args* a, dsa_stream_t stream) {
  return cache_rows(a, true, stream);
}

dsa_status dsa_cache_read(const dsa_cache_rows_args* a, dsa_stream_t stream) {
  return cache_rows(a, false, stream);
}

#ifdef DSA_TEST_HOOKS
// Test build only (libdsa_testhooks.so; include/dsa_testhooks.h).
void dsa_test_inject_stall(int kernel) { dsa::g_test_stall = kernel; }
#endif

}  // extern "C"
