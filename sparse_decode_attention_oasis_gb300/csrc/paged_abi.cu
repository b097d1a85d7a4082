// C ABI entry points of the paged 8-bit cache: argument validation, then the launches.
// No exception leaves an entry point: a message that cannot be built is a failed call.
#include <cmath>
#include <string>

#include "paged.cuh"

namespace oasis {
void set_last_error(const std::string& msg);
cudaError_t launch_extend_tables(const PagedShape&, const int*, const int*, const int*, const int*, int*, int*, int*,
                                 int*, int*, int, unsigned*, cudaStream_t);
cudaError_t launch_release_tables(const PagedShape&, const int*, const int*, const int*, int*, const int*, int*,
                                  unsigned*, cudaStream_t);
cudaError_t launch_store_kv_q8(const PagedShape&, const uint16_t*, size_t, const uint16_t*, size_t, const int*, int,
                               uint8_t*, float*, unsigned*, cudaStream_t);
size_t paged_attn_workspace_bytes(const PagedShape&);
cudaError_t launch_paged_decode_attn(const PagedShape&, const uint16_t*, size_t, const uint8_t*, const float*,
                                     const int*, const int*, const int*, const int*, int, float, void*, uint16_t*,
                                     unsigned*, cudaStream_t);
cudaError_t launch_prompt_attn(const PagedShape&, const uint16_t*, size_t, const uint16_t*, size_t, const uint16_t*,
                               size_t, const int*, int, float, uint16_t*, size_t, unsigned*, cudaStream_t);
}  // namespace oasis

namespace {

using oasis::PagedShape;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Call {  // a refused argument: the status and its text
  oasis_status status = OASIS_OK;
  const char* text = nullptr;
  bool refuse(bool bad, const char* why, oasis_status st = OASIS_ERR_INVALID) {
    if (bad && status == OASIS_OK) {
      status = st;
      text = why;
    }
    return status != OASIS_OK;
  }
};

oasis_status finish(const char* fn, const Call& c, cudaError_t e) noexcept {
  if (c.status == OASIS_OK && e == cudaSuccess) return OASIS_OK;
  try {
    oasis::set_last_error(c.status != OASIS_OK ? std::string(fn) + ": " + c.text
                                               : std::string(fn) + ": " + cudaGetErrorName(e) + " (" +
                                                     cudaGetErrorString(e) + ")");
  } catch (...) {
  }
  return c.status != OASIS_OK ? c.status : OASIS_ERR_CUDA;
}

PagedShape check_shape(const oasis_paged_shape* sh, Call* c) {
  if (c->refuse(!sh, "shape is NULL")) return PagedShape{};
  const oasis_paged_shape& s = *sh;
  if (c->refuse(s.B < 1 || s.Hq < 1 || s.Hkv < 1 || s.nb_max < 1 || s.n_pages < 1,
                "every shape field must be >= 1") ||
      c->refuse(s.Hq % s.Hkv != 0, "Hq must be a multiple of Hkv"))
    return PagedShape{};
  c->refuse(s.d != oasis::kD, "head dim must be 128", OASIS_ERR_UNSUPPORTED);
  c->refuse(s.bs != oasis::kBS, "block size must be 16 tokens", OASIS_ERR_UNSUPPORTED);
  c->refuse(s.Hq / s.Hkv > 8, "GQA group must be 1 .. 8", OASIS_ERR_UNSUPPORTED);
  c->refuse(s.B > 65535, "B must be <= 65535", OASIS_ERR_UNSUPPORTED);
  c->refuse(s.Hkv > 1024 || (long long)s.B * s.Hkv > (1 << 20), "Hkv must be <= 1024 and B * Hkv <= 2^20",
            OASIS_ERR_UNSUPPORTED);
  c->refuse(s.nb_max > (1 << 24), "nb_max must be <= 2^24", OASIS_ERR_UNSUPPORTED);
  c->refuse(s.n_pages > (1 << 27) - 1, "n_pages must be <= 2^27 - 1", OASIS_ERR_UNSUPPORTED);
  return PagedShape{s.B, s.Hq, s.Hkv, s.nb_max, s.n_pages};
}

// int32 arrays that must be there
bool ints(const void* p) { return p && aligned(p, 4); }

// rows of `width` elements of bf16, `stride` apart
bool rows_ok(const void* p, size_t stride, int width) {
  return p && aligned(p, 16) && stride % 8 == 0 && stride >= (size_t)width && stride < (size_t(1) << 32);
}

bool scale_ok(float scale) { return std::isfinite(scale) && scale > 0.f; }

}  // namespace

extern "C" {

oasis_status oasis_extend_tables(const oasis_paged_shape* shape, const int32_t* old_len, const int32_t* new_len,
                                 const int32_t* free_pages, const int32_t* n_free, int32_t* block_table,
                                 int32_t* len_out, int32_t* n_free_out, int32_t* row_start, int32_t* slot_map,
                                 int32_t n_rows, uint32_t* err_word, oasis_stream_t stream) {
  static const char* fn = "oasis_extend_tables";
  Call c;
  const PagedShape s = check_shape(shape, &c);
  c.refuse(!(ints(old_len) && ints(new_len) && ints(free_pages) && ints(n_free) && ints(block_table) &&
             ints(len_out) && ints(n_free_out) && ints(row_start)),
           "int32 arrays must be 4-byte aligned and non-NULL");
  c.refuse(n_rows < 0 || n_rows > (1 << 28), "n_rows must be in [0, 2^28]");
  c.refuse(n_rows > 0 && !ints(slot_map), "slot_map must be 4-byte aligned and non-NULL");
  c.refuse(!aligned(err_word, 4), "err_word must be 4-byte aligned");
  if (c.status == OASIS_OK) {
    auto overlap = [&](const int32_t* a, size_t na, const int32_t* b, size_t nb) { return a < b + nb && b < a + na; };
    const size_t B = (size_t)s.B;
    c.refuse(overlap(len_out, B, old_len, B) || overlap(len_out, B, new_len, B) || overlap(len_out, B, n_free, 1) ||
                 overlap(n_free_out, 1, old_len, B) || overlap(n_free_out, 1, new_len, B) || n_free_out == n_free,
             "len_out and n_free_out must not overlap old_len, new_len or n_free");
  }
  cudaError_t e = cudaSuccess;
  if (c.status == OASIS_OK)
    e = oasis::launch_extend_tables(s, old_len, new_len, free_pages, n_free, block_table, len_out, n_free_out,
                                    row_start, slot_map, n_rows, err_word, (cudaStream_t)stream);
  return finish(fn, c, e);
}

oasis_status oasis_release_tables(const oasis_paged_shape* shape, const int32_t* len, const int32_t* keep_len,
                                  const int32_t* block_table, int32_t* free_pages, const int32_t* n_free,
                                  int32_t* n_free_out, uint32_t* err_word, oasis_stream_t stream) {
  static const char* fn = "oasis_release_tables";
  Call c;
  const PagedShape s = check_shape(shape, &c);
  c.refuse(!(ints(len) && ints(keep_len) && ints(block_table) && ints(free_pages) && ints(n_free) && ints(n_free_out)),
           "int32 arrays must be 4-byte aligned and non-NULL");
  c.refuse(n_free_out == n_free, "n_free_out must not be n_free");
  c.refuse(!aligned(err_word, 4), "err_word must be 4-byte aligned");
  cudaError_t e = cudaSuccess;
  if (c.status == OASIS_OK)
    e = oasis::launch_release_tables(s, len, keep_len, block_table, free_pages, n_free, n_free_out, err_word,
                                     (cudaStream_t)stream);
  return finish(fn, c, e);
}

oasis_status oasis_store_kv_q8(const oasis_paged_shape* shape, const void* k, size_t k_stride, const void* v,
                               size_t v_stride, const int32_t* slot_map, int32_t n_rows, void* kv_pages,
                               float* kv_scale, uint32_t* err_word, oasis_stream_t stream) {
  static const char* fn = "oasis_store_kv_q8";
  Call c;
  const PagedShape s = check_shape(shape, &c);
  c.refuse(n_rows < 0 || n_rows > (1 << 28), "n_rows must be in [0, 2^28]");
  if (n_rows > 0) {
    c.refuse(!rows_ok(k, k_stride, s.Hkv * oasis::kD) || !rows_ok(v, v_stride, s.Hkv * oasis::kD),
             "k and v must be 16-byte aligned with strides that are multiples of 8 and at least Hkv * d");
    c.refuse(!ints(slot_map), "slot_map must be 4-byte aligned and non-NULL");
  }
  c.refuse(!kv_pages || !aligned(kv_pages, 16) || !kv_scale || !aligned(kv_scale, 8),
           "kv_pages must be 16-byte and kv_scale 8-byte aligned device pointers");
  c.refuse(!aligned(err_word, 4), "err_word must be 4-byte aligned");
  cudaError_t e = cudaSuccess;
  if (c.status == OASIS_OK)
    e = oasis::launch_store_kv_q8(s, (const uint16_t*)k, k_stride, (const uint16_t*)v, v_stride, slot_map, n_rows,
                                  (uint8_t*)kv_pages, kv_scale, err_word, (cudaStream_t)stream);
  return finish(fn, c, e);
}

size_t oasis_paged_attn_workspace_bytes(const oasis_paged_shape* shape) {
  Call c;
  const PagedShape s = check_shape(shape, &c);
  return finish("oasis_paged_attn_workspace_bytes", c, cudaSuccess) == OASIS_OK ? oasis::paged_attn_workspace_bytes(s)
                                                                                 : 0;
}

oasis_status oasis_paged_decode_attn_q8(const oasis_paged_shape* shape, const void* q, size_t q_stride,
                                        const void* kv_pages, const float* kv_scale, const int32_t* block_table,
                                        const int32_t* ctx_len, const int32_t* sel, const int32_t* nsel,
                                        int32_t sel_max, float scale, void* workspace, size_t ws_bytes, void* out,
                                        uint32_t* err_word, oasis_stream_t stream) {
  static const char* fn = "oasis_paged_decode_attn_q8";
  Call c;
  const PagedShape s = check_shape(shape, &c);
  c.refuse(!rows_ok(q, q_stride, s.Hq * oasis::kD),
           "q must be 16-byte aligned with a stride that is a multiple of 8 and at least Hq * d");
  c.refuse(!kv_pages || !aligned(kv_pages, 16) || !kv_scale || !aligned(kv_scale, 8),
           "kv_pages must be 16-byte and kv_scale 8-byte aligned device pointers");
  c.refuse(!ints(block_table) || !ints(ctx_len), "block_table and ctx_len must be 4-byte aligned and non-NULL");
  c.refuse((sel == nullptr) != (nsel == nullptr), "sel and nsel must be given together");
  c.refuse(!aligned(sel, 4) || !aligned(nsel, 4) || !aligned(err_word, 4), "int32 arrays must be 4-byte aligned");
  c.refuse(sel && (sel_max < 1 || sel_max > 65536), "sel_max must be in [1, 65536]");
  c.refuse(!scale_ok(scale), "scale must be a positive finite number");
  c.refuse(!out || !aligned(out, 16), "out must be a 16-byte aligned device pointer");
  c.refuse(!workspace || !aligned(workspace, 16), "workspace must be a 16-byte aligned device pointer");
  c.refuse(c.status == OASIS_OK && ws_bytes < oasis::paged_attn_workspace_bytes(s),
           "workspace too small (see oasis_paged_attn_workspace_bytes)");
  cudaError_t e = cudaSuccess;
  if (c.status == OASIS_OK)
    e = oasis::launch_paged_decode_attn(s, (const uint16_t*)q, q_stride, (const uint8_t*)kv_pages, kv_scale,
                                        block_table, ctx_len, sel, nsel, sel_max, scale, workspace, (uint16_t*)out,
                                        err_word, (cudaStream_t)stream);
  return finish(fn, c, e);
}

oasis_status oasis_prompt_attn(const oasis_paged_shape* shape, const void* q, size_t q_stride, const void* k,
                               size_t k_stride, const void* v, size_t v_stride, const int32_t* row_start,
                               int32_t n_rows, float scale, void* out, size_t out_stride, uint32_t* err_word,
                               oasis_stream_t stream) {
  static const char* fn = "oasis_prompt_attn";
  Call c;
  const PagedShape s = check_shape(shape, &c);
  c.refuse(n_rows < 0 || n_rows > (1 << 26), "n_rows must be in [0, 2^26]");
  c.refuse(!ints(row_start), "row_start must be 4-byte aligned and non-NULL");
  if (n_rows > 0) {
    c.refuse(!rows_ok(q, q_stride, s.Hq * oasis::kD) || !rows_ok(out, out_stride, s.Hq * oasis::kD),
             "q and out must be 16-byte aligned with strides that are multiples of 8 and at least Hq * d");
    c.refuse(!rows_ok(k, k_stride, s.Hkv * oasis::kD) || !rows_ok(v, v_stride, s.Hkv * oasis::kD),
             "k and v must be 16-byte aligned with strides that are multiples of 8 and at least Hkv * d");
  }
  c.refuse(!scale_ok(scale), "scale must be a positive finite number");
  c.refuse(!aligned(err_word, 4), "err_word must be 4-byte aligned");
  cudaError_t e = cudaSuccess;
  if (c.status == OASIS_OK)
    e = oasis::launch_prompt_attn(s, (const uint16_t*)q, q_stride, (const uint16_t*)k, k_stride, (const uint16_t*)v,
                                  v_stride, row_start, n_rows, scale, (uint16_t*)out, out_stride, err_word,
                                  (cudaStream_t)stream);
  return finish(fn, c, e);
}

}  // extern "C"
