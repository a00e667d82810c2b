// Host-side argument validation of the entry points of forge_ops.h (pure C++,
// no HIP).
#include "validate_ops.hpp"

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

namespace forge {

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Byte ranges of one call, read only or written.
struct Range {
  uintptr_t begin, end;
  bool written;
};

// Collects a call's ranges and looks for a written one that overlaps another.
// Sorting instead of comparing pairs keeps a list of thousands of tensors
// cheap; the caller's order is usually ascending already.
class Ranges {
 public:
  explicit Ranges(int64_t room) : r_(new (std::nothrow) Range[size_t(room)]) {}
  bool ok() const { return r_ != nullptr; }
  void add(const void* p, uint64_t bytes, bool written) {
    if (bytes == 0) return;
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    r_[n_++] = Range{b, b + bytes, written};
  }
  bool clash() {
    std::sort(r_.get(), r_.get() + n_, [](const Range& a, const Range& b) { return a.begin < b.begin; });
    uintptr_t any = 0, written = 0;      // ends of what came before
    for (int64_t k = 0; k < n_; ++k) {
      if (r_[k].begin < written || (r_[k].written && r_[k].begin < any)) return true;
      any = std::max(any, r_[k].end);
      if (r_[k].written) written = std::max(written, r_[k].end);
    }
    return false;
  }

 private:
  std::unique_ptr<Range[]> r_;
  int64_t n_ = 0;
};

// An array of a list: its table holds addresses below 2^52 (which all are).
bool aligned_entry(const void* p) { return aligned16(p) && uint64_t(reinterpret_cast<uintptr_t>(p)) >> 52 == 0; }

// Which of a tensor's fields a call uses, beside grad, n and grad_dtype.
enum : int { USE_OUT = 1, USE_W_M = 2, USE_V = 4 };

forge_status check_list(const forge_tensor* tensors, int32_t count, int use) {
  if (count < 0 || count > FORGE_MAX_TENSORS) return FORGE_ERR_SHAPE;
  if (count > 0 && !tensors) return FORGE_ERR_NULL;
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    const forge_tensor& t = tensors[i];
    if (t.n == 0) continue;
    if (t.n < 0 || t.n > kMaxElems) return FORGE_ERR_SHAPE;
    if (dtype_bytes(t.grad_dtype) == 0) return FORGE_ERR_DTYPE;
    if (!t.grad || ((use & USE_OUT) && !t.out) || ((use & USE_W_M) && (!t.W || !t.m)) ||
        ((use & USE_V) && !t.v))
      return FORGE_ERR_NULL;
    if (!aligned_entry(t.grad) || ((use & USE_OUT) && !aligned_entry(t.out)) ||
        ((use & USE_W_M) && (!aligned_entry(t.W) || !aligned_entry(t.m))) ||
        ((use & USE_V) && !aligned_entry(t.v)))
      return FORGE_ERR_ALIGN;
    total += t.n;
    if (total > kMaxListElems) return FORGE_ERR_SHAPE;
  }
  return FORGE_OK;
}

forge_status check_list_overlap(const forge_tensor* tensors, int32_t count, const float* coef,
                                int use) {
  Ranges r(4 * int64_t(count) + 1);
  if (!r.ok()) return FORGE_ERR_SHAPE;
  r.add(coef, 4, false);
  for (int32_t i = 0; i < count; ++i) {
    const forge_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const uint64_t gb = uint64_t(t.n) * uint64_t(dtype_bytes(t.grad_dtype));
    const uint64_t sb = uint64_t(t.n) * 4u;
    if (!((use & USE_OUT) && t.out == t.grad)) r.add(t.grad, gb, false);
    if (use & USE_OUT) r.add(t.out, gb, true);
    if (use & USE_W_M) {
      r.add(t.W, sb, true);
      r.add(t.m, sb, true);
    }
    if (use & USE_V) r.add(t.v, sb, true);
  }
  return r.clash() ? FORGE_ERR_ALIAS : FORGE_OK;
}

forge_status check_clipped(const forge_tensor* tensors, int32_t count, const float* coef, int use) {
  if (!coef) return FORGE_ERR_NULL;
  if (forge_status s = check_list(tensors, count, use)) return s;
  if (!aligned4(coef)) return FORGE_ERR_ALIGN;
  return check_list_overlap(tensors, count, coef, use);
}

}  // namespace

// A launch takes at least 256 tensors and leaves at most 2048 float64 partial sums.
int64_t grad_norm_workspace(int32_t count) {
  if (count < 0 || count > FORGE_MAX_TENSORS) return 0;
  return std::max<int64_t>(16, (int64_t(count) + 255) / 256 * 2048 * 8);
}

forge_status validate_grad_norm(const forge_tensor* tensors, int32_t count, double max_norm,
                                const float* norm_coef, const void* workspace,
                                int64_t workspace_bytes) {
  if (!norm_coef || !workspace) return FORGE_ERR_NULL;
  if (forge_status s = check_list(tensors, count, 0)) return s;
  if (workspace_bytes < grad_norm_workspace(count)) return FORGE_ERR_SHAPE;
  if (!aligned4(norm_coef) || !aligned16(workspace)) return FORGE_ERR_ALIGN;
  const Span out{norm_coef, 8}, ws{workspace, uint64_t(workspace_bytes)};
  if (spans_overlap(out, ws)) return FORGE_ERR_ALIAS;
  for (int32_t i = 0; i < count; ++i) {
    const Span g{tensors[i].grad, uint64_t(tensors[i].n) * uint64_t(dtype_bytes(tensors[i].grad_dtype))};
    if (spans_overlap(out, g) || spans_overlap(ws, g)) return FORGE_ERR_ALIAS;
  }
  return std::isnan(max_norm) || max_norm < 0.0 ? FORGE_ERR_HPARAM : FORGE_OK;
}

forge_status validate_clip_grads(const forge_tensor* tensors, int32_t count, const float* coef) {
  return check_clipped(tensors, count, coef, USE_OUT);
}

forge_status validate_adamw_clipped(const forge_tensor* tensors, int32_t count, const float* coef,
                                    const forge_adamw_params* p) {
  if (!p) return FORGE_ERR_NULL;
  if (forge_status s = check_clipped(tensors, count, coef, USE_W_M | USE_V)) return s;
  return check_adamw_params(p);
}

forge_status validate_sgdm_clipped(const forge_tensor* tensors, int32_t count, const float* coef,
                                   const forge_sgdm_params* p) {
  if (!p) return FORGE_ERR_NULL;
  if (forge_status s = check_clipped(tensors, count, coef, USE_W_M)) return s;
  return check_sgdm_params(p);
}

bool embedding_sizes_ok(int64_t T, int64_t V, int64_t d) {
  return T >= 0 && T <= kMaxTokens && V >= 0 && V <= kMaxDim && d >= 0 && d <= kMaxDim;
}

// Two copies of (key, position) for the sort's passes, its digit counts (512
// for each tile of 1024 tokens, and in all), the rows' bounds, and the sums of chunks of
// tokens.
EmbeddingWorkspace embedding_workspace(int64_t T, int64_t V, int64_t d) {
  EmbeddingWorkspace w{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  for (int k = 0; k < 2; ++k) {
    w.keys[k] = take(4 * T);
    w.pos[k] = take(4 * T);
  }
  w.count = take(((T + 1023) / 1024 + 1) * 512 * 4);
  w.bound = take(4 * (V + 1));
  w.chunk = take((T >> embedding_chunk_bits(T)) * d * 4);
  w.bytes = at;
  return w;
}

namespace {

bool ids_ok(int32_t id_bytes) { return id_bytes == 4 || id_bytes == 8; }
bool aligned_ids(const void* p, int32_t id_bytes) {
  return (reinterpret_cast<uintptr_t>(p) & uintptr_t(id_bytes - 1)) == 0;
}
bool finite_scale(double scale) { return std::isfinite(scale) && std::isfinite(float(scale)); }

}  // namespace

forge_status validate_embedding(const void* table, forge_dtype table_dtype, const void* ids,
                                int32_t id_bytes, const void* out, forge_dtype out_dtype,
                                int64_t T, int64_t V, int64_t d, double scale) {
  const int tb = dtype_bytes(table_dtype), ob = dtype_bytes(out_dtype);
  if (tb == 0 || ob == 0 || !ids_ok(id_bytes)) return FORGE_ERR_DTYPE;
  if (T > 0 && d > 0 && (!ids || !out || (V > 0 && !table))) return FORGE_ERR_NULL;
  if (!embedding_sizes_ok(T, V, d)) return FORGE_ERR_SHAPE;
  if (T > 0 && d > 0) {
    if (d % 8 != 0 || !aligned16(out) || !aligned_ids(ids, id_bytes) || (V > 0 && !aligned16(table)))
      return FORGE_ERR_ALIGN;
    const Span so{out, uint64_t(T) * uint64_t(d) * uint64_t(ob)};
    if (spans_overlap(so, Span{ids, uint64_t(T) * uint64_t(id_bytes)}) ||
        spans_overlap(so, Span{table, uint64_t(V) * uint64_t(d) * uint64_t(tb)}))
      return FORGE_ERR_ALIAS;
  }
  return finite_scale(scale) ? FORGE_OK : FORGE_ERR_HPARAM;
}

forge_status validate_embedding_grad(const void* ids, int32_t id_bytes, const void* dY,
                                     forge_dtype dY_dtype, const void* const* outs, int n_outs,
                                     int64_t T, int64_t V, int64_t d, double scale,
                                     const void* workspace, int64_t workspace_bytes) {
  const int yb = dtype_bytes(dY_dtype);
  if (yb == 0 || !ids_ok(id_bytes)) return FORGE_ERR_DTYPE;
  const bool work = V > 0 && d > 0;
  if (work) {
    if (!workspace || (T > 0 && (!ids || !dY))) return FORGE_ERR_NULL;
    for (int k = 0; k < n_outs; ++k)
      if (!outs[k]) return FORGE_ERR_NULL;
  }
  if (!embedding_sizes_ok(T, V, d)) return FORGE_ERR_SHAPE;
  if (work) {
    if (workspace_bytes < embedding_workspace(T, V, d).bytes) return FORGE_ERR_SHAPE;
    if (d % 8 != 0 || !aligned16(workspace)) return FORGE_ERR_ALIGN;
    if (T > 0 && (!aligned_ids(ids, id_bytes) || !aligned16(dY))) return FORGE_ERR_ALIGN;
    Span spans[6] = {};
    int n = 0;
    for (int k = 0; k < n_outs; ++k) {
      if (!aligned16(outs[k])) return FORGE_ERR_ALIGN;
      spans[n++] = Span{outs[k], uint64_t(V) * uint64_t(d) * 4u};
    }
    spans[n++] = Span{workspace, uint64_t(workspace_bytes)};
    const int written = n;
    spans[n++] = Span{ids, uint64_t(T) * uint64_t(id_bytes)};
    spans[n++] = Span{dY, uint64_t(T) * uint64_t(d) * uint64_t(yb)};
    for (int k = 0; k < written; ++k)
      for (int j = k + 1; j < n; ++j)
        if (spans_overlap(spans[k], spans[j])) return FORGE_ERR_ALIAS;
  }
  return finite_scale(scale) ? FORGE_OK : FORGE_ERR_HPARAM;
}

namespace {

Span codes_span(const void* p, int64_t R, int64_t Kp) { return Span{p, uint64_t(R) * uint64_t(Kp / 2)}; }
Span scales_span(const void* p, int64_t R, int64_t Kp) { return Span{p, uint64_t(R) * uint64_t(Kp / 32)}; }

// The product of operands I (N rows) and O (M rows) into the outputs [M, N].
forge_status check_product(const void* i_codes, const void* i_scales, const void* o_codes,
                           const void* o_scales, const void* const* outs, const int* elem_bytes,
                           int n_outs, int64_t N, int64_t M, int64_t Kp) {
  if (M < 0 || N < 0 || Kp < 0) return FORGE_ERR_SHAPE;
  const bool work = M > 0 && N > 0;
  const void* const in[4] = {i_codes, i_scales, o_codes, o_scales};
  if (work) {
    for (int k = 0; k < n_outs; ++k)
      if (!outs[k]) return FORGE_ERR_NULL;
    for (const void* p : in)
      if (Kp > 0 && !p) return FORGE_ERR_NULL;
  }
  if (M > kMaxDim || N > kMaxDim || Kp > FORGE_MXFP4_MAX_K || M * N > kMaxElems) return FORGE_ERR_SHAPE;
  if (!work) return FORGE_OK;
  if (N % 8 != 0 || Kp % 128 != 0) return FORGE_ERR_ALIGN;
  Span spans[7] = {};
  int n = 0;
  for (int k = 0; k < n_outs; ++k) {
    if (!aligned16(outs[k])) return FORGE_ERR_ALIGN;
    spans[n++] = Span{outs[k], uint64_t(M) * uint64_t(N) * uint64_t(elem_bytes[k])};
  }
  if (Kp > 0)
    for (const void* p : in)
      if (!aligned16(p)) return FORGE_ERR_ALIGN;
  spans[n++] = codes_span(i_codes, N, Kp);
  spans[n++] = scales_span(i_scales, N, Kp);
  spans[n++] = codes_span(o_codes, M, Kp);
  spans[n++] = scales_span(o_scales, M, Kp);
  for (int k = 0; k < n_outs; ++k)
    for (int j = k + 1; j < n; ++j)
      if (spans_overlap(spans[k], spans[j])) return FORGE_ERR_ALIAS;
  return FORGE_OK;
}

}  // namespace

forge_status validate_quantize_mxfp4(const void* x, forge_dtype x_dtype, int64_t R, int64_t C,
                                     const void* row_codes, const void* row_scales,
                                     const void* col_codes, const void* col_scales) {
  const int xb = dtype_bytes(x_dtype);
  if (xb == 0) return FORGE_ERR_DTYPE;
  if (!row_codes != !row_scales || !col_codes != !col_scales || (!row_codes && !col_codes))
    return FORGE_ERR_NULL;
  if (R > 0 && C > 0 && !x) return FORGE_ERR_NULL;
  if (R < 0 || C < 0 || R > kMaxTokens || C > kMaxTokens) return FORGE_ERR_SHAPE;
  if ((row_codes && (C > FORGE_MXFP4_MAX_K || R > kMaxDim)) ||
      (col_codes && (R > FORGE_MXFP4_MAX_K || C > kMaxDim)))
    return FORGE_ERR_SHAPE;
  if (R == 0 || C == 0) return FORGE_OK;
  if (C % 8 != 0 || !aligned16(x)) return FORGE_ERR_ALIGN;
  Span spans[5] = {};
  int n = 0;
  if (row_codes) {
    if (!aligned16(row_codes) || !aligned16(row_scales)) return FORGE_ERR_ALIGN;
    spans[n++] = codes_span(row_codes, R, FORGE_MXFP4_K(C));
    spans[n++] = scales_span(row_scales, R, FORGE_MXFP4_K(C));
  }
  if (col_codes) {
    if (!aligned16(col_codes) || !aligned16(col_scales)) return FORGE_ERR_ALIGN;
    spans[n++] = codes_span(col_codes, C, FORGE_MXFP4_K(R));
    spans[n++] = scales_span(col_scales, C, FORGE_MXFP4_K(R));
  }
  const int written = n;
  spans[n++] = Span{x, uint64_t(R) * uint64_t(C) * uint64_t(xb)};
  for (int k = 0; k < written; ++k)
    for (int j = k + 1; j < n; ++j)
      if (spans_overlap(spans[k], spans[j])) return FORGE_ERR_ALIAS;
  return FORGE_OK;
}

forge_status validate_matmul_mxfp4(const void* a_codes, const void* a_scales, const void* b_codes,
                                   const void* b_scales, const void* out, forge_dtype out_dtype,
                                   int64_t M, int64_t N, int64_t Kp, forge_tile tile) {
  const int ob[1] = {dtype_bytes(out_dtype)};
  if (ob[0] == 0) return FORGE_ERR_DTYPE;
  const void* outs[1] = {out};
  if (forge_status s = check_product(b_codes, b_scales, a_codes, a_scales, outs, ob, 1, N, M, Kp))
    return s;
  return check_tile(tile);
}

forge_status validate_wgrad_adamw_mxfp4(const void* x_codes, const void* x_scales,
                                        const void* dy_codes, const void* dy_scales,
                                        const float* W, const float* m, const float* v, int64_t Kp,
                                        int64_t d_in, int64_t d_out, const forge_adamw_params* p,
                                        forge_tile tile) {
  const int four[3] = {4, 4, 4};
  const void* outs[3] = {W, m, v};
  if (!p) return FORGE_ERR_NULL;
  if (forge_status s = check_product(x_codes, x_scales, dy_codes, dy_scales, outs, four, 3, d_in,
                                     d_out, Kp))
    return s;
  if (forge_status s = check_adamw_params(p)) return s;
  return check_tile(tile);
}

}  // namespace forge
