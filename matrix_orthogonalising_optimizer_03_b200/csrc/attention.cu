// Softmax attention of packed sequences and its backward pass (muon_attention_t): host checks
// and C entry points.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attention.h"
#include "muon.h"
#include "validate.h"

namespace muon {
namespace {

// ------------------------------------------------------------------ host checks
// A BF16 tensor tokens x heads x head_dim as the checks see it (strides of axes of one
// element do not matter and are set to the smallest legal ones).
struct Span {
  const void* ptr;
  int64_t tokens, heads, dim, ld, head;
};

Span span_of(const muon_heads_t& t, int64_t tokens, int64_t heads, int64_t dim) {
  Span s{t.ptr, tokens, heads, dim, t.ld, t.head};
  if (heads == 1) s.head = dim;
  if (tokens <= 1) s.ld = heads * (s.head > dim ? s.head : dim);
  return s;
}

// Rows of one token side by side inside the token stride, or the tokens of one head side by
// side inside the head stride: no element has two addresses.
bool nested(const Span& s) {
  return (s.head >= s.dim && s.ld >= (s.heads - 1) * s.head + s.dim) ||
         (s.ld >= s.dim && s.head >= (s.tokens - 1) * s.ld + s.dim);
}

size_t extent(const Span& s) {
  return s.tokens < 1 ? 0 : static_cast<size_t>((s.tokens - 1) * s.ld + (s.heads - 1) * s.head + s.dim) * 2;
}

// Whether two tensors may share an address. Interleaved views of one buffer do not: with
// the same outer stride, the spans of one outer index lie side by side inside it.
bool may_overlap(const Span& x, const Span& y) {
  if (!ranges_overlap(x.ptr, extent(x), y.ptr, extent(y))) return false;
  const int64_t d0 = (reinterpret_cast<intptr_t>(y.ptr) - reinterpret_cast<intptr_t>(x.ptr)) / 2;
  auto beside = [&](int64_t outer_x, int64_t outer_y, int64_t inner_x, int64_t inner_y) {
    if (outer_x != outer_y) return false;
    const int64_t d = ((d0 % outer_x) + outer_x) % outer_x;
    return d >= inner_x && d + inner_y <= outer_x;
  };
  if (beside(x.ld, y.ld, (x.heads - 1) * x.head + x.dim, (y.heads - 1) * y.head + y.dim)) return false;
  if (beside(x.head, y.head, (x.tokens - 1) * x.ld + x.dim, (y.tokens - 1) * y.ld + y.dim)) return false;
  return true;
}

}  // namespace

muon_status_t validate_attention(const muon_attention_t* p, bool backward) {
  if (p == nullptr) return MUON_ERR_INVALID_ARG;
  const muon_attention_t& a = *p;
  const int64_t lim = int64_t(1) << 31;
  if (a.q_tokens < 0 || a.k_tokens < 0 || a.q_tokens > lim - 65536 || a.k_tokens > lim - 65536 ||
      a.n_seq < 1 || a.n_seq > (1 << 20) || a.heads < 1 || a.kv_heads < 1 || a.heads > 65535 ||
      a.heads % a.kv_heads != 0 || a.head_dim < 8 || a.head_dim > 128 || a.head_dim % 8 != 0)
    return MUON_ERR_SHAPE;
  if ((a.causal != 0 && a.causal != 1) || !std::isfinite(a.scale) || !(a.scale > 0.f))
    return MUON_ERR_INVALID_ARG;
  if (a.n_seq > 1 && (a.q_offsets == nullptr || a.k_offsets == nullptr)) return MUON_ERR_INVALID_ARG;
  // tensors: the first n_ptr are used; which of them are written
  const muon_heads_t* t[8] = {&a.q, &a.k, &a.v, &a.o, &a.dout, &a.dq, &a.dk, &a.dv};
  const bool on_keys[8] = {false, true, true, false, false, false, true, true};
  const bool written[8] = {false, false, false, !backward, false, true, true, true};
  const int nt = backward ? 8 : 4;
  Span s[8];
  for (int i = 0; i < nt; ++i) {
    const int64_t tokens = on_keys[i] ? a.k_tokens : a.q_tokens;
    s[i] = span_of(*t[i], tokens, on_keys[i] ? a.kv_heads : a.heads, a.head_dim);
    if (tokens == 0) continue;
    if (t[i]->ptr == nullptr || reinterpret_cast<uintptr_t>(t[i]->ptr) % 16) return MUON_ERR_INVALID_ARG;
    if (s[i].ld < 1 || s[i].head < 1 || s[i].ld >= (int64_t(1) << 38) || s[i].head >= (int64_t(1) << 38) ||
        s[i].ld % 8 || s[i].head % 8 || s[i].ld > (int64_t(1) << 44) / tokens || !nested(s[i]))
      return MUON_ERR_SHAPE;
  }
  struct Flat {
    const void* p;
    size_t n;
    bool w;
  };
  const size_t off_bytes = (static_cast<size_t>(a.n_seq) + 1) * 4;
  const Flat f[5] = {
      {a.lse, a.q_tokens > 0 ? static_cast<size_t>(a.heads) * a.q_tokens * 4 : 0, !backward},
      {a.s_max, a.s_max != nullptr && !backward ? static_cast<size_t>(a.heads) * 4 : 0, true},
      {a.q_offsets, a.q_offsets != nullptr ? off_bytes : 0, false},
      {a.k_offsets, a.k_offsets != nullptr ? off_bytes : 0, false},
      {a.status_dev, a.status_dev != nullptr ? size_t(4) : 0, true}};
  if (a.q_tokens > 0 && a.lse == nullptr) return MUON_ERR_INVALID_ARG;
  for (int i = 0; i < 5; ++i)
    if (reinterpret_cast<uintptr_t>(f[i].p) % 4) return MUON_ERR_INVALID_ARG;
  for (int i = 0; i < nt; ++i) {
    for (int j = 0; j < nt; ++j)
      if (i != j && written[i] && may_overlap(s[i], s[j])) return MUON_ERR_ALIAS;
    for (int j = 0; j < 5; ++j)
      if ((written[i] || f[j].w) && ranges_overlap(s[i].ptr, extent(s[i]), f[j].p, f[j].n)) return MUON_ERR_ALIAS;
  }
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if ((f[i].w || f[j].w) && ranges_overlap(f[i].p, f[i].n, f[j].p, f[j].n)) return MUON_ERR_ALIAS;
  return MUON_OK;
}

}  // namespace muon

extern "C" MUON_API muon_status_t muon_attention_forward(const muon_attention_t* a, void* stream) {
  using namespace muon;
  const muon_status_t v = validate_attention(a, false);
  if (v != MUON_OK || a->q_tokens == 0) return v;
  int dev = 0, sms = 0;
  const muon_status_t d = current_device(&dev, &sms);
  if (d != MUON_OK) return d;
  return launch_attention_forward(*a, dev, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" MUON_API size_t muon_attention_workspace_size(const muon_attention_t* a) {
  if (muon::validate_attention(a, true) != MUON_OK) return 0;
  return (static_cast<size_t>(a->heads) * a->q_tokens * 4 + 255) / 256 * 256;
}

extern "C" MUON_API muon_status_t muon_attention_backward(const muon_attention_t* a, void* workspace,
                                                          size_t ws_bytes, void* stream) {
  using namespace muon;
  const muon_status_t v = validate_attention(a, true);
  if (v != MUON_OK) return v;
  const size_t need = muon_attention_workspace_size(a);
  if (need > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 || ws_bytes < need))
    return MUON_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  const muon_status_t d = current_device(&dev, &sms);
  if (d != MUON_OK) return d;
  return launch_attention_backward(*a, static_cast<float*>(workspace), dev, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? MUON_OK : MUON_ERR_CUDA;
}
