// layer_ops.cu — C ABI of the operators around the attention (declared in
// include/sol_attn.h): argument checks in front of the launches.  They hold no workspace: every call reads its inputs
// and writes its outputs only, so calls on several streams, devices or
// captured graphs do not meet.
#include <algorithm>
#include <climits>
#include <cmath>
#include <numeric>

#include "host.h"
#include "layer_launch.h"

using namespace solattn;

namespace {

constexpr int kMaxC = 16384;
constexpr int kMaxLinearK = 131071;   // 128 * 128 * K < 2^31

size_t dtype_size(int dtype) { return dtype == SOL_ATTN_FP32 ? 4 : 2; }

bool dtype_ok(int dtype) { return dtype == SOL_ATTN_BF16 || dtype == SOL_ATTN_FP16 || dtype == SOL_ATTN_FP32; }

int sm_count(int dev, int* n) {
  static int cached[kMaxDevices] = {0};
  if (!cached[dev]) CUDA_TRY(cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev));
  *n = cached[dev];
  return SOL_ATTN_OK;
}

// The current device, checked, and its number of SMs.
int device(int* dev, int* sms) {
  int rc;
  if ((rc = current_device(dev)) || (rc = check_arch(*dev))) return rc;
  return sm_count(*dev, sms);
}

// Rows [B, L] of `width` elements of `size` bytes.
struct Span {
  const char* p;
  long long sb, sl;   // bytes
  int B, L;
  long long width;    // bytes
  const char* end() const { return p + (B - 1) * sb + (L - 1) * sl + width; }
};

Span span(const void* p, size_t size, long long sb, long long sl, int B, int L, long long width) {
  const long long s = static_cast<long long>(size);
  return Span{static_cast<const char*>(p), B > 1 ? sb * s : 0, L > 1 ? sl * s : 0, B, L, width * s};
}

// Whether two sets of rows share a byte.  Where all of their strides are
// multiples of one pitch and the columns lie side by side within it, they do not
// (two slices of one buffer); any other two whose address ranges meet are taken
// to.
bool overlap(const Span& a, const Span& b) {
  if (a.end() <= b.p || b.end() <= a.p) return false;
  long long pitch = 0;
  for (long long s : {a.sb, a.sl, b.sb, b.sl})
    if (s && (!pitch || s < pitch)) pitch = s;
  if (!pitch || a.sb % pitch || a.sl % pitch || b.sb % pitch || b.sl % pitch) return true;
  const long long d = ((b.p - a.p) % pitch + pitch) % pitch;
  return d < a.width || d + b.width > pitch;
}

// Rows that are written: distinct rows may not share elements.
bool rows_distinct(const Span& s) {
  if (s.L > 1 && s.sl < s.width) return false;
  return s.B <= 1 || s.sb >= (s.L - 1) * s.sl + s.width ||
         (s.sb >= s.width && s.sl >= (s.B - 1) * s.sb + s.width);
}

bool aligned(size_t to, const void* p, size_t size, std::initializer_list<long long> strides) {
  if (reinterpret_cast<uintptr_t>(p) % to) return false;
  for (long long s : strides)
    if (s * static_cast<long long>(size) % static_cast<long long>(to)) return false;
  return true;
}
bool vec16(const void* p, size_t size, std::initializer_list<long long> strides) { return aligned(16, p, size, strides); }
// Eight elements at a time: 16 bytes, or 32 of fp32.
bool vec8(const void* p, size_t size, std::initializer_list<long long> strides) { return aligned(8 * size, p, size, strides); }

int check_rows(const sol_attn_rows& r, const char* name, int B, int L) {
  if (!dtype_ok(r.dtype)) return fail(SOL_ATTN_ERR_ARG, "%s: unknown dtype %d", name, r.dtype);
  if (reinterpret_cast<uintptr_t>(r.data) % dtype_size(r.dtype))
    return fail(SOL_ATTN_ERR_ALIGN, "%s is not aligned to its elements", name);
  if ((B > 1 && r.stride_b < 0) || (L > 1 && r.stride_l < 0))
    return fail(SOL_ATTN_ERR_ARG, "%s has a negative stride", name);
  return SOL_ATTN_OK;
}

int convert(const sol_attn_vectors& v, const char* name, int B, int L, Vectors* out, bool* vec) {
  *out = Vectors{};
  if (!v.data) return SOL_ATTN_OK;
  if (!dtype_ok(v.dtype)) return fail(SOL_ATTN_ERR_ARG, "%s: unknown dtype %d", name, v.dtype);
  if (v.groups < 1 || L % v.groups)
    return fail(SOL_ATTN_ERR_ARG, "%s: %d groups do not divide %d tokens", name, v.groups, L);
  const size_t size = dtype_size(v.dtype);
  if (reinterpret_cast<uintptr_t>(v.data) % size)
    return fail(SOL_ATTN_ERR_ALIGN, "%s is not aligned to its elements", name);
  if ((B > 1 && v.stride_b < 0) || (v.groups > 1 && v.stride_g < 0))
    return fail(SOL_ATTN_ERR_ARG, "%s has a negative stride", name);
  out->p = v.data;
  out->dtype = v.dtype;
  out->sb = B > 1 ? v.stride_b : 0;
  out->sg = v.groups > 1 ? v.stride_g : 0;
  out->per = L / v.groups;
  *vec = *vec && vec16(v.data, size, {out->sb, out->sg});
  return SOL_ATTN_OK;
}

}  // namespace

extern "C" {

int sol_attn_norm_modulate(const sol_attn_norm_args* a, void* stream) {
  if (!a) return fail(SOL_ATTN_ERR_ARG, "args is NULL");
  const int B = a->B, L = a->L, C = a->C;
  int rc;
  if (B < 0 || L < 0 || C < 1) return fail(SOL_ATTN_ERR_ARG, "bad sizes B = %d, L = %d, C = %d", B, L, C);
  if (C > kMaxC) return fail(SOL_ATTN_ERR_UNSUPPORTED, "C = %d exceeds the supported maximum %d", C, kMaxC);
  if (a->norm < 0 || a->norm > 2 || a->post_norm < 0 || a->post_norm > 2)
    return fail(SOL_ATTN_ERR_ARG, "unknown norm %d or %d", a->norm, a->post_norm);
  if (!(a->eps >= 0.f) || !(a->post_eps >= 0.f)) return fail(SOL_ATTN_ERR_ARG, "eps must not be negative or NaN");
  if (B == 0 || L == 0) return SOL_ATTN_OK;
  if (static_cast<long long>(B) * L > INT_MAX) return fail(SOL_ATTN_ERR_UNSUPPORTED, "B*L exceeds 2^31 - 1");
  if (!a->x.data) return fail(SOL_ATTN_ERR_ARG, "x is NULL");
  if (!a->h.data && !a->q && !(a->x_out.data && a->y.data))
    return fail(SOL_ATTN_ERR_ARG, "no output is asked for (x_out needs y)");
  if (a->x_out.data && !a->y.data) return fail(SOL_ATTN_ERR_ARG, "x_out needs y");
  if (a->x_inner < 1 || C % a->x_inner) return fail(SOL_ATTN_ERR_ARG, "x_inner %d does not divide C", a->x_inner);
  if ((a->q == nullptr) != (a->q_scale == nullptr)) return fail(SOL_ATTN_ERR_ARG, "q and q_scale come together");

  NormParams p{};
  p.B = B, p.L = L, p.C = C;
  if ((rc = check_rows(a->x, "x", B, L))) return rc;
  const size_t xs = dtype_size(a->x.dtype);
  int ydt = a->x.dtype;   // type of y and h
  if (a->y.data) {
    if ((rc = check_rows(a->y, "y", B, L))) return rc;
    ydt = a->y.dtype;
    if (a->h.data && a->h.dtype != ydt) return fail(SOL_ATTN_ERR_UNSUPPORTED, "h must have the type of y");
  } else if (a->h.data) {
    ydt = a->h.dtype;
  }
  if (ydt != a->x.dtype && a->x.dtype != SOL_ATTN_FP32)
    return fail(SOL_ATTN_ERR_UNSUPPORTED, "y and h must have the type of x, or x must be fp32");
  const size_t ys = dtype_size(ydt);
  p.x = a->x.data;
  p.x_sb = B > 1 ? a->x.stride_b : 0, p.x_sl = L > 1 ? a->x.stride_l : 0;
  p.x_inner = a->x_inner, p.x_sh = a->x_inner < C ? a->x_stride_h : 0;
  if (p.x_sh < 0) return fail(SOL_ATTN_ERR_ARG, "x has a negative stride");
  bool vec = C % 8 == 0 && p.x_inner % 8 == 0 && vec8(p.x, xs, {p.x_sb, p.x_sl, p.x_sh});
  const Span x = span(p.x, xs, p.x_sb, p.x_sl, B, L, (C / p.x_inner - 1) * p.x_sh + p.x_inner);
  Span y{}, outs[4];
  int nouts = 0;
  if (a->y.data) {
    p.y = a->y.data, p.y_sb = B > 1 ? a->y.stride_b : 0, p.y_sl = L > 1 ? a->y.stride_l : 0;
    vec = vec && vec8(p.y, ys, {p.y_sb, p.y_sl});
    y = span(p.y, ys, p.y_sb, p.y_sl, B, L, C);
  }
  if (a->x_out.data) {
    if ((rc = check_rows(a->x_out, "x_out", B, L))) return rc;
    if (a->x_out.dtype != a->x.dtype) return fail(SOL_ATTN_ERR_UNSUPPORTED, "x_out must have the type of x");
    p.xo = a->x_out.data, p.xo_sb = B > 1 ? a->x_out.stride_b : 0, p.xo_sl = L > 1 ? a->x_out.stride_l : 0;
    vec = vec && vec8(p.xo, xs, {p.xo_sb, p.xo_sl});
    const Span s = span(p.xo, xs, p.xo_sb, p.xo_sl, B, L, C);
    // in place: each row is read whole before it is written, by the same team
    const bool in_place = p.xo == p.x && p.xo_sb == p.x_sb && p.xo_sl == p.x_sl && p.x_inner == C;
    if (!rows_distinct(s)) return fail(SOL_ATTN_ERR_ARG, "rows of x_out share elements");
    if ((!in_place && overlap(s, x)) || overlap(s, y))
      return fail(SOL_ATTN_ERR_ARG, "x_out overlaps an input (only x_out = x is allowed)");
    outs[nouts++] = s;
  }
  if (a->h.data) {
    if ((rc = check_rows(a->h, "h", B, L))) return rc;
    p.h = a->h.data, p.h_sb = B > 1 ? a->h.stride_b : 0, p.h_sl = L > 1 ? a->h.stride_l : 0;
    vec = vec && vec8(p.h, ys, {p.h_sb, p.h_sl});
    outs[nouts++] = span(p.h, ys, p.h_sb, p.h_sl, B, L, C);
    if (!rows_distinct(outs[nouts - 1])) return fail(SOL_ATTN_ERR_ARG, "rows of h share elements");
    if (overlap(outs[nouts - 1], x) || (p.y && overlap(outs[nouts - 1], y)))
      return fail(SOL_ATTN_ERR_ARG, "h overlaps an input");
  }
  if (a->q) {
    if (a->q_stride < C) return fail(SOL_ATTN_ERR_ARG, "q_stride %lld is below C", a->q_stride);
    if (reinterpret_cast<uintptr_t>(a->q_scale) % 4) return fail(SOL_ATTN_ERR_ALIGN, "q_scale is misaligned");
    p.q = a->q, p.q_sl = a->q_stride, p.q_scale = a->q_scale;
    vec = vec && reinterpret_cast<uintptr_t>(p.q) % 8 == 0 && p.q_sl % 8 == 0;
    outs[nouts++] = span(p.q, 1, p.q_sl * L, p.q_sl, B, L, C);
    outs[nouts++] = span(p.q_scale, sizeof(float), 0, 0, 1, 1, static_cast<long long>(B) * L);
    for (int i = nouts - 2; i < nouts; ++i)
      if (overlap(outs[i], x) || (p.y && overlap(outs[i], y))) return fail(SOL_ATTN_ERR_ARG, "q or q_scale overlaps an input");
  }
  for (int i = 0; i < nouts; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return fail(SOL_ATTN_ERR_ARG, "two outputs overlap");
  if ((rc = convert(a->scale, "scale", B, L, &p.scale, &vec)) || (rc = convert(a->shift, "shift", B, L, &p.shift, &vec)) ||
      (rc = convert(a->gate, "gate", B, L, &p.gate, &vec)) || (rc = convert(a->weight, "weight", B, L, &p.weight, &vec)) ||
      (rc = convert(a->bias, "bias", B, L, &p.bias, &vec)) ||
      (rc = convert(a->post_weight, "post_weight", B, L, &p.post_weight, &vec)) ||
      (rc = convert(a->post_bias, "post_bias", B, L, &p.post_bias, &vec)))
    return rc;
  const sol_attn_vectors* vectors[7] = {&a->scale, &a->shift, &a->gate, &a->weight, &a->bias, &a->post_weight, &a->post_bias};
  for (const sol_attn_vectors* v : vectors) {
    if (!v->data) continue;
    const Span s = span(v->data, dtype_size(v->dtype), v->stride_b, v->stride_g, B, v->groups, C);
    for (int i = 0; i < nouts; ++i)
      if (overlap(outs[i], s)) return fail(SOL_ATTN_ERR_ARG, "an output overlaps a vector of parameters");
  }
  p.group = L;
  for (const Vectors* v : {&p.scale, &p.shift, &p.gate})
    if (v->p) p.group = std::gcd(p.group, v->per);
  p.channels = static_cast<float>(C), p.inv_channels = 1.f / p.channels;
  p.rs = a->residual_scale;
  p.pre = a->norm, p.post = a->post_norm;
  p.pre_eps = a->eps, p.post_eps = a->post_eps;

  // whether 32-byte vectors can read and write the rows of a 16-bit type
  const bool wide = p.x_inner % 16 == 0 && aligned(32, p.x, xs, {p.x_sb, p.x_sl, p.x_sh}) && aligned(32, p.y, ys, {p.y_sb, p.y_sl}) &&
                    aligned(32, p.xo, xs, {p.xo_sb, p.xo_sl}) && aligned(32, p.h, ys, {p.h_sb, p.h_sl}) &&
                    aligned(16, p.q, 1, {p.q_sl});
  int dev, sms;
  if ((rc = device(&dev, &sms))) return rc;
  auto st = static_cast<cudaStream_t>(stream);
  LaunchNorm* const launch = a->x.dtype == SOL_ATTN_BF16   ? launch_norm_bf16
                             : a->x.dtype == SOL_ATTN_FP16 ? launch_norm_fp16
                             : ydt == SOL_ATTN_BF16        ? launch_norm_fp32_bf16
                             : ydt == SOL_ATTN_FP16        ? launch_norm_fp32_fp16
                                                           : launch_norm_fp32;
  return launch(p, vec, wide, dev, sms, st);
}

int sol_attn_rope(const sol_attn_rope_args* a, void* stream) {
  if (!a) return fail(SOL_ATTN_ERR_ARG, "args is NULL");
  const int B = a->B, L = a->L, H = a->H, d = a->d;
  int rc;
  if (B < 0 || L < 0 || H < 1 || d < 1) return fail(SOL_ATTN_ERR_ARG, "bad sizes B = %d, L = %d, H = %d, d = %d", B, L, H, d);
  if (d % 16 || d > kRopeMaxD) return fail(SOL_ATTN_ERR_UNSUPPORTED, "d must be a multiple of 16 up to 256 (got %d)", d);
  if (static_cast<long long>(H) * d > kMaxC)
    return fail(SOL_ATTN_ERR_UNSUPPORTED, "H*d = %lld exceeds the supported maximum %d", static_cast<long long>(H) * d, kMaxC);
  if (!dtype_ok(a->dtype)) return fail(SOL_ATTN_ERR_ARG, "unknown dtype %d", a->dtype);
  if (a->norm < 0 || a->norm > 2) return fail(SOL_ATTN_ERR_ARG, "unknown norm %d", a->norm);
  if (!(a->eps >= 0.f)) return fail(SOL_ATTN_ERR_ARG, "eps must not be negative or NaN");
  if (a->pairing != SOL_ATTN_PAIR_INTERLEAVED && a->pairing != SOL_ATTN_PAIR_HALF)
    return fail(SOL_ATTN_ERR_ARG, "unknown pairing %d", a->pairing);
  if (!a->freqs || !a->axis) return fail(SOL_ATTN_ERR_ARG, "freqs or axis is NULL");
  if (a->axes < 1 || a->axes > kRopeMaxAxes) return fail(SOL_ATTN_ERR_UNSUPPORTED, "%d axes (1 to %d)", a->axes, kRopeMaxAxes);
  RopeParams p{};
  for (int i = 0; i < d / 2; ++i) {
    if (!std::isfinite(a->freqs[i])) return fail(SOL_ATTN_ERR_ARG, "frequency %d is not finite", i);
    if (a->axis[i] >= a->axes) return fail(SOL_ATTN_ERR_ARG, "pair %d is on axis %d of %d", i, a->axis[i], a->axes);
    p.turns[i] = a->freqs[i] / 6.283185307179586476925286766559;
    p.axis[i] = a->axis[i];
  }
  if (a->pos_kind == SOL_ATTN_POS_GRID) {
    const long long f = a->grid_f, h = a->grid_h, w = a->grid_w;
    if (a->axes != 3) return fail(SOL_ATTN_ERR_ARG, "a grid has 3 axes");
    if (f < 1 || h < 1 || w < 1 || f > INT_MAX / h || f * h > INT_MAX / w)
      return fail(SOL_ATTN_ERR_ARG, "bad grid %lld x %lld x %lld", f, h, w);
    if (a->start < 0) return fail(SOL_ATTN_ERR_ARG, "start is negative");
    p.grid_h = a->grid_h, p.grid_w = a->grid_w, p.grid_tokens = f * h * w, p.start = a->start;
  } else {
    if (a->pos_kind < SOL_ATTN_POS_GRID || a->pos_kind > SOL_ATTN_POS_F64)
      return fail(SOL_ATTN_ERR_ARG, "unknown kind of positions %d", a->pos_kind);
    p.pos = a->positions;
    p.pos_sb = B > 1 ? a->pos_stride_b : 0, p.pos_sl = L > 1 ? a->pos_stride_l : 0, p.pos_sa = a->axes > 1 ? a->pos_stride_a : 0;
    if (p.pos_sb < 0 || p.pos_sl < 0 || p.pos_sa < 0) return fail(SOL_ATTN_ERR_ARG, "positions has a negative stride");
  }
  p.pos_kind = a->pos_kind;
  if (B == 0 || L == 0) return SOL_ATTN_OK;
  if (static_cast<long long>(B) * L > INT_MAX) return fail(SOL_ATTN_ERR_UNSUPPORTED, "B*L exceeds 2^31 - 1");
  if (p.pos_kind != kPosGrid) {
    const size_t s = p.pos_kind == kPosI32 || p.pos_kind == kPosF32 ? 4 : 8;
    if (!p.pos) return fail(SOL_ATTN_ERR_ARG, "positions is NULL");
    if (reinterpret_cast<uintptr_t>(p.pos) % s) return fail(SOL_ATTN_ERR_ALIGN, "positions is not aligned to its elements");
  }
  p.B = B, p.L = L, p.H = H, p.d = d;
  p.norm = a->norm, p.eps = a->eps;
  p.inv_channels = 1.f / static_cast<float>(p.norm == kRopeNormToken ? H * d : d);
  p.half = a->pairing == SOL_ATTN_PAIR_HALF;
  const size_t size = dtype_size(a->dtype);
  const long long n = static_cast<long long>(B) * H * L * d;
  const sol_attn_rope_tensor* in[3] = {&a->q, &a->k, &a->v};
  RopeTensor* out[3] = {&p.q, &p.k, &p.v};
  const char* names[3] = {"q", "k", "v"};
  for (int i = 0; i < 3; ++i) {
    const sol_attn_rope_tensor& t = *in[i];
    if (i == 2 && !t.in && !t.out) continue;
    if ((rc = check_ptr(t.in, names[i])) || (rc = check_ptr(t.out, names[i]))) return rc;
    RopeTensor& r = *out[i];
    r.in = t.in, r.out = t.out;
    r.sb = B > 1 ? t.stride_b : 0, r.sl = L > 1 ? t.stride_l : 0, r.sh = H > 1 ? t.stride_h : 0;
    if (r.sb < 0 || r.sl < 0 || r.sh < 0) return fail(SOL_ATTN_ERR_ARG, "%s has a negative stride", names[i]);
    if (!vec8(t.in, size, {r.sb, r.sl, r.sh}) || !vec8(t.out, size, {}))
      return fail(SOL_ATTN_ERR_ALIGN, "%s: base and strides must be multiples of 8 elements", names[i]);
    if (i < 2 && t.weight) {
      if (a->norm == kRopeNormNone) return fail(SOL_ATTN_ERR_ARG, "%s has a weight but no norm", names[i]);
      if (!dtype_ok(t.weight_dtype)) return fail(SOL_ATTN_ERR_ARG, "%s weight: unknown dtype %d", names[i], t.weight_dtype);
      if (reinterpret_cast<uintptr_t>(t.weight) % 16) return fail(SOL_ATTN_ERR_ALIGN, "%s weight is not 16-byte aligned", names[i]);
      r.weight = t.weight, r.weight_dtype = t.weight_dtype;
    }
  }
  const int tensors = p.v.in ? 3 : 2;
  p.packed = 1;
  for (int i = 0; i < tensors; ++i) p.packed = p.packed && (out[i]->sh == d || H == 1);
  // a head's place in the output is kept in 32 bits, by 8 elements
  if (static_cast<long long>(H) * d / 8 * L > UINT_MAX)
    return fail(SOL_ATTN_ERR_UNSUPPORTED, "H*L*d = %lld exceeds 2^35", static_cast<long long>(H) * d * L);
  for (int i = 0; i < tensors; ++i) {
    const char* o = static_cast<const char*>(out[i]->out);
    const char* o_end = o + n * static_cast<long long>(size);
    for (int j = 0; j < tensors; ++j) {
      const RopeTensor& t = *out[j];
      const char* x = static_cast<const char*>(t.in);
      const char* x_end = x + ((B - 1) * t.sb + (L - 1) * t.sl + (H - 1) * t.sh + d) * static_cast<long long>(size);
      if (o < x_end && x < o_end) return fail(SOL_ATTN_ERR_ARG, "an output overlaps an input tensor");
      const char* o2 = static_cast<const char*>(t.out);
      if (j != i && o < o2 + n * static_cast<long long>(size) && o2 < o_end)
        return fail(SOL_ATTN_ERR_ARG, "two outputs overlap");
    }
  }
  for (int i = 0; i < tensors; ++i) {
    const Span o = span(out[i]->out, size, 0, 0, 1, 1, n);
    for (int j = 0; j < 2; ++j)
      if (out[j]->weight &&
          overlap(o, span(out[j]->weight, dtype_size(out[j]->weight_dtype), 0, 0, 1, 1, p.norm == kRopeNormToken ? H * d : d)))
        return fail(SOL_ATTN_ERR_ARG, "an output overlaps a weight");
    if (p.pos && overlap(o, span(p.pos, p.pos_kind == kPosI32 || p.pos_kind == kPosF32 ? 4 : 8, 0, 0, 1, 1,
                                 (B - 1) * p.pos_sb + (L - 1) * p.pos_sl + (a->axes - 1) * p.pos_sa + 1)))
      return fail(SOL_ATTN_ERR_ARG, "an output overlaps the positions");
  }
  int dev, sms;
  if ((rc = device(&dev, &sms))) return rc;
  auto st = static_cast<cudaStream_t>(stream);
  return launch_rope(p, a->dtype, dev, sms, st);
}

int sol_attn_quantized_linear(const sol_attn_linear_args* a, void* stream) {
  if (!a) return fail(SOL_ATTN_ERR_ARG, "args is NULL");
  const int M = a->M, N = a->N, K = a->K;
  int rc;
  if (M < 0 || N < 0 || K < 1) return fail(SOL_ATTN_ERR_ARG, "bad sizes M = %d, N = %d, K = %d", M, N, K);
  if (M > INT_MAX - 512 || N > INT_MAX - 512) return fail(SOL_ATTN_ERR_UNSUPPORTED, "M = %d or N = %d is too large", M, N);
  if (a->flags & ~SOL_ATTN_FLAG_TEST_STALL) return fail(SOL_ATTN_ERR_ARG, "unknown flag bits 0x%x", a->flags);
  if (K > kMaxLinearK) return fail(SOL_ATTN_ERR_UNSUPPORTED, "K = %d exceeds %d, up to which the sums fit 32 bits", K, kMaxLinearK);
  if (!dtype_ok(a->out_dtype)) return fail(SOL_ATTN_ERR_ARG, "out: unknown dtype %d", a->out_dtype);
  if (M == 0 || N == 0) return SOL_ATTN_OK;
  if ((rc = check_ptr(a->a, "a")) || (rc = check_ptr(a->w, "w"))) return rc;
  if (!a->a_scale || !a->w_scale || !a->out) return fail(SOL_ATTN_ERR_ARG, "a_scale, w_scale or out is NULL");
  if ((M > 1 && a->a_stride < K) || (N > 1 && a->w_stride < K))
    return fail(SOL_ATTN_ERR_ARG, "a row pitch is below K");
  if ((M > 1 && a->a_stride % 16) || (N > 1 && a->w_stride % 16))
    return fail(SOL_ATTN_ERR_ALIGN, "the rows of a and w must start at multiples of 16 bytes");
  if (M > 1 && a->out_stride < N) return fail(SOL_ATTN_ERR_ARG, "out_stride is below N");
  const size_t size = dtype_size(a->out_dtype);
  if (reinterpret_cast<uintptr_t>(a->a_scale) % 4 || reinterpret_cast<uintptr_t>(a->w_scale) % 4 ||
      reinterpret_cast<uintptr_t>(a->out) % size)
    return fail(SOL_ATTN_ERR_ALIGN, "a_scale, w_scale or out is not aligned to its elements");
  LinearParams p{};
  p.M = M, p.N = N, p.K = K;
  p.a_scale = a->a_scale, p.w_scale = a->w_scale;
  p.stall = (a->flags & SOL_ATTN_FLAG_TEST_STALL) != 0;
  p.timeout_ns = p.stall ? 1000000ull : 2000000000ull;
  if (a->bias) {
    if (!dtype_ok(a->bias_dtype)) return fail(SOL_ATTN_ERR_ARG, "bias: unknown dtype %d", a->bias_dtype);
    if (reinterpret_cast<uintptr_t>(a->bias) % dtype_size(a->bias_dtype))
      return fail(SOL_ATTN_ERR_ALIGN, "bias is not aligned to its elements");
    p.bias = a->bias, p.bias_dtype = a->bias_dtype;
  }
  // a pitch that no row uses may be anything: the maps take one that fits
  const long long fit = (K + 15LL) / 16 * 16;
  LinearOperands o{a->a, M > 1 ? a->a_stride : fit, a->w, N > 1 ? a->w_stride : fit};
  p.out = a->out;
  p.out_pitch = M > 1 ? a->out_stride : (N + 7LL) / 8 * 8;
  const Span out = span(p.out, size, 0, p.out_pitch, 1, M, N);
  if (overlap(out, span(o.a, 1, 0, o.a_pitch, 1, M, K)) || overlap(out, span(o.w, 1, 0, o.w_pitch, 1, N, K)) ||
      overlap(out, span(p.a_scale, 4, 0, 0, 1, 1, M)) || overlap(out, span(p.w_scale, 4, 0, 0, 1, 1, N)) ||
      (p.bias && overlap(out, span(p.bias, dtype_size(p.bias_dtype), 0, 0, 1, 1, N))))
    return fail(SOL_ATTN_ERR_ARG, "out overlaps an input");
  int dev, sms;
  if ((rc = device(&dev, &sms))) return rc;
  auto st = static_cast<cudaStream_t>(stream);
  return launch_linear(p, o, a->out_dtype, dev, sms, st);
}

int sol_attn_linear_status(void* stream) {
  int dev, sms, rc;
  if ((rc = device(&dev, &sms))) return rc;
  unsigned h = 0;
  if ((rc = read_linear_status(static_cast<cudaStream_t>(stream), &h))) return rc;
  if (!h) return SOL_ATTN_OK;
  if (h & 1u) return fail(SOL_ATTN_ERR_TIMEOUT, "a bounded device wait of a product gave up (status 0x%x)", h);
  return fail(SOL_ATTN_ERR_DEVICE, "a product's shared memory is not aligned to its tiles (status 0x%x)", h);
}

}  // extern "C"
