// api_linear.cpp -- the C ABI of linear attention with a decay for each head (declared in include/sss.h):
// packed prompts, the single-token step on cache slots, and the gradients.
#include "sss.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "api_util.h"
#include "kernels.h"
#include "linear_attention.h"

using namespace sss;

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // token numbers are 32-bit on the device
constexpr int64_t kMaxHeads = (int64_t)1 << 16;
constexpr int64_t kMaxHeadDim = 256;
constexpr int64_t kMaxStride = (int64_t)1 << 24;      // between tokens
constexpr int64_t kMaxHeadStride = (int64_t)1 << 40;  // between heads
constexpr double kMaxThreads = 4294967295.0;  // of a launch

int64_t dtype_size(int t) { return t == SSS_BF16 ? 2 : 4; }
int status_of(hipError_t e) { return e == hipSuccess ? SSS_OK : SSS_ERR_HIP; }
size_t align(size_t v) { return (v + 255) / 256 * 256; }
int pad(int64_t n) { return n <= 64 ? 64 : n <= 128 ? 128 : 256; }

int dims_status(int64_t tokens, int64_t nseq, int64_t slots, int64_t heads, int64_t q_heads, int64_t k_heads, int64_t dk,
                int64_t dv) {
  if (tokens < 0 || nseq < 0 || slots < 0 || tokens > kMaxTokens || nseq > kMaxTokens || slots > kMaxTokens || heads < 1 ||
      heads > kMaxHeads || q_heads < 1 || k_heads < 1 || heads % q_heads != 0 || heads % k_heads != 0 || dk < 1 || dv < 1)
    return SSS_ERR_BAD_DIM;
  if (dk > kMaxHeadDim || dv > kMaxHeadDim) return SSS_ERR_UNSUPPORTED;
  if ((double)slots * (double)heads * (double)(dk * dv) > 1.0e18) return SSS_ERR_BAD_DIM;  // bytes in 64 bits
  return SSS_OK;
}

// Elements of (rows, heads, width): rows of any stride, heads of any other
struct Side {
  const void* p;
  int64_t st, sh, heads, width;
  bool ok(int64_t rows) const {
    return st >= 0 && sh >= 0 && st <= kMaxStride && sh <= kMaxHeadStride &&
           (double)rows * (double)st + (double)heads * (double)sh < 1.0e18;
  }
  int64_t bytes(int64_t rows, int64_t es) const {
    return rows < 1 ? 0 : ((rows - 1) * st + (heads - 1) * sh + width) * es;
  }
  LaSide on(int64_t all) const {
    LaSide s{};
    s.p = static_cast<const char*>(p);
    s.st = st;
    s.sh = sh;
    s.rep = (int)(all / heads);
    s.width = (int)width;
    return s;
  }
};

struct Plan {
  int nseg;
  int64_t K;
  size_t end, enter, begin, rend, renter, sum, rsum, flag, rflag;  // states at the segments' edges
  size_t rows, cols, cols2, within, edge, last, trace, gpart, dq, dk;      // gradients
  size_t total;
};

// Segments: one round of the workgroups that the GPU holds at a time, two per CU, one where a side of the states is above
// 128 (LDS); of the gradients' walks one round of dq and dk, and dv, where it is in their launch, follows into the places
// that dk leaves, half as long.  Each segment is of a tile of fp32 at least.  Measured, 8192 tokens where not said,
// prompts: 32768 x 16 heads of 128 x 128 248 us in 32 segments, one round, 291-355 in 16 or 12; 8 heads of
// 256 x 256 169 in 32, 208 in 16, 243 in 64; 8 of 128 x 256 85, 107 and 115.  Gradients: 16 heads of 64 x 64 93 us in 16,
// 128 in 10, 114 in 21, 98 in 32; 16 of 128 x 128 209 in 16, 225 in 10, 236 in 32, 384 in 4; 16 of 128 x 64 161 in 16,
// 233 in 10, 217 in 21; 8 of 128 x 256 236 in 16, 358 in 10, 258 in 32; 8 of 256 x 256 457 in 16, 545 in 10, 543 in
// 32; 1001 tokens x 6 heads of 64 x 50 in fp32 46 us in 32, 46 in 16, 57 in 8, 85 in 4.  The other way: gradients of 8 fp32
// heads of 128 x 128 288 in 32, 278 in 21; prompts of 300 heads of 64 x 64, for which a round is rounded down to one
// segment, 481, 372 in two.
Plan plan(int64_t tokens, int64_t nseq, int64_t heads, int64_t q_heads, int64_t k_heads, int64_t dk, int64_t dv, bool grads,
          int cus) {
  Plan p{};
  const int64_t walks = grads ? 2 : 1, per_cu = std::max(dk, dv) > 128 ? 1 : 2;
  const int64_t round = std::max<int64_t>(1, cus * per_cu / (walks * heads));
  int64_t S = std::min<int64_t>(round, (tokens + kLaTile / 2 - 1) / (kLaTile / 2));
  const int forced = env_int("SSS_FORCE_SEGMENTS", 0);
  if (forced > 0) S = std::min<int64_t>(forced, tokens);
  S = std::max<int64_t>(S, 1);
  int64_t K = (tokens + S - 1) / S;
  if (forced <= 0) K = (K + kLaTile / 2 - 1) / (kLaTile / 2) * (kLaTile / 2);
  p.K = std::max<int64_t>(1, K);
  p.nseg = (int)((tokens + p.K - 1) / p.K);
  size_t at = 0;
  auto take = [&](int64_t n) {
    const size_t here = at;
    at += align((size_t)n * 4);
    return here;
  };
  const int64_t states = p.nseg > 1 ? p.nseg * heads * dk * dv : 0;
  p.end = take(states);
  p.enter = take(states);
  p.sum = take(p.nseg * heads);
  p.flag = take(p.nseg);
  if (!grads) {
    p.begin = take(states);
  } else {
    p.rend = take(states);
    p.renter = take(states);
    p.rsum = take(p.nseg * heads);
    p.rflag = take(p.nseg);
    p.rows = take(tokens * heads);
    p.cols = take(tokens * heads);
    p.cols2 = take(tokens * heads);
    p.within = take(tokens * heads);
    p.edge = take(p.nseg * heads);
    p.last = take(nseq * heads);
    p.trace = take(p.nseg * heads);
    p.gpart = take(p.nseg * heads);
    p.dq = take(q_heads < heads ? tokens * heads * dk : 0);
    p.dk = take(k_heads < heads ? tokens * heads * dk : 0);
  }
  p.total = at;
  return p;
}

// workgroups of the walks have at most 512 threads, of the step 256
bool launch_ok(int64_t groups, int threads = 512) { return (double)groups * (double)threads <= kMaxThreads; }

struct Fwd {
  Side q, k, v;
  const float* g;
  int64_t g_st;
  const float* beta;
  int64_t beta_st;
  const float* D;
  float scale;
  int64_t heads, dk, dv;
  int dtype;
};

int check_inputs(const Fwd& f, int64_t rows, Regions& r) {
  if (f.dtype != SSS_F32 && f.dtype != SSS_BF16) return SSS_ERR_UNSUPPORTED;
  const int64_t es = dtype_size(f.dtype);
  for (const Side* s : {&f.q, &f.k, &f.v})
    if (!s->ok(rows)) return SSS_ERR_BAD_DIM;
  for (const int64_t st : {f.g_st, f.beta ? f.beta_st : f.heads})
    if (st != 0 && (st < f.heads || st > kMaxStride)) return SSS_ERR_BAD_DIM;
  if (f.beta && f.beta_st == 0) return SSS_ERR_BAD_DIM;
  r.in(f.q.p, f.q.bytes(rows, es), es);
  r.in(f.k.p, f.k.bytes(rows, es), es);
  r.in(f.v.p, f.v.bytes(rows, es), es);
  r.in(f.g, f.g_st == 0 ? f.heads * 4 : span(rows, f.g_st, f.heads, 4), 4);
  r.in(f.beta, span(rows, f.beta_st, f.heads, 4), 4);
  r.in(f.D, f.heads * 4, 4);
  return SSS_OK;
}

LaWalk walk_of(const Fwd& f, const Plan& p, int64_t tokens, int64_t nseq) {
  LaWalk w{};
  w.g = f.g;
  w.g_st = f.g_st;
  w.beta = f.beta;
  w.beta_st = f.beta_st;
  w.D = f.D;
  w.scale = f.scale;
  w.hs = f.dk * f.dv;
  w.tokens = (int)tokens;
  w.nseq = (int)nseq;
  w.H = (int)f.heads;
  w.K = (int)p.K;
  w.nseg = p.nseg;
  return w;
}

}  // namespace

extern "C" {

size_t linear_attention_packed_fwd_workspace_size(int64_t tokens, int64_t heads, int64_t dk, int64_t dv, int device) {
  if (dims_status(tokens, 0, 0, heads, heads, heads, dk, dv) != SSS_OK) return 0;
  int cus = device_cus(device);
  if (cus <= 0) cus = 256;
  const Plan p = plan(tokens, 0, heads, heads, heads, dk, dv, false, cus);
  return p.nseg > 1 ? p.total : 0;
}

int linear_attention_packed_fwd(const void* q, int64_t q_stride, int64_t q_head_stride, int64_t q_heads, const void* k,
                                int64_t k_stride, int64_t k_head_stride, int64_t k_heads, const void* v, int64_t v_stride,
                                int64_t v_head_stride, const float* log_decay, int64_t decay_stride, const float* beta,
                                int64_t beta_stride, const float* D_skip, float scale, float* state, const int32_t* cu_seqlens,
                                const int32_t* state_indices, const uint8_t* has_initial, void* out, int64_t tokens,
                                int64_t nseq, int64_t slots, int64_t heads, int64_t dk, int64_t dv, int io_dtype,
                                void* workspace, size_t workspace_bytes, sss_stream_t stream) {
  if (!q || !k || !v || !log_decay || !cu_seqlens || !out) return SSS_ERR_NULL_ARG;
  const int st = dims_status(tokens, nseq, slots, heads, q_heads, k_heads, dk, dv);
  if (st != SSS_OK) return st;
  if (state && (slots < 1 || (!state_indices && nseq > slots))) return SSS_ERR_BAD_DIM;
  const Fwd f{{q, q_stride, q_head_stride, q_heads, dk}, {k, k_stride, k_head_stride, k_heads, dk},
              {v, v_stride, v_head_stride, heads, dv}, log_decay, decay_stride, beta, beta_stride, D_skip, scale, heads, dk, dv,
              io_dtype};
  Regions r;
  const int in = check_inputs(f, tokens, r);
  if (in != SSS_OK) return in;
  const int64_t es = dtype_size(io_dtype);
  r.in(cu_seqlens, (nseq + 1) * 4, 4);
  r.in(state_indices, nseq * 4, 4);
  r.in(has_initial, nseq, 1);
  r.output(state, slots * heads * dk * dv * 4, 4);
  r.output(out, tokens * heads * dv * es, es);
  if (workspace && !aligned16(workspace)) return SSS_ERR_UNSUPPORTED;
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  if (tokens == 0 || nseq == 0) return SSS_OK;
  const int cus = current_device_cus();
  if (cus <= 0) return SSS_ERR_HIP;
  const Plan p = plan(tokens, nseq, heads, q_heads, k_heads, dk, dv, false, cus);
  if (!launch_ok(p.nseg * heads)) return SSS_ERR_BAD_DIM;
  if (p.nseg > 1) {
    if (workspace == nullptr || workspace_bytes < p.total) return SSS_ERR_WORKSPACE;
    r.output(workspace, (int64_t)p.total, 16);
    if (!r.ok()) return SSS_ERR_ALIAS;
  }
  if (env_int("SSS_LOG", 0))
    std::fprintf(stderr, "[sss] linear_attention_packed_fwd T=%lld seqs=%lld H=%lld %lldx%lld %s: segments=%d of %lld ws=%zu\n",
                 (long long)tokens, (long long)nseq, (long long)heads, (long long)dk, (long long)dv,
                 io_dtype == SSS_BF16 ? "bf16" : "f32", p.nseg, (long long)p.K, p.total);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool bf16 = io_dtype == SSS_BF16;
  char* const ws = static_cast<char*>(workspace);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  LaWalk w = walk_of(f, p, tokens, nseq);
  w.x = f.q.on(heads);
  w.y = f.k.on(heads);
  w.z = f.v.on(heads);
  w.out = static_cast<char*>(out);
  w.out_st = heads * dv;
  w.out_sh = dv;
  w.cu = cu_seqlens;
  w.sidx = state_indices;
  w.init = has_initial;
  w.state = state;
  w.slots = (int)slots;
  w.se = dv;
  w.sf = 1;
  if (p.nseg > 1) {
    w.end = at(p.end);
    w.begin = at(p.begin);
    w.enter = at(p.enter);
    w.sum = at(p.sum);
    w.flag = reinterpret_cast<int32_t*>(ws + p.flag);
    hipError_t e = la_launch(pad(dk), pad(dv), kLaFoldFwd, bf16, w, (unsigned)((p.nseg - 1) * heads), s);
    if (e == hipSuccess) e = la_carry({w.end, w.sum, w.flag, at(p.enter)}, nullptr, w.hs, (int)heads, p.nseg, s);
    if (e != hipSuccess) return SSS_ERR_HIP;
  }
  return status_of(la_launch(pad(dk), pad(dv), kLaFwd, bf16, w, (unsigned)(p.nseg * heads), s));
}

int linear_attention_update_slots(const void* q, int64_t q_stride, int64_t q_head_stride, int64_t q_heads, const void* k,
                                  int64_t k_stride, int64_t k_head_stride, int64_t k_heads, const void* v, int64_t v_stride,
                                  int64_t v_head_stride, const float* log_decay, int64_t decay_stride, const float* beta,
                                  int64_t beta_stride, const float* D_skip, float scale, float* state,
                                  const int32_t* state_indices, void* out, int64_t batch, int64_t slots, int64_t heads, int64_t dk,
                                  int64_t dv, int io_dtype, sss_stream_t stream) {
  if (!q || !k || !v || !log_decay || !state || !out) return SSS_ERR_NULL_ARG;
  const int st = dims_status(batch, 0, slots, heads, q_heads, k_heads, dk, dv);
  if (st != SSS_OK) return st;
  if (slots < 1 || (!state_indices && batch > slots)) return SSS_ERR_BAD_DIM;
  const Fwd f{{q, q_stride, q_head_stride, q_heads, dk}, {k, k_stride, k_head_stride, k_heads, dk},
              {v, v_stride, v_head_stride, heads, dv}, log_decay, decay_stride, beta, beta_stride, D_skip, scale, heads, dk, dv,
              io_dtype};
  Regions r;
  const int in = check_inputs(f, batch, r);
  if (in != SSS_OK) return in;
  const int64_t es = dtype_size(io_dtype);
  r.in(state_indices, batch * 4, 4);
  r.output(state, slots * heads * dk * dv * 4, 4);
  r.output(out, batch * heads * dv * es, es);
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  if (!launch_ok(batch * heads, 256)) return SSS_ERR_BAD_DIM;
  if (batch == 0) return SSS_OK;
  LaStep a{};
  a.q = f.q.on(heads);
  a.k = f.k.on(heads);
  a.v = f.v.on(heads);
  a.out = static_cast<char*>(out);
  a.g = log_decay;
  a.g_st = decay_stride;
  a.beta = beta;
  a.beta_st = beta_stride;
  a.D = D_skip;
  a.scale = scale;
  a.state = state;
  a.sidx = state_indices;
  a.rows = batch;
  a.slots = (int)slots;
  a.H = (int)heads;
  return status_of(la_step(a, io_dtype == SSS_BF16, reinterpret_cast<hipStream_t>(stream)));
}

size_t linear_attention_packed_bwd_workspace_size(int64_t tokens, int64_t nseq, int64_t heads, int64_t q_heads, int64_t k_heads,
                                                  int64_t dk, int64_t dv, int device) {
  if (dims_status(tokens, nseq, 0, heads, q_heads, k_heads, dk, dv) != SSS_OK) return 0;
  int cus = device_cus(device);
  if (cus <= 0) cus = 256;
  return plan(tokens, nseq, heads, q_heads, k_heads, dk, dv, true, cus).total;
}

int linear_attention_packed_bwd(const void* q, int64_t q_stride, int64_t q_head_stride, int64_t q_heads, const void* k,
                                int64_t k_stride, int64_t k_head_stride, int64_t k_heads, const void* v, int64_t v_stride,
                                int64_t v_head_stride, const float* log_decay, int64_t decay_stride, const float* beta,
                                int64_t beta_stride, const float* D_skip, float scale, const void* dout,
                                const int32_t* cu_seqlens, const float* initial_state, const float* dfinal_state, void* dq,
                                void* dk_out, void* dv_out, float* dlog_decay, float* dbeta, float* dD, float* dinitial_state,
                                int64_t tokens, int64_t nseq, int64_t heads, int64_t dk, int64_t dv, int io_dtype,
                                void* workspace, size_t workspace_bytes, sss_stream_t stream) {
  if (!cu_seqlens || (D_skip && !dD) || (decay_stride == 0 && (!log_decay || !dlog_decay)) ||
      (tokens != 0 && (!q || !k || !v || !log_decay || !dout || !dq || !dk_out || !dv_out || !dlog_decay || (beta && !dbeta))))
    return SSS_ERR_NULL_ARG;
  const int st = dims_status(tokens, nseq, 0, heads, q_heads, k_heads, dk, dv);
  if (st != SSS_OK) return st;
  const Fwd f{{q, q_stride, q_head_stride, q_heads, dk}, {k, k_stride, k_head_stride, k_heads, dk},
              {v, v_stride, v_head_stride, heads, dv}, log_decay, decay_stride, beta, beta_stride, D_skip, scale, heads, dk, dv,
              io_dtype};
  const Side d{dout, heads * dv, dv, heads, dv};
  Regions r;
  const int in = check_inputs(f, tokens, r);
  if (in != SSS_OK) return in;
  const int64_t es = dtype_size(io_dtype), states = nseq * heads * dk * dv * 4;
  if ((double)nseq * (double)heads * (double)(dk * dv) > 1.0e18) return SSS_ERR_BAD_DIM;
  r.in(dout, tokens * heads * dv * es, es);
  r.in(cu_seqlens, (nseq + 1) * 4, 4);
  r.in(initial_state, states, 4);
  r.in(dfinal_state, states, 4);
  r.output(dq, tokens * q_heads * dk * es, es);
  r.output(dk_out, tokens * k_heads * dk * es, es);
  r.output(dv_out, tokens * heads * dv * es, es);
  r.output(dlog_decay, (decay_stride == 0 ? 1 : tokens) * heads * 4, 4);
  r.output(beta ? dbeta : nullptr, tokens * heads * 4, 4);
  r.output(D_skip ? dD : nullptr, heads * 4, 4);
  r.output(dinitial_state, states, 4);
  if (workspace && !aligned16(workspace)) return SSS_ERR_UNSUPPORTED;
  if (!r.aligned) return SSS_ERR_UNSUPPORTED;
  if (!r.ok()) return SSS_ERR_ALIAS;
  const int cus = current_device_cus();
  if (cus <= 0) return SSS_ERR_HIP;
  const Plan p = plan(tokens, nseq, heads, q_heads, k_heads, dk, dv, true, cus);
  if (!launch_ok(3 * p.nseg * heads)) return SSS_ERR_BAD_DIM;
  if (p.total > 0) {
    if (workspace == nullptr || workspace_bytes < p.total) return SSS_ERR_WORKSPACE;
    r.output(workspace, (int64_t)p.total, 16);
    if (!r.ok()) return SSS_ERR_ALIAS;
  }
  if (env_int("SSS_LOG", 0))
    std::fprintf(stderr, "[sss] linear_attention_packed_bwd T=%lld seqs=%lld H=%lld %lldx%lld %s: segments=%d of %lld ws=%zu\n",
                 (long long)tokens, (long long)nseq, (long long)heads, (long long)dk, (long long)dv,
                 io_dtype == SSS_BF16 ? "bf16" : "f32", p.nseg, (long long)p.K, p.total);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool bf16 = io_dtype == SSS_BF16;
  char* const ws = static_cast<char*>(workspace);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  const int H = (int)heads, ek = pad(dk), ev = pad(dv);
  const unsigned grid = (unsigned)(p.nseg * heads), folds = p.nseg > 0 ? (unsigned)((p.nseg - 1) * heads) : 0;
  LaWalk w = walk_of(f, p, tokens, nseq);
  w.cu = cu_seqlens;
  w.dfinal = dfinal_state;
  const LaSide sq = f.q.on(heads), sk = f.k.on(heads), sv = f.v.on(heads), so = d.on(heads);
  hipError_t e = hipSuccess;
  if (p.nseg > 1) {  // the states and the adjoints that enter the segments
    LaWalk a = w;
    a.y = sk;
    a.z = sv;
    a.se = dv;
    a.sf = 1;
    a.from = initial_state;
    a.end = at(p.end);
    a.sum = at(p.sum);
    a.flag = reinterpret_cast<int32_t*>(ws + p.flag);
    LaWalk b = a;
    b.y = sq;
    b.z = so;
    b.from = dfinal_state;
    b.end = at(p.rend);
    b.sum = at(p.rsum);
    b.flag = reinterpret_cast<int32_t*>(ws + p.rflag);
    e = la_launch_folds(ek, ev, bf16, a, b, folds, s);
    const LaCarry back{b.end, b.sum, b.flag, at(p.renter)};
    if (e == hipSuccess) e = la_carry({a.end, a.sum, a.flag, at(p.enter)}, &back, w.hs, H, p.nseg, s);
  }
  if (e == hipSuccess && p.nseg > 0) {
    LaWalk a = w;  // dq
    a.x = so;
    a.y = sv;
    a.z = sk;
    a.w = sq;
    a.out_f32 = q_heads < heads;
    a.out = a.out_f32 ? ws + p.dq : static_cast<char*>(dq);
    a.out_st = heads * dk;
    a.out_sh = dk;
    a.se = 1;
    a.sf = dv;
    a.from = initial_state;
    a.enter = at(p.enter);
    a.back = at(p.renter);
    a.rows = at(p.rows);
    a.cols = at(p.cols);
    a.within = at(p.within);
    a.edge = at(p.edge);
    a.last = at(p.last);
    a.trace = D_skip ? at(p.trace) : nullptr;
    LaWalk b = a;  // dk
    b.x = sv;
    b.y = so;
    b.z = sq;
    b.w = sk;
    b.out_f32 = k_heads < heads;
    b.out = b.out_f32 ? ws + p.dk : static_cast<char*>(dk_out);
    b.from = dfinal_state;
    b.to = dinitial_state;
    b.enter = at(p.renter);
    b.cols2 = at(p.cols2);
    LaWalk c = b;  // dv
    c.x = sk;
    c.y = sq;
    c.z = so;
    c.out_f32 = 0;
    c.out = static_cast<char*>(dv_out);
    c.out_st = heads * dv;
    c.out_sh = dv;
    c.se = dv;
    c.sf = 1;
    e = la_launch_grads(ev, ek, bf16, a, b, c, grid, s);
    if (e == hipSuccess && ek != ev) e = la_launch(ek, ev, kLaDv, bf16, c, grid, s);
    const LaSum of_q{at(p.dq), dq, (int)(heads / q_heads)}, of_k{at(p.dk), dk_out, (int)(heads / k_heads)};
    const bool sum_q = q_heads < heads, sum_k = k_heads < heads;
    if (e == hipSuccess && (sum_q || sum_k))
      e = la_sum_heads(sum_q ? of_q : of_k, sum_q && sum_k ? &of_k : nullptr, tokens, H, (int)dk, bf16, s);
  }
  if (e == hipSuccess) {
    LaFinish a{};
    a.rows = at(p.rows);
    a.cols = at(p.cols);
    a.cols2 = at(p.cols2);
    a.within = at(p.within);
    a.edge = at(p.edge);
    a.last = at(p.last);
    a.g = log_decay;
    a.g_st = decay_stride;
    a.beta = beta;
    a.beta_st = beta_stride;
    a.cu = cu_seqlens;
    a.dg = dlog_decay;
    a.part = decay_stride == 0 ? at(p.gpart) : nullptr;
    a.dbeta = beta ? dbeta : nullptr;
    a.trace = at(p.trace);
    a.dD = D_skip ? dD : nullptr;
    a.tokens = (int)tokens;
    a.nseq = (int)nseq;
    a.H = H;
    a.K = (int)p.K;
    a.nseg = p.nseg;
    a.tile = bf16 ? kLaTile : kLaTile / 2;
    e = la_finish(a, s);
  }
  if (e == hipSuccess && dinitial_state && nseq > 0)
    e = la_empty(cu_seqlens, dfinal_state, dinitial_state, (int)nseq, (int)tokens, heads * dk * dv, s);
  return status_of(e);
}

}  // extern "C"
