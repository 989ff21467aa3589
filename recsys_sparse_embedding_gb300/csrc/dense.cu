// The dense operators of any width (declared in dinsparse.h): the calls and
// their checks.
#include "dense_host.cuh"

namespace dsf {
namespace dense {
namespace {

// x W^T with the forward's epilogue (dz null) or the backward's into dz.
bool layer_product(const Ctx& c, const float* xs, const void* in, long long ldi, void* y, long long ldy, bool dz,
                   float* sums) {
  const dsf_dense* l = c.l;
  const bool f32 = l->dtype == DSF_F32;
  Product p{};
  p.A = c.X;
  p.B = c.W;
  p.major = kKK;
  p.gated = c.gated;
  p.f32 = f32;
  p.epi = dz ? kEpiDz : (in ? kEpiRes : kEpiFwd);
  const long long nkb = (l->K + c.kbe - 1) / c.kbe;
  p.a.part = sums;
  plan(p, c.M, c.N, 1, nkb, 1, !dz);
  Job& o = p.a.job[0];
  o.a_term = 1;
  o.b_term = 1;
  p.a.act = l->act;
  p.a.bias = l->bias;
  p.a.xs = xs;
  p.a.ws = l->scale;
  p.a.status = c.status;
  if (o.splits > 1) {
    set_part(p, c);
  } else {
    p.a.in = in;
    p.a.ldi = ldi;
    p.a.in_vec = in && vec_rows(in, ldi, c.eo);
    set_out(o, y, ldy, dz ? 2 : c.eo);
  }
  const bool ok = dz ? run_dz_product(p, c.s) : (l->dtype == DSF_E4M3 ? run_e4m3_product(p, c.s) : run_fwd_product(p, c.s));
  if (!ok || o.splits == 1) return ok;
  FinishArgs f{};
  f.fwd = true;
  f.gated = c.gated;
  f.planes = c.halves;
  f.bias = l->bias;
  f.xs = xs;
  f.ws = l->scale;
  f.res = in;
  f.ldr = ldi;
  f.out = y;
  f.ldo = ldy;
  f.act = l->act;
  return finish(c, p, f, f32);
}

int fwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const float* xs, const void* res, long long ldr,
        long long M, void* y, long long ldy, void* ws, int* status, cudaStream_t s) {
  bool ok;
  if (small_call(l->dtype, M, l->R, l->K)) {
    const int N = gated ? l->R / 2 : l->R;
    const SmallArgs a{x, l->W, ldx, l->ldw, l->bias, xs, l->scale, res, ldr, y, ldy, int(M), N, l->K, l->act, 0};
    const bool vec = (l->K * esize(l->dtype)) % 16 == 0;
    ok = l->dtype == DSF_F32    ? launch_small<float, float>(a, gated, vec, s)
         : l->dtype == DSF_BF16 ? launch_small<__nv_bfloat16, __nv_bfloat16>(a, gated, vec, s)
                                : launch_small<__nv_fp8_e4m3, __nv_bfloat16>(a, gated, vec, s);
  } else {
    const Ctx c = context(l, gated, x, ldx, M, ws, false, status, s);
    ok = lay_operands(c, x, ldx, nullptr, 0) && layer_product(c, xs, res, ldr, y, ldy, false, nullptr);
  }
  return ok ? DSF_OK : DSF_ECUDA;
}

int bwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const void* dy, long long lddy, long long M,
        void* dx, long long lddx, void* dW, float* db, void* ws, int* status, cudaStream_t s) {
  const Ctx c = context(l, gated, x, ldx, M, ws, true, status, s);
  const bool f32 = l->dtype == DSF_F32, own_dz = gated || l->act != DSF_ACT_NONE;
  float* sums = reinterpret_cast<float*>(c.ws + c.w.sums);
  if (!dx && !dW && !db) return DSF_OK;
  if ((own_dz || dx || dW) && !lay_operands(c, x, ldx, own_dz ? nullptr : dy, lddy)) return DSF_ECUDA;
  Mat dz;
  if (own_dz) {
    void* d = c.ws + c.w.dz;
    if (!layer_product(c, nullptr, dy, lddy, d, c.w.np, true, db ? sums : nullptr)) return DSF_ECUDA;
    if (db && !colsum(sums, (M + 31) / 32, l->R, db, s)) return DSF_ECUDA;
    dz = Mat{d, M, c.N, c.w.np, (long long)c.terms * c.halves, M * c.w.np};
  } else {
    if (db) {
      const long long blocks = (M + kSumRows - 1) / kSumRows;
      const bool laid = !f32 && laid_out(l->dtype, c.N) && (dx || dW);  // (the aligned copy of dy)
      const bool ok = f32    ? row_block_sums<float>(dy, lddy, false, M, c.N, sums, s)
                      : laid ? row_block_sums<__nv_bfloat16>(c.ws + c.w.gp, c.w.np, true, M, c.N, sums, s)
                             : row_block_sums<__nv_bfloat16>(dy, lddy, false, M, c.N, sums, s);
      if (!ok || !colsum(sums, blocks, c.N, db, s)) return DSF_ECUDA;
    }
    dz = laid_out(l->dtype, c.N) ? Mat{c.ws + c.w.gp, M, c.N, c.w.np, c.terms, M * c.w.np} : Mat{dy, M, c.N, lddy, 1, 0};
  }
  return grad_products(c, dz, dx, lddx, dW) ? DSF_OK : DSF_ECUDA;
}

int run_fwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const float* xs, const void* res,
            long long ldr, long long M, void* y, long long ldy, void* ws, size_t ws_bytes, int* status,
            void* stream) {
  if (int rc = check_layer(l, gated)) return rc;
  if (M < 0 || M > kMaxM) return DSF_EINVAL;
  if (M == 0) return DSF_OK;
  const int N = gated ? l->R / 2 : l->R, eo = osize(l->dtype);
  if (!rows_ok(x, ldx, l->K, esize(l->dtype))) return DSF_EINVAL;
  if ((l->dtype == DSF_E4M3) != (xs != nullptr) || !at(xs, 4)) return DSF_EINVAL;
  if (!y || ldy < N || !at(y, eo) || (res && (ldr < N || !at(res, eo)))) return DSF_EINVAL;
  if (!ws || !at(ws, 256) || ws_bytes < ws_bytes_of(l, M, gated, false)) return DSF_EWORKSPACE;
  return fwd(l, gated, x, ldx, xs, res, ldr, M, y, ldy, ws, status, static_cast<cudaStream_t>(stream));
}

int run_bwd(const dsf_dense* l, bool gated, const void* x, long long ldx, const void* dy, long long lddy, long long M,
            void* dx, long long lddx, void* dW, float* db, void* ws, size_t ws_bytes, int* status, void* stream) {
  if (int rc = check_layer(l, gated)) return rc;
  if (l->dtype == DSF_E4M3) return DSF_EUNSUPPORTED;
  if (M < 0 || M > kMaxM) return DSF_EINVAL;
  const int N = gated ? l->R / 2 : l->R, es = esize(l->dtype);
  if (!at(dW, es) || !at(db, 4)) return DSF_EINVAL;
  if (M > 0 && (!rows_ok(x, ldx, l->K, es) || !rows_ok(dy, lddy, N, es) || (dx && (lddx < l->K || !at(dx, es)))))
    return DSF_EINVAL;
  if (!ws || !at(ws, 256) || ws_bytes < ws_bytes_of(l, M, gated, true)) return DSF_EWORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (dW && !succeeded(cudaMemsetAsync(dW, 0, size_t(l->R) * l->K * es, s))) return DSF_ECUDA;
    if (db && !succeeded(cudaMemsetAsync(db, 0, size_t(l->R) * 4, s))) return DSF_ECUDA;
    return DSF_OK;
  }
  return bwd(l, gated, x, ldx, dy, lddy, M, dx, lddx, dW, db, ws, status, s);
}

}  // namespace
}  // namespace dense
}  // namespace dsf

using namespace dsf::dense;

extern "C" {

size_t dsf_dense_workspace_bytes(const dsf_dense* l, int64_t M, int32_t gated, int32_t backward) {
  if (check_layer(l, gated != 0) != DSF_OK || M < 0 || M > kMaxM || gated < 0 || gated > 1 || backward < 0 ||
      backward > 1)
    return 0;
  if (backward && l->dtype == DSF_E4M3) return 0;
  return ws_bytes_of(l, M, gated != 0, backward != 0);
}

int ctr_dense_fwd(const dsf_dense* l, const void* x, int64_t ldx, const float* xs, const void* res, int64_t ldr,
                  int64_t M, void* y, int64_t ldy, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_fwd(l, false, x, ldx, xs, res, ldr, M, y, ldy, ws, ws_bytes, status, stream);
}

int ctr_glu_fwd(const dsf_dense* l, const void* x, int64_t ldx, const float* xs, int64_t M, void* h, int64_t ldh,
                void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_fwd(l, true, x, ldx, xs, nullptr, 0, M, h, ldh, ws, ws_bytes, status, stream);
}

int ctr_dense_bwd(const dsf_dense* l, const void* x, int64_t ldx, const void* dy, int64_t lddy, int64_t M, void* dx,
                  int64_t lddx, void* dW, float* db, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_bwd(l, false, x, ldx, dy, lddy, M, dx, lddx, dW, db, ws, ws_bytes, status, stream);
}

int ctr_glu_bwd(const dsf_dense* l, const void* x, int64_t ldx, const void* dh, int64_t lddh, int64_t M, void* dx,
                int64_t lddx, void* dW, float* db, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return run_bwd(l, true, x, ldx, dh, lddh, M, dx, lddx, dW, db, ws, ws_bytes, status, stream);
}

}  // extern "C"
