// C ABI of linear layers in MX form: argument checks, then one launch per
// call.  Nothing throws across the ABI.
#include <cstdint>

#include "fp8q.h"
#include "mx_linear.cuh"
#include "mx_matmul_plan.cuh"

using namespace fp8q;

static bool multiple16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A matrix's description; *v receives what the kernels take.
static int check_matrix(const mx_matrix* m, MxView* v) {
  if (!m) return FP8Q_EINVAL;
  if (m->format != FP8Q_E4M3 && m->format != FP8Q_E5M2 && m->format != FP8Q_E2M1) return FP8Q_EDTYPE;
  if (m->rows < 0 || m->rows > 0x7FFFFFFF || m->cols <= 0 || m->cols % 32 != 0 || m->cols > (int64_t(1) << 31))
    return FP8Q_EINVAL;
  *v = {m->q, m->e8m0, m->rows, m->cols, m->q_stride, m->e8m0_stride, m->format};
  if (m->rows == 0) return FP8Q_OK;
  if (!m->q || !m->e8m0) return FP8Q_EINVAL;
  if (!multiple16(m->q)) return FP8Q_EALIGN;
  if (m->rows == 1) {
    v->q_stride = v->row_bytes();
    v->e_stride = m->cols / 32;
    return FP8Q_OK;
  }
  if (m->q_stride % 16 != 0) return FP8Q_EALIGN;
  if (m->q_stride < v->row_bytes() || m->e8m0_stride < m->cols / 32 || m->q_stride >= (int64_t(1) << 40) ||
      m->e8m0_stride >= (int64_t(1) << 40))
    return FP8Q_EINVAL;
  return FP8Q_OK;
}

// Rows of a plain tensor: base and stride a multiple of `align` bytes.  A
// single row's stride is not used.
static int check_plain(const void* x, int dtype, int64_t rows, int64_t cols, int64_t stride, int align) {
  if (!x) return FP8Q_EINVAL;
  const int64_t size = dtype == FP8Q_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % align != 0) return FP8Q_EALIGN;
  if (rows <= 1) return FP8Q_OK;
  if (stride % (align / size) != 0) return FP8Q_EALIGN;
  return stride < cols || stride >= (int64_t(1) << 40) ? FP8Q_EINVAL : FP8Q_OK;
}

static bool known_dtype(int d) { return d == FP8Q_F32 || d == FP8Q_BF16; }
static bool known_act(int a) { return a >= MX_ACT_SILU && a <= MX_ACT_GELU_TANH; }

static int finish(cudaError_t e, int launches) {
  note_launches(launches);
  return e == cudaSuccess ? FP8Q_OK : record_cuda_error(e);
}

// A matrix of `rows` x `cols` (any format, or an 8-bit one) that may be left out.
static int check_kept(const mx_matrix* m, int64_t rows, int64_t cols, bool eight, MxView* v) {
  *v = MxView{};
  if (!m) return FP8Q_OK;
  const int st = check_matrix(m, v);
  if (st != FP8Q_OK) return st;
  if (eight && m->format == FP8Q_E2M1) return FP8Q_EDTYPE;
  return m->rows == rows && m->cols == cols ? FP8Q_OK : FP8Q_EINVAL;
}

// A product's arguments; rows of a or b may be none, and the rest is then not looked at.
static int check_product(const mx_matrix* a, const mx_matrix* b, void* out, int dtype, int64_t out_stride,
                         const void* add, int64_t add_stride, MxProduct* p) {
  int st = check_matrix(a, &p->a);
  if (st == FP8Q_OK) st = check_matrix(b, &p->b);
  if (st != FP8Q_OK) return st;
  if (!known_dtype(dtype) || (a->format == FP8Q_E2M1) != (b->format == FP8Q_E2M1)) return FP8Q_EDTYPE;
  if (a->cols != b->cols || a->cols > MX_MATMUL_MAX_K) return FP8Q_EINVAL;
  if (a->rows == 0 || b->rows == 0) return FP8Q_OK;
  const int size = dtype == FP8Q_F32 ? 4 : 2;
  st = check_plain(out, dtype, a->rows, b->rows, out_stride, size);
  if (st == FP8Q_OK && add) st = check_plain(add, dtype, a->rows, b->rows, add_stride, size);
  p->out = out;
  p->add = add;
  p->out_stride = out_stride;
  p->add_stride = add_stride;
  p->fp32 = dtype == FP8Q_F32;
  return st;
}

extern "C" {

FP8Q_API int mx_decode(const mx_matrix* m, void* out, int dtype, int64_t out_stride, void* stream) {
  FP8Q_TRACE_CALL();
  MxView v;
  int st = check_matrix(m, &v);
  if (st != FP8Q_OK) return st;
  if (!known_dtype(dtype)) return FP8Q_EDTYPE;
  if (v.rows == 0) return FP8Q_OK;
  st = check_plain(out, dtype, v.rows, v.cols, out_stride, 16);
  if (st != FP8Q_OK) return st;
  int launches = 0;
  const cudaError_t e = launch_mx_decode(v, out, dtype, out_stride, reinterpret_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

FP8Q_API int mx_matmul(const mx_matrix* a, const mx_matrix* b, void* out, int dtype, int64_t out_stride,
                       const void* add, int64_t add_stride, void* stream) {
  FP8Q_TRACE_CALL();
  MxProduct p;
  const int st = check_product(a, b, out, dtype, out_stride, add, add_stride, &p);
  if (st != FP8Q_OK) return st;
  if (p.a.rows == 0 || p.b.rows == 0) return FP8Q_OK;
  int launches = 0;
  const auto launch = a->format == FP8Q_E2M1 ? launch_mx_matmul_4 : launch_mx_matmul_8;
  const cudaError_t e = launch(p, reinterpret_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

FP8Q_API int mx_matmul_plan(const mx_matrix* a, const mx_matrix* b, const void* out, int dtype, int64_t out_stride,
                            const void* add, int64_t add_stride, int sms, mx_matmul_form* form) {
  FP8Q_TRACE_CALL();
  if (!form || sms < 2) return FP8Q_EINVAL;
  MxProduct p;
  const int st = check_product(a, b, const_cast<void*>(out), dtype, out_stride, add, add_stride, &p);
  if (st != FP8Q_OK) return st;
  *form = mx_matmul_form{};
  if (p.a.rows == 0 || p.b.rows == 0) return FP8Q_OK;
  const MmPlan plan = plan_product(p, sms);
  form->pair = plan.pair;
  form->columns = plan.columns;
  form->way_out = plan.pair ? static_cast<int32_t>(plan.out) : 0;
  form->splits = plan.splits;
  form->tiles = plan.tiles;
  return FP8Q_OK;
}

FP8Q_API int mx_act_forward(int act, const void* z, int64_t z_stride, const void* u, int64_t u_stride, int dtype,
                            int64_t rows, int64_t cols, const mx_matrix* z_saved, const mx_matrix* u_saved, int rule,
                            void* h, int64_t h_stride, const mx_matrix* h_mx, void* stream) {
  FP8Q_TRACE_CALL();
  if (!known_act(act) || rule < FP8Q_MX_FLOOR || rule > FP8Q_MX_NEAREST) return FP8Q_EINVAL;
  if (!known_dtype(dtype)) return FP8Q_EDTYPE;
  if (rows < 0 || rows > 0x7FFFFFFF || cols <= 0 || cols % 32 != 0 || cols > (int64_t(1) << 31)) return FP8Q_EINVAL;
  // without rows a tensor that is there may have no address either
  if (rows && ((!h && !h_mx && !z_saved) || (u_saved && !u) || (u && !u_saved != !z_saved))) return FP8Q_EINVAL;
  MxActForward a;
  int st = check_kept(z_saved, rows, cols, true, &a.z_saved);
  if (st == FP8Q_OK) st = check_kept(u_saved, rows, cols, true, &a.u_saved);
  if (st == FP8Q_OK) st = check_kept(h_mx, rows, cols, false, &a.h_mx);
  if (st == FP8Q_OK && u_saved && z_saved && u_saved->format != z_saved->format) st = FP8Q_EDTYPE;
  if (st != FP8Q_OK) return st;
  if (rows == 0) return FP8Q_OK;
  st = check_plain(z, dtype, rows, cols, z_stride, 16);
  if (st == FP8Q_OK && u) st = check_plain(u, dtype, rows, cols, u_stride, 16);
  if (st == FP8Q_OK && h) st = check_plain(h, dtype, rows, cols, h_stride, 16);
  if (st != FP8Q_OK) return st;
  a.z = z;
  a.u = u;
  a.z_stride = z_stride;
  a.u_stride = u_stride;
  a.h = h;
  a.h_stride = h_stride;
  a.rule = rule;
  int launches = 0;
  const cudaError_t e = launch_mx_act_forward(a, act, dtype, rows, cols, reinterpret_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

FP8Q_API int mx_act_backward(int act, const mx_matrix* z_saved, const mx_matrix* u_saved, const void* dh,
                             int64_t dh_stride, int dtype, void* dz, int64_t dz_stride, void* du, int64_t du_stride,
                             void* h, int64_t h_stride, void* stream) {
  FP8Q_TRACE_CALL();
  if (!known_act(act) || !z_saved) return FP8Q_EINVAL;
  const int64_t rows = z_saved->rows, cols = z_saved->cols;
  if (rows && !u_saved != !du) return FP8Q_EINVAL;
  if (!known_dtype(dtype)) return FP8Q_EDTYPE;
  MxActBackward a;
  int st = check_kept(z_saved, rows, cols, true, &a.z);
  if (st == FP8Q_OK) st = check_kept(u_saved, rows, cols, true, &a.u);
  if (st == FP8Q_OK && u_saved && u_saved->format != z_saved->format) st = FP8Q_EDTYPE;
  if (st != FP8Q_OK) return st;
  if (rows == 0) return FP8Q_OK;
  st = check_plain(dh, dtype, rows, cols, dh_stride, 16);
  if (st == FP8Q_OK) st = check_plain(dz, dtype, rows, cols, dz_stride, 16);
  if (st == FP8Q_OK && du) st = check_plain(du, dtype, rows, cols, du_stride, 16);
  if (st == FP8Q_OK && h) st = check_plain(h, dtype, rows, cols, h_stride, 16);
  if (st != FP8Q_OK) return st;
  a.dh = dh;
  a.dh_stride = dh_stride;
  a.dz = dz;
  a.du = du;
  a.h = h;
  a.dz_stride = dz_stride;
  a.du_stride = du_stride;
  a.h_stride = h_stride;
  int launches = 0;
  const cudaError_t e = launch_mx_act_backward(a, act, dtype, reinterpret_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

}  // extern "C"
