// C ABI of the INT8 path and of the several-axis rotary: argument validation and
// launches (vitq.h gives each entry point's contract).
namespace vitq {
namespace {

inline int elem_bytes(int dtype) { return dtype == VITQ_FP32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == VITQ_BF16 || dtype == VITQ_FP16 || dtype == VITQ_FP32; }
inline bool al(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }

int rows_int8_check(const void* x, int M, int K, int ldx, const int8_t* q, int ldq, const float* s, int es) {
  VITQ_CHECK(M == 0 || (x && q && s), VITQ_ERR_INVALID_ARG);
  VITQ_CHECK(M >= 0 && K > 0 && ldx >= K && ldq >= K, VITQ_ERR_INVALID_ARG);
  VITQ_CHECK(M <= VITQ_MAX_ROWS && K <= VITQ_MAX_DIM && ldq % 16 == 0, VITQ_ERR_SHAPE);
  VITQ_CHECK(al(x, es) && al16(q) && al(s, 4), VITQ_ERR_ALIGN);
  return VITQ_OK;
}

}  // namespace
}  // namespace vitq

extern "C" {

int vit_quant_int8(const void* x, int dtype, int M, int K, int ldx, int8_t* q, int ldq, float* s, void* stream) {
  VITQ_CHECK(dtype_ok(dtype), VITQ_ERR_INVALID_ARG);
  int r = rows_int8_check(x, M, K, ldx, q, ldq, s, elem_bytes(dtype));
  if (r) return r;
  int sms = 0;
  r = current_device_ok(&sms);
  if (r) return r;
  if (M == 0) return VITQ_OK;
  const RowsInt8 a{x, ldx, M, K, nullptr, nullptr, 0.0, q, ldq, s};
  VITQ_LAUNCH("quant_int8", S(stream), 0, (double)M * K * (elem_bytes(dtype) + 1) + 4.0 * M,
              launch_quant_int8(a, dtype, sms, S(stream)));
  return VITQ_OK;
}

int vit_ln_quant_int8(const void* x, int M, int K, int ldx, const void* gamma, const void* beta, float eps, int8_t* q,
                      int ldq, float* s, void* stream) {
  VITQ_CHECK(gamma && beta && eps >= 0.f, VITQ_ERR_INVALID_ARG);
  int r = rows_int8_check(x, M, K, ldx, q, ldq, s, 2);
  if (r) return r;
  VITQ_CHECK(al(gamma, 2) && al(beta, 2), VITQ_ERR_ALIGN);
  int sms = 0;
  r = current_device_ok(&sms);
  if (r) return r;
  if (M == 0) return VITQ_OK;
  const RowsInt8 a{x, ldx, M, K, (const __nv_bfloat16*)gamma, (const __nv_bfloat16*)beta, (double)eps, q, ldq, s};
  VITQ_LAUNCH("ln_quant_int8", S(stream), 0, 3.0 * M * K + 4.0 * M + 4.0 * K, launch_ln_quant_int8(a, sms, S(stream)));
  return VITQ_OK;
}

int vit_gelu_quant_int8(const void* f, int M, int K, int ldf, int8_t* q, int ldq, float* s, void* stream) {
  int r = rows_int8_check(f, M, K, ldf, q, ldq, s, 2);
  if (r) return r;
  int sms = 0;
  r = current_device_ok(&sms);
  if (r) return r;
  if (M == 0) return VITQ_OK;
  const RowsInt8 a{f, ldf, M, K, nullptr, nullptr, 0.0, q, ldq, s};
  VITQ_LAUNCH("gelu_quant_int8", S(stream), 0, 3.0 * M * K + 4.0 * M, launch_gelu_quant_int8(a, sms, S(stream)));
  return VITQ_OK;
}

int int8_gemm(const int8_t* A, int lda, const float* sA, const int8_t* W, int ldw, const float* sW, const void* bias,
              const void* residual, int ldr, void* C, int ldc, int dtype, int M, int N, int K, void* stream) {
  VITQ_CHECK(W && sW && dtype_ok(dtype) && (M == 0 || (A && sA && C)), VITQ_ERR_INVALID_ARG);
  VITQ_CHECK(M >= 0 && N > 0 && K > 0 && lda >= K && ldw >= K && ldc >= N && (!residual || ldr >= N),
             VITQ_ERR_INVALID_ARG);
  VITQ_CHECK(!residual || residual != C || ldr == ldc || M <= 1, VITQ_ERR_INVALID_ARG);
  VITQ_CHECK(M <= VITQ_MAX_ROWS && N <= VITQ_MAX_DIM && K <= VITQ_MAX_DIM, VITQ_ERR_SHAPE);
  VITQ_CHECK(lda % 16 == 0 && ldw % 16 == 0, VITQ_ERR_SHAPE);
  const int es = elem_bytes(dtype);
  VITQ_CHECK(al16(A) && al16(W) && al(sA, 4) && al(sW, 4) && al(C, es) && al(bias, es) && al(residual, es),
             VITQ_ERR_ALIGN);
  int sms = 0;
  const int r = current_device_ok(&sms);
  if (r) return r;
  if (M == 0) return VITQ_OK;
  const Int8Gemm p{A, lda, sA, W, ldw, sW, bias, residual, ldr, C, ldc, dtype, M, N, K};
  const double mn = (double)M * N;
  VITQ_LAUNCH("int8_gemm", S(stream), 2.0 * mn * K,
              (double)M * K + (double)N * K + 4.0 * (M + N) + es * (mn * (residual ? 2 : 1) + (bias ? N : 0)),
              launch_int8_gemm(p, sms, S(stream)));
  return VITQ_OK;
}

int vit_rope_axes(const vitq_rope_axes* p, const void* q, void* q_out, const void* k, void* k_out,
                  const int32_t* pos, int n_tokens, void* stream) {
  VITQ_CHECK(p && (pos || n_tokens == 0) && n_tokens >= 0 && dtype_ok(p->dtype), VITQ_ERR_INVALID_ARG);
  VITQ_CHECK(p->heads_q >= 0 && p->heads_k >= 0 && p->head_dim > 0, VITQ_ERR_INVALID_ARG);
  VITQ_CHECK(n_tokens == 0 || ((p->heads_q == 0 || (q && q_out)) && (p->heads_k == 0 || (k && k_out))),
             VITQ_ERR_INVALID_ARG);
  VITQ_CHECK((p->flags & ~(VITQ_ROPE_INTERLEAVED | VITQ_ROPE_AXIS_FREQ | VITQ_ROPE_ADJACENT | VITQ_ROPE_INVERSE)) == 0,
             VITQ_ERR_INVALID_ARG);
  VITQ_CHECK(p->theta > 0.0 && std::isfinite(p->theta), VITQ_ERR_INVALID_ARG);
  VITQ_CHECK(p->n_axes >= 1 && p->n_axes <= VITQ_ROPE_MAX_AXES, VITQ_ERR_SHAPE);
  VITQ_CHECK(n_tokens <= VITQ_MAX_ROWS && p->heads_q <= 1024 && p->heads_k <= 1024 && p->head_dim <= 2 * kRopeMaxPairs,
             VITQ_ERR_SHAPE);
  int pairs = 0;
  for (int a = 0; a < p->n_axes; ++a) {
    VITQ_CHECK(p->sections[a] >= 0 && p->sections[a] <= kRopeMaxPairs, VITQ_ERR_SHAPE);
    pairs += p->sections[a];
  }
  VITQ_CHECK(pairs > 0 && 2 * pairs <= p->head_dim, VITQ_ERR_SHAPE);
  const int64_t strides[10] = {p->q_token,   p->q_head,     p->q_out_token, p->q_out_head, p->k_token,
                               p->k_head,    p->k_out_token, p->k_out_head, p->pos_token,  p->pos_axis};
  for (int64_t v : strides) VITQ_CHECK(v >= 0 && v < (1ll << 31), VITQ_ERR_SHAPE);
  // each output element is written once: one of the two strides spans the other's extent
  auto apart = [&](int64_t t, int64_t h, int heads) {
    return (h >= p->head_dim || heads <= 1) && (t >= (int64_t)(heads - 1) * h + p->head_dim || n_tokens <= 1) ? true
           : (t >= p->head_dim || n_tokens <= 1) && (h >= (int64_t)(n_tokens - 1) * t + p->head_dim || heads <= 1);
  };
  VITQ_CHECK(p->heads_q == 0 || apart(p->q_out_token, p->q_out_head, p->heads_q), VITQ_ERR_SHAPE);
  VITQ_CHECK(p->heads_k == 0 || apart(p->k_out_token, p->k_out_head, p->heads_k), VITQ_ERR_SHAPE);
  VITQ_CHECK(p->heads_q == 0 || q != q_out || (p->q_token == p->q_out_token && p->q_head == p->q_out_head),
             VITQ_ERR_INVALID_ARG);
  VITQ_CHECK(p->heads_k == 0 || k != k_out || (p->k_token == p->k_out_token && p->k_head == p->k_out_head),
             VITQ_ERR_INVALID_ARG);
  const int es = elem_bytes(p->dtype);
  VITQ_CHECK(al(q, es) && al(q_out, es) && al(k, es) && al(k_out, es) && al(pos, 4), VITQ_ERR_ALIGN);

  RopeAxes r = {};
  r.side[0] = RopeSide{q, q_out, (int)p->q_token, (int)p->q_head, (int)p->q_out_token, (int)p->q_out_head, p->heads_q};
  r.side[1] = RopeSide{k, k_out, (int)p->k_token, (int)p->k_head, (int)p->k_out_token, (int)p->k_out_head, p->heads_k};
  r.pos = pos;
  r.pos_t = p->pos_token;
  r.pos_a = p->pos_axis;
  r.n = n_tokens;
  r.d = p->head_dim;
  r.pairs = pairs;
  r.inverse = (p->flags & VITQ_ROPE_INVERSE) != 0;
  r.adjacent = (p->flags & VITQ_ROPE_ADJACENT) != 0;
  // axis of every pair
  int first = 0;
  for (int a = 0; a < p->n_axes; ++a) {
    for (int i = 0; i < p->sections[a]; ++i) r.axis[first + i] = (uint8_t)a;
    first += p->sections[a];
  }
  if (p->flags & VITQ_ROPE_INTERLEAVED) {
    for (int j = 0; j < pairs; ++j) r.axis[j] = 0;
    for (int a = 1; a < p->n_axes; ++a) {
      VITQ_CHECK(p->sections[a] == 0 || a + p->n_axes * (p->sections[a] - 1) < pairs, VITQ_ERR_SHAPE);
      for (int i = 0; i < p->sections[a]; ++i) r.axis[a + p->n_axes * i] = (uint8_t)a;
    }
  }
  // an output may be its own input, not the other side's tensor
  VITQ_CHECK(n_tokens == 0 || p->heads_q == 0 || p->heads_k == 0 || (q_out != k_out && q_out != k && k_out != q),
             VITQ_ERR_INVALID_ARG);
  // frequencies in turns, each from the one before it: theta^(-1/count) steps, 2^-52 of error each
  const double turn = 0.15915494309189533577;   // 1 / (2 pi)
  if (p->flags & VITQ_ROPE_AXIS_FREQ) {
    double f[VITQ_ROPE_MAX_AXES], step[VITQ_ROPE_MAX_AXES];
    for (int a = 0; a < p->n_axes; ++a) {
      f[a] = turn;
      step[a] = p->sections[a] ? std::pow(p->theta, -1.0 / p->sections[a]) : 1.0;
    }
    for (int j = 0; j < pairs; ++j) {
      r.turns[j] = f[r.axis[j]];
      f[r.axis[j]] *= step[r.axis[j]];
    }
  } else {
    const double step = std::pow(p->theta, -1.0 / pairs);
    double f = turn;
    for (int j = 0; j < pairs; ++j, f *= step) r.turns[j] = f;
  }
  int sms = 0;
  const int s = current_device_ok(&sms);
  if (s) return s;
  if (n_tokens == 0 || p->heads_q + p->heads_k == 0) return VITQ_OK;
  VITQ_LAUNCH("rope_axes", S(stream), 0,
              2.0 * n_tokens * (p->heads_q + p->heads_k) * p->head_dim * es + 4.0 * n_tokens * p->n_axes,
              launch_rope_axes(r, p->dtype, sms, S(stream)));
  return VITQ_OK;
}

}  // extern "C"
