// C ABI of the RMS norm, the 4-bit rows and their products, and the whole expert
// layer (declared in include/sgemm.h): argument validation, the choice of kernel, tile and
// split, the TMA descriptors and the launches.
#include <climits>

#include "api_common.h"
#include "fp4.cuh"

namespace {

bool known_format(int f) { return f == SGEMM_FP4_MX || f == SGEMM_FP4_NV; }

// The scales of rows of K elements: whole tiles of 128 rows x 4 blocks.
Range scales_of(const void *S, int format, int rows, int K) {
    return Range(S, S ? 1 : 0, cdiv(rows, 128) * sg::fp4_words(format, K) * 512, 1, 1);
}
Range floats_of(const float *p, int n) { return Range(p, p ? 1 : 0, n, n, 4); }

// What rows in 4 bits need: the scales' alignment and, of format NV, the row scales.
int check_fp4_rows(int format, int K, const void *Q, const void *S, const float *row) {
    if ((K > 0 && (Q == nullptr || S == nullptr)) || (format == SGEMM_FP4_NV && row == nullptr)) return SGEMM_ERR_NULL;
    return aligned(S, 16) && aligned(row, 4) ? SGEMM_OK : SGEMM_ERR_INVALID_VALUE;
}

bool meets_any(const Range &r, std::initializer_list<Range> others) {
    for (const Range &o : others)
        if (r.meets(o)) return true;
    return false;
}

// The residual's sum may replace either of the rows that it is made of, in place.
bool in_place(const void *p, int ldp, const void *q, int ldq) { return p == q && ldp == ldq; }

// The norm's inputs; y: what else the call writes.
int check_norm(int type, int M, int K, const void *X, int ldx, const void *R, int ldr, const void *weight, float eps,
               const void *H, int ldh) {
    if (M < 0 || check_row(type, K, ldx) != SGEMM_OK || (R && ldr < std::max(1, K)) || (H && ldh < std::max(1, K)) || !(eps >= 0.f))
        return SGEMM_ERR_INVALID_VALUE;
    if (M == 0 || K == 0) return SGEMM_OK;
    if (X == nullptr || weight == nullptr || (R && H == nullptr)) return SGEMM_ERR_NULL;
    const int size = size_of(type);
    return aligned(X, size) && aligned(R, size) && aligned(weight, size) && aligned(H, size) ? SGEMM_OK : SGEMM_ERR_INVALID_VALUE;
}

int norm_aliases(int type, int M, int K, const void *X, int ldx, const void *R, int ldr, const void *weight, const void *H, int ldh,
                 std::initializer_list<Range> outputs) {
    const int size = size_of(type);
    const Range x(X, M, K, ldx, size), r(R, R ? M : 0, K, ldr, size), w(weight, 1, K, K, size), hh(H, H ? M : 0, K, ldh, size);
    if (hh.meets(w) || (hh.meets(x) && !in_place(H, ldh, X, ldx)) || (hh.meets(r) && !in_place(H, ldh, R, ldr))) return SGEMM_ERR_ALIAS;
    for (const Range &o : outputs) {
        if (meets_any(o, {x, r, w, hh})) return SGEMM_ERR_ALIAS;
        for (const Range &p : outputs)
            if (&p != &o && o.meets(p)) return SGEMM_ERR_ALIAS;
    }
    return SGEMM_OK;
}

sg::RowArgs norm_args(int M, int K, const void *X, int ldx, const void *R, int ldr, const void *weight, float eps, void *H, int ldh,
                      void *Y, int ldy, float *row) {
    sg::RowArgs a{};
    a.X = X;
    a.ldx = ldx;
    a.R = R;
    a.ldr = ldr;
    a.W = weight;
    a.eps = eps;
    a.H = H;
    a.ldh = ldh;
    a.M = M;
    a.K = K;
    a.Y = Y;
    a.ldy = ldy;
    a.row = row;
    return a;
}

int check_fp4(int format, int out_type, int M, int N, int K, const uint8_t *A, int lda, const uint8_t *SA, const float *rowA,
              const uint8_t *B, int ldb, const uint8_t *SB, const float *rowB, const float *bias, const void *C, int ldc) {
    if (!known_format(format) || !known_type(out_type) || M < 0 || N < 0 || K < 0 || M > kMaxExtent || N > kMaxExtent || K > kMaxExtent)
        return SGEMM_ERR_INVALID_VALUE;
    const int bytes = (K + 1) / 2;
    if (lda < std::max(1, bytes) || ldb < std::max(1, bytes) || ldc < std::max(1, N)) return SGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (C == nullptr) return SGEMM_ERR_NULL;
    for (int st : {check_fp4_rows(format, K, A, SA, rowA), check_fp4_rows(format, K, B, SB, rowB)})
        if (st != SGEMM_OK) return st;
    if (!aligned(C, size_of(out_type)) || !aligned(bias, 4)) return SGEMM_ERR_INVALID_VALUE;
    const Range c(C, M, N, ldc, size_of(out_type));
    if (meets_any(c, {floats_of(rowA, M), floats_of(rowB, N), floats_of(bias, N)})) return SGEMM_ERR_ALIAS;
    if (K > 0 && meets_any(c, {Range(A, M, bytes, lda, 1), Range(B, N, bytes, ldb, 1), scales_of(SA, format, M, K), scales_of(SB, format, N, K)}))
        return SGEMM_ERR_ALIAS;
    return SGEMM_OK;
}

struct Fp4Choice {
    int nt, ksplit;
};
// Tile and split (us in graphs, NV).  CTA pairs from a fifth of the SMs' worth of their tiles on
// (200 x 8192 x 4096 9.7 against 11.0 in tiles of 128, 2048 x 4096 x 4096 16.3 against 22.8; 300 x 2048
// x 4096, 16 tiles, 9.0 against 7.7).  Otherwise the smallest tile that holds all tokens, and K split
// while the CTAs make one wave and each split saves enough stages of 0.23 us for the exchange's 0.8 (1
// x 4096 x 4096: whole 5.9, in two 4.9, four 4.0, eight, two CTAs an SM, 4.5; 1 x 8192 x 1024, four
// stages: 3.1, 3.4, 3.9; 64 x 8192 x 8192: 12.9, 9.9, 10.5; 128 x 4096 x 4096: 8.8, 7.6, 7.0, 11.0).
Fp4Choice choose_fp4(int M, int N, int K, int num_sms, bool pairs) {
    if (pairs && M > 128 && cdiv(M, 256) * cdiv(N, 256) >= num_sms / 5) return {256, 1};
    const int nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    const long long tiles = cdiv(M, nt) * cdiv(N, 128);
    const int stages = static_cast<int>(cdiv(K, sg::kFp4StageK));
    int split = 1;
    while (split < 8 && 10 * tiles * split * 2 <= 11 * num_sms && stages >= std::max(8, 4 * split)) split *= 2;
    return {nt, split};
}

int run_fp4(sgemm_handle_t h, sg::Fp4Args a, cudaStream_t stream) {
    sg::HandleView v;
    sg::view_of(h, &v);
    a.words = sg::fp4_words(a.format, a.K);
    a.status = v.d_status;
    const int bytes = (a.K + 1) / 2, ld = static_cast<int>(cdiv(bytes, 16) * 16);
    const bool a_stored = aligned(a.A, 16) && a.lda % 16 == 0, b_stored = aligned(a.B, 16) && a.ldb % 16 == 0;
    const size_t a_bytes = a_stored ? 0 : static_cast<size_t>(cdiv(static_cast<long long>(a.M) * ld, 1024) * 1024);
    const size_t b_bytes = b_stored ? 0 : static_cast<size_t>(a.N) * ld;
    const bool copies = !a_stored || !b_stored;
    bool tc = a.K > 0 && v.pinned != SGEMM_VARIANT_GENERIC && v.pinned != SGEMM_VARIANT_GENERIC_F4 &&
              (!copies || (v.d_rl != nullptr && v.relayout_mode != SGEMM_RELAYOUT_OFF && a_bytes + b_bytes <= v.rl_bytes)) &&
              std::max(cdiv(a.M, 128), cdiv(a.N, 128)) * a.words < INT_MAX;
    Fp4Choice pick = choose_fp4(a.M, a.N, a.K, v.num_sms, v.pinned != SGEMM_VARIANT_TC_F4);
    if (v.f4_tokens) {
        pick = {v.f4_tokens, v.f4_split};
        // (a tile of fewer than 128 tokens has to be the call's only one)
        while (pick.nt < 128 && pick.nt < a.M) pick.nt *= 2;
        while (pick.ksplit > 1 && pick.ksplit > cdiv(a.K, sg::kFp4StageK)) pick.ksplit /= 2;
    }
    if (v.pinned == SGEMM_VARIANT_TC_F4_PAIR) pick = {256, 1};
    a.nt = pick.nt;
    a.ksplit = pick.ksplit;
    tc = tc && cdiv(a.M, a.nt) * cdiv(a.N, 128) * a.ksplit < INT_MAX;
    int launches = 0;
    if (tc) {
        sg::Int8Copies c{};
        const uint8_t *A = a.A, *B = a.B;
        long long lda = a.lda, ldb = a.ldb;
        if (copies) {
            uint8_t *ws = reinterpret_cast<uint8_t *>(v.d_rl);
            c.A = reinterpret_cast<const int8_t *>(a.A);
            c.lda = a.lda;
            c.a_rows = a.M;
            c.K = bytes;
            c.a_ld = c.b_ld = ld;
            c.B = reinterpret_cast<const int8_t *>(a.B);
            c.ldb = a.ldb;
            c.b_trans = 1;
            c.experts = 1;
            c.N = a.N;
            if (!a_stored) {
                c.a_dst = ws;
                A = ws;
                lda = ld;
            }
            if (!b_stored) {
                c.b_dst = reinterpret_cast<int8_t *>(ws + a_bytes);
                B = ws + a_bytes;
                ldb = ld;
            }
        }
        sg::Fp4Maps m;
        const int stage_words = sg::kFp4StageK / (4 * sg::fp4_block(a.format));
        tc = sg::encode_map(&m.A, sg::MapType::kInt8, 2, A, bytes, a.M, 1, lda, 0, 128, std::min(a.nt, 128)) &&
             sg::encode_map(&m.B, sg::MapType::kInt8, 2, B, bytes, a.N, 1, ldb, 0, 128, 128) &&
             sg::encode_map(&m.SA, sg::MapType::kWords, 2, a.SA, 128, cdiv(a.M, 128) * a.words, 1, 512, 0, 128, stage_words) &&
             sg::encode_map(&m.SB, sg::MapType::kWords, 2, a.SB, 128, cdiv(a.N, 128) * a.words, 1, 512, 0, 128, stage_words);
        if (tc) {
            if (copies) {
                const cudaError_t e = sg::launch_int8_copies(&c, stream);
                if (e != cudaSuccess) return from_cuda(e);
                ++launches;
            }
            const cudaError_t e = sg::launch_fp4_tc(a, m, v.num_sms, v.smem_override, stream);
            if (e != cudaSuccess) return from_cuda(e);
            ++launches;
        }
    }
    if (!tc) {
        a.ksplit = 1;
        const cudaError_t e = sg::launch_fp4_generic(a, stream);
        if (e != cudaSuccess) return from_cuda(e);
        ++launches;
    }
    sg::record_call(h, !tc ? SGEMM_VARIANT_GENERIC_F4 : a.nt == 256 ? SGEMM_VARIANT_TC_F4_PAIR : SGEMM_VARIANT_TC_F4, a.ksplit, launches,
                    tc ? (a_stored ? 0 : 1) | (b_stored ? 0 : 2) : 0);
    return SGEMM_OK;
}

}  // namespace

extern "C" {

int64_t sgemm_fp4_scale_bytes(int format, int rows, int K) {
    if (!known_format(format) || rows < 0 || K < 0 || rows > kMaxExtent || K > kMaxExtent) return -1;
    return cdiv(rows, 128) * sg::fp4_words(format, K) * 512;
}

int sgemm_quantize_fp4(sgemm_handle_t h, int type, int format, int M, int K, const void *X, int ldx, uint8_t *Q, int ldq,
                       uint8_t *S, float *row, void *stream) {
    const int st = enter(h);
    if (st != SGEMM_OK) return st;
    if (!known_format(format) || M < 0 || M > kMaxExtent || check_row(type, K, ldx) != SGEMM_OK || ldq < std::max(1, (K + 1) / 2))
        return SGEMM_ERR_INVALID_VALUE;
    if (M == 0 || K == 0) return nothing(h);
    if (X == nullptr) return SGEMM_ERR_NULL;
    const int bad = check_fp4_rows(format, K, Q, S, row);
    if (bad != SGEMM_OK) return bad;
    if (!aligned(X, size_of(type))) return SGEMM_ERR_INVALID_VALUE;
    const Range x(X, M, K, ldx, size_of(type)), q(Q, M, (K + 1) / 2, ldq, 1), s = scales_of(S, format, M, K), r = floats_of(row, M);
    if (meets_any(x, {q, s, r}) || meets_any(q, {s, r}) || s.meets(r)) return SGEMM_ERR_ALIAS;
    sg::HandleView v;
    sg::view_of(h, &v);
    sg::RowArgs a = norm_args(M, K, X, ldx, nullptr, 0, nullptr, 0.f, nullptr, 0, Q, ldq, row);
    a.S = S;
    a.format = format;
    a.words = sg::fp4_words(format, K);
    return launched(h, sg::launch_quantize_fp4(type, a, v.num_sms, static_cast<cudaStream_t>(stream)));
}

int sgemm_dequantize_fp4(sgemm_handle_t h, int type, int format, int M, int K, const uint8_t *Q, int ldq, const uint8_t *S,
                         const float *row, void *Y, int ldy, void *stream) {
    const int st = enter(h);
    if (st != SGEMM_OK) return st;
    if (!known_format(format) || M < 0 || M > kMaxExtent || check_row(type, K, ldy) != SGEMM_OK || ldq < std::max(1, (K + 1) / 2))
        return SGEMM_ERR_INVALID_VALUE;
    if (M == 0 || K == 0) return nothing(h);
    if (Y == nullptr) return SGEMM_ERR_NULL;
    const int bad = check_fp4_rows(format, K, Q, S, row);
    if (bad != SGEMM_OK) return bad;
    if (!aligned(Y, size_of(type))) return SGEMM_ERR_INVALID_VALUE;
    const Range y(Y, M, K, ldy, size_of(type));
    if (meets_any(y, {Range(Q, M, (K + 1) / 2, ldq, 1), scales_of(S, format, M, K), floats_of(row, M)})) return SGEMM_ERR_ALIAS;
    sg::HandleView v;
    sg::view_of(h, &v);
    sg::RowArgs a = norm_args(M, K, Q, ldq, nullptr, 0, nullptr, 0.f, nullptr, 0, Y, ldy, const_cast<float *>(row));
    a.S = const_cast<uint8_t *>(S);
    a.format = format;
    a.words = sg::fp4_words(format, K);
    return launched(h, sg::launch_dequantize_fp4(type, a, v.num_sms, static_cast<cudaStream_t>(stream)));
}

int sgemm_check_args_fp4(int format, int out_type, int M, int N, int K, const uint8_t *A, int lda, const uint8_t *SA, const float *rowA,
                         const uint8_t *B, int ldb, const uint8_t *SB, const float *rowB, const float *bias, const void *C, int ldc) {
    return check_fp4(format, out_type, M, N, K, A, lda, SA, rowA, B, ldb, SB, rowB, bias, C, ldc);
}

int sgemm_run_fp4(sgemm_handle_t h, int format, int out_type, int M, int N, int K, const uint8_t *A, int lda, const uint8_t *SA,
                  const float *rowA, const uint8_t *B, int ldb, const uint8_t *SB, const float *rowB, const float *bias, void *C, int ldc,
                  void *stream) {
    int st = enter(h);
    if (st == SGEMM_OK) st = check_fp4(format, out_type, M, N, K, A, lda, SA, rowA, B, ldb, SB, rowB, bias, C, ldc);
    if (st != SGEMM_OK) return st;
    if (M == 0 || N == 0) return nothing(h);
    sg::Fp4Args a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.format = format;
    a.A = A;
    a.lda = lda;
    a.SA = SA;
    a.rowA = rowA;
    a.B = B;
    a.ldb = ldb;
    a.SB = SB;
    a.rowB = rowB;
    a.bias = bias;
    a.C = C;
    a.ldc = ldc;
    a.out_type = out_type;
    return run_fp4(h, a, static_cast<cudaStream_t>(stream));
}

int sgemm_rms_norm(sgemm_handle_t h, int type, int M, int K, const void *X, int ldx, const void *R, int ldr, const void *weight,
                   float eps, void *H, int ldh, void *Y, int ldy, float *rstd, void *stream) {
    int st = enter(h);
    if (st != SGEMM_OK) return st;
    if (ldy < std::max(1, K)) return SGEMM_ERR_INVALID_VALUE;
    if ((st = check_norm(type, M, K, X, ldx, R, ldr, weight, eps, H, ldh)) != SGEMM_OK) return st;
    if (M == 0 || K == 0) return nothing(h);
    if (Y == nullptr) return SGEMM_ERR_NULL;
    if (!aligned(Y, size_of(type)) || !aligned(rstd, 4)) return SGEMM_ERR_INVALID_VALUE;
    if ((st = norm_aliases(type, M, K, X, ldx, R, ldr, weight, H, ldh, {Range(Y, M, K, ldy, size_of(type)), floats_of(rstd, M)})) != SGEMM_OK)
        return st;
    sg::HandleView v;
    sg::view_of(h, &v);
    return launched(h, sg::launch_rms_norm(type, sg::RowOut::kSame, norm_args(M, K, X, ldx, R, ldr, weight, eps, H, ldh, Y, ldy, rstd), v.num_sms,
                                           static_cast<cudaStream_t>(stream)));
}

int sgemm_rms_norm_int8(sgemm_handle_t h, int type, int M, int K, const void *X, int ldx, const void *R, int ldr, const void *weight,
                        float eps, void *H, int ldh, int8_t *Q, int ldq, float *scale, void *stream) {
    int st = enter(h);
    if (st != SGEMM_OK) return st;
    if (ldq < std::max(1, K)) return SGEMM_ERR_INVALID_VALUE;
    if ((st = check_norm(type, M, K, X, ldx, R, ldr, weight, eps, H, ldh)) != SGEMM_OK) return st;
    if (M == 0 || K == 0) return nothing(h);
    if (Q == nullptr || scale == nullptr) return SGEMM_ERR_NULL;
    if (!aligned(scale, 4)) return SGEMM_ERR_INVALID_VALUE;
    if ((st = norm_aliases(type, M, K, X, ldx, R, ldr, weight, H, ldh, {Range(Q, M, K, ldq, 1), floats_of(scale, M)})) != SGEMM_OK) return st;
    sg::HandleView v;
    sg::view_of(h, &v);
    return launched(h, sg::launch_rms_norm(type, sg::RowOut::kInt8, norm_args(M, K, X, ldx, R, ldr, weight, eps, H, ldh, Q, ldq, scale), v.num_sms,
                                           static_cast<cudaStream_t>(stream)));
}

int sgemm_rms_norm_fp4(sgemm_handle_t h, int type, int format, int M, int K, const void *X, int ldx, const void *R, int ldr,
                       const void *weight, float eps, void *H, int ldh, uint8_t *Q, int ldq, uint8_t *S, float *row, void *stream) {
    int st = enter(h);
    if (st != SGEMM_OK) return st;
    if (!known_format(format) || M > kMaxExtent || K < 0 || ldq < std::max(1, (K + 1) / 2)) return SGEMM_ERR_INVALID_VALUE;
    if ((st = check_norm(type, M, K, X, ldx, R, ldr, weight, eps, H, ldh)) != SGEMM_OK) return st;
    if (M == 0 || K == 0) return nothing(h);
    if (row == nullptr) return SGEMM_ERR_NULL;
    if ((st = check_fp4_rows(format, K, Q, S, row)) != SGEMM_OK) return st;
    if ((st = norm_aliases(type, M, K, X, ldx, R, ldr, weight, H, ldh,
                           {Range(Q, M, (K + 1) / 2, ldq, 1), scales_of(S, format, M, K), floats_of(row, M)})) != SGEMM_OK)
        return st;
    sg::HandleView v;
    sg::view_of(h, &v);
    sg::RowArgs a = norm_args(M, K, X, ldx, R, ldr, weight, eps, H, ldh, Q, ldq, row);
    a.S = S;
    a.format = format;
    a.words = sg::fp4_words(format, K);
    return launched(h, sg::launch_rms_norm(type, sg::RowOut::kFp4, a, v.num_sms, static_cast<cudaStream_t>(stream)));
}

int sgemm_rms_norm_grad(sgemm_handle_t h, int type, int M, int K, const void *dY, int lddy, const void *dH, int lddh, const void *H,
                        int ldh, const void *weight, const float *rstd, void *dX, int lddx, float *dweight, void *stream) {
    const int st = enter(h);
    if (st != SGEMM_OK) return st;
    if (M < 0 || check_row(type, K, lddy) != SGEMM_OK || (dH && lddh < std::max(1, K)) || ldh < std::max(1, K) || lddx < std::max(1, K))
        return SGEMM_ERR_INVALID_VALUE;
    sg::HandleView v;
    sg::view_of(h, &v);
    if (static_cast<size_t>(K) > v.ws_floats) return SGEMM_ERR_INVALID_VALUE;
    if (K == 0) return nothing(h);
    if (dweight == nullptr || (M > 0 && (dY == nullptr || H == nullptr || weight == nullptr || rstd == nullptr || dX == nullptr)))
        return SGEMM_ERR_NULL;
    const int size = size_of(type);
    if (!aligned(dweight, 4) || !aligned(rstd, 4) || !aligned(dY, size) || !aligned(dH, size) || !aligned(H, size) || !aligned(weight, size) ||
        !aligned(dX, size))
        return SGEMM_ERR_INVALID_VALUE;
    const Range y(dY, M, K, lddy, size), e(dH, dH ? M : 0, K, lddh, size), x(H, M, K, ldh, size), w(weight, M ? 1 : 0, K, K, size),
        r = floats_of(rstd, M), d(dX, M, K, lddx, size), dw(dweight, 1, K, K, 4);
    if (meets_any(d, {y, x, w, r, dw}) || meets_any(dw, {y, e, x, w, r}) || (d.meets(e) && !in_place(dX, lddx, dH, lddh))) return SGEMM_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {  // no rows: the sum over them is 0
        const cudaError_t c = cudaMemsetAsync(dweight, 0, static_cast<size_t>(K) * sizeof(float), s);
        if (c != cudaSuccess) {
            (void)cudaGetLastError();
            return from_cuda(c);
        }
        return nothing(h);
    }
    sg::NormGradArgs a{};
    a.dY = dY;
    a.lddy = lddy;
    a.dH = dH;
    a.lddh = lddh;
    a.H = H;
    a.ldh = ldh;
    a.W = weight;
    a.rstd = rstd;
    a.M = M;
    a.K = K;
    a.dX = dX;
    a.lddx = lddx;
    a.dW = dweight;
    a.parts = v.d_ws;
    a.status = v.d_status;
    const int rc = from_cuda(sg::launch_rms_norm_grad(type, a, v.num_sms, v.ws_floats, s));
    if (rc == SGEMM_OK) sg::record_call(h, -1, 1, sg::norm_grad_launches(K), 0);
    return rc;
}

int sgemm_expert_layer_int8(sgemm_handle_t h, int type, int gated, int tokens, int choices, int experts, int width, int hidden,
                            const void *X, int ldx, const int *ids, const float *weights, const int8_t *up, const float *up_scale,
                            const int8_t *down, const float *down_scale, void *out, int ldo, void *stream) {
    const int st = enter(h);
    if (st != SGEMM_OK) return st;
    if ((gated != 0 && gated != 1) || tokens < 0 || tokens > sg::kLayerTokens || choices < 1 || experts < 1 || experts > sg::kMaxExperts ||
        hidden < 0 || check_row(type, width, ldx) != SGEMM_OK || check_row(type, width, ldo) != SGEMM_OK)
        return SGEMM_ERR_INVALID_VALUE;
    sg::HandleView v;
    sg::view_of(h, &v);
    const long long slots = static_cast<long long>(tokens) * choices;
    if (slots > sg::kLayerSlots || hidden > kMaxExtent || sg::layer_floats(type, static_cast<int>(slots), hidden) > v.ws_floats)
        return SGEMM_ERR_INVALID_VALUE;
    if (tokens == 0 || width == 0) return nothing(h);
    if (X == nullptr || ids == nullptr || weights == nullptr || out == nullptr ||
        (hidden > 0 && (up == nullptr || up_scale == nullptr || down == nullptr)) || down_scale == nullptr)
        return SGEMM_ERR_NULL;
    const int size = size_of(type), rows = (gated ? 2 : 1) * hidden;
    if (!aligned(X, size) || !aligned(out, size) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(up_scale, 4) || !aligned(down_scale, 4))
        return SGEMM_ERR_INVALID_VALUE;
    const Range o(out, tokens, width, ldo, size);
    if (meets_any(o, {Range(X, tokens, width, ldx, size), Range(ids, 1, slots, 1, 4), floats_of(weights, static_cast<int>(slots)),
                      Range(up, experts, static_cast<long long>(rows) * width, static_cast<long long>(rows) * width, 1),
                      Range(up_scale, experts, rows, rows, 4),
                      Range(down, experts, static_cast<long long>(width) * hidden, static_cast<long long>(width) * hidden, 1),
                      Range(down_scale, experts, width, width, 4)}))
        return SGEMM_ERR_ALIAS;
    sg::LayerArgs a{};
    a.tokens = tokens;
    a.choices = choices;
    a.experts = experts;
    a.width = width;
    a.hidden = hidden;
    a.gated = gated;
    a.X = X;
    a.ldx = ldx;
    a.ids = ids;
    a.weights = weights;
    a.up = up;
    a.up_scale = up_scale;
    a.down = down;
    a.down_scale = down_scale;
    a.out = out;
    a.ldo = ldo;
    a.h = reinterpret_cast<uint16_t *>(v.d_ws);
    a.status = v.d_status;
    const int rc = from_cuda(sg::launch_expert_layer(type, a, v.num_sms, static_cast<cudaStream_t>(stream)));
    if (rc == SGEMM_OK) sg::record_call(h, -1, 1, 2, 0);
    return rc;
}

}  // extern "C"
