// C ABI of the int8 products and of the expert routing (declared in
// include/sgemm.h): argument validation, the choice of path, tile and split,
// the TMA descriptors and the launches.  Every computation is done by the
// kernels in sgemm_int8.cu and sgemm_experts.cu.
#include <algorithm>
#include <climits>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "api_common.h"
#include "context.h"
#include "internal.h"
#include "sgemm.h"

namespace {

// K up to which a sum of K products of two int8 stays inside int32.
constexpr int kMaxInt8K = 131071;

// Token tile and K split of a tensor-core call, by the time that this model
// gives each choice (microseconds, from calls measured back to back in CUDA
// graphs over M 1 .. 8192, N and K 256 .. 8192; it orders the choices right
// where they differ by more than a tenth):
//   direct tiles: a launch, the exchange of partial sums, and a stage of 128 k at
//     a time -- `alone` with one CTA on an SM, `shared` a CTA with two;
//   pair tiles: two launches, the conversion of the tokens to FP16 (one read and
//     one write of HBM), and the stages of complete waves of pairs.
// E.g. 4096 x 4096 weights: M = 16 on tiles of 16, four-way split, 7.7 us (whole
// K 15.8, tiles of 64 11.0); M = 256 on tiles of 64, two-way, 20.8 (pairs of
// 128: 22.3, whole K 22.0); M = 512 on pairs of 128 24.8 (tiles of 64 32.2, pairs of
// 256 30.0); M = 2048 on pairs of 256 56 (of 128 72).
struct TileChoice {
    int nt, ksplit;
    double us;
};
TileChoice choose_tile(int rows, int experts, int N, int K, int num_sms, bool direct_copy) {
    struct Direct {
        int nt;
        double alone, shared, exchange;
    };
    constexpr Direct kDirect[] = {{16, 0.36, 0.35, 0.7}, {32, 0.42, 0.34, 1.2}, {64, 0.53, 0.43, 2.2}};
    struct Pair {
        int nt;
        double fixed, stage;
    };
    constexpr Pair kPair[] = {{128, 7.0, 0.49}, {256, 7.5, 0.68}};
    const int owners = std::min(experts, std::max(rows, 1));
    const long long each = cdiv(rows, owners);
    const int stages = static_cast<int>(cdiv(K, sg::kI8StageK));
    TileChoice best{256, 1, 1e30};
    for (const Direct &d : kDirect) {
        const long long tiles = owners * cdiv(each, d.nt) * cdiv(N, sg::kI8TileN);
        for (int s = 1; s <= 8 && s <= stages; s *= 2) {
            const long long ctas = tiles * s;
            if (s > 1 && ctas > 2 * num_sms) break;
            const double stage = ctas <= num_sms ? d.alone : 2 * d.shared;
            const double t = 4.3 + (direct_copy ? 2.0 : 0.0) + (s > 1 ? d.exchange + 0.1 * s : 0.0) +
                             static_cast<double>(cdiv(ctas, 2LL * num_sms)) * static_cast<double>(cdiv(stages, s)) * stage;
            if (t < best.us) best = {d.nt, s, t};
        }
    }
    for (const Pair &p : kPair) {
        const long long units = owners * cdiv(each, p.nt) * cdiv(N, 2 * sg::kI8TileN);
        const double t = p.fixed + 3.0 * rows * K / 5.5e6 + static_cast<double>(cdiv(units, num_sms / 2)) * stages * p.stage;
        if (t < best.us) best = {p.nt, 1, t};
    }
    return best;
}

// Whether the kernel for few tokens beats the tensor cores' `tc_us` (by the same
// kind of model; B's copy, which only they need, counted): a launch, B at the rate
// that a warp's arithmetic leaves (lower on rows that have to be shifted), and
// the tokens' way into shared memory.  E.g. one token 4.9 us against 6.8 (4096 x 4096),
// 17.0 against 36.7 (8190 x 8190, rows on no boundary), 4 tokens 18.4 against 14.7 (8192 x
// 8192) and 2.7 against 6.1 (700 x 701), 8 tokens 11.3 against 6.9 and 3.0 against 6.1.
// (Eight tokens on shifted rows take 0.42 to 0.65 us a MB; 0.9 makes up for what `tc_us`
// overestimates there: 8 x 4096 x 4097 15.4 us against 13.9, x 2048 x 2049 8.5 against 8.4.)
bool choose_few(int rows, int N, int K, bool b_aligned, double tc_us) {
    constexpr double kAligned[] = {0.14, 0.17, 0.23, 0.43}, kShifted[] = {0.205, 0.23, 0.3, 0.9};  // us a MB
    const int i = rows <= 1 ? 0 : rows <= 2 ? 1 : rows <= 4 ? 2 : 3;
    const double mb = 1e-6 * N * K;
    const double few = 2.9 + (b_aligned ? kAligned[i] : kShifted[i]) * mb;
    return few + 5e-5 * rows * K < tc_us + (b_aligned ? 0.0 : 2.0 + 0.28 * mb);
}

// Whether the kernel for few tokens beats the generic one, where the tensor cores
// cannot run (B needs a copy that it may not or cannot have).  The generic kernel takes
// 1.4 us for every 64 of K and computes 64 rows whatever the tokens: 1 token x 4096 x 4097
// 91 us against 6.1, 8 tokens x 700 x 701 17 against 3.1, 4 x 16384 x 129 8.7 against 6.2.
// On a short K its tiles are the better use of a wave, where channels make many: 8 x
// 30000 x 17 7.6 us against 15.5, 4 x 16384 x 17 4.4 against 6.1 (8 x 100000 x 129 42
// against 49; one to four tokens 42 against 26 to 30).
bool few_beats_generic(int N, int K) { return N <= 8192 || K > 128; }

int check_int8(int transB, int out_type, int experts, int rows, int N, int K, const int *offsets, bool grouped,
               const int8_t *A, int lda, const float *scaleA, const int8_t *B, int ldb, long long strideB,
               const float *scaleB, const float *bias, const void *C, int ldc) {
    if (!known_type(out_type) || (transB != 0 && transB != 1)) return SGEMM_ERR_INVALID_VALUE;
    if (rows < 0 || N < 0 || K < 0 || K > kMaxInt8K || rows > kMaxExtent || N > kMaxExtent) return SGEMM_ERR_INVALID_VALUE;
    if (experts < 1 || experts > sg::kMaxExperts) return SGEMM_ERR_INVALID_VALUE;
    const int b_rows = transB ? N : K, b_cols = transB ? K : N;  // B as stored
    if (lda < std::max(1, K) || ldb < std::max(1, b_cols) || ldc < std::max(1, N) || strideB < 0)
        return SGEMM_ERR_INVALID_VALUE;
    if (rows == 0 || N == 0) return SGEMM_OK;
    if (C == nullptr || scaleA == nullptr || scaleB == nullptr) return SGEMM_ERR_NULL;
    if (K > 0 && (A == nullptr || B == nullptr)) return SGEMM_ERR_NULL;
    if (grouped && offsets == nullptr) return SGEMM_ERR_NULL;
    if (!aligned(C, size_of(out_type)) || !aligned(scaleA, 4) || !aligned(scaleB, 4) || !aligned(bias, 4) ||
        !aligned(offsets, 4))
        return SGEMM_ERR_INVALID_VALUE;
    const Range c(C, rows, N, ldc, size_of(out_type)), a(A, rows, K, lda, 1), sa(scaleA, 1, rows, rows, 4);
    const Range sb(scaleB, experts, N, N, 4), bi(bias, bias ? experts : 0, N, N, 4);
    const Range of(offsets, offsets ? 1 : 0, experts + 1, experts + 1, 4);
    Range b(B, b_rows, b_cols, ldb, 1);
    if (K > 0) b.hi += static_cast<uintptr_t>(experts - 1) * static_cast<uintptr_t>(strideB);
    if ((K > 0 && (c.meets(a) || c.meets(b))) || c.meets(sa) || c.meets(sb) || c.meets(bi) || c.meets(of))
        return SGEMM_ERR_ALIAS;
    return SGEMM_OK;
}

int run_int8(sgemm_handle_t h, int transB, int out_type, int experts, int rows, int N, int K, const int *offsets,
             const int8_t *A, int lda, const float *scaleA, const int8_t *B, int ldb, long long strideB,
             const float *scaleB, const float *bias, void *C, int ldc, cudaStream_t stream) {
    sg::HandleView v;
    sg::view_of(h, &v);
    int launches = 0, copied = 0, variant = SGEMM_VARIANT_GENERIC_I8;
    sg::Int8Args a{};
    a.rows = a.total_rows = rows;
    a.N = N;
    a.K = K;
    a.experts = experts;
    a.offsets = offsets;
    a.A = A;
    a.lda = lda;
    a.B = B;
    a.ldb = ldb;
    a.strideB = strideB;
    a.transB = transB;
    a.scaleA = scaleA;
    a.scaleB = scaleB;
    a.bias = bias;
    a.C = C;
    a.ldc = ldc;
    a.out_type = out_type;
    a.status = v.d_status;
    a.ksplit = 1;

    // Tiles of up to 64 tokens read the tokens' int8 rows, by TMA: rows on other
    // than 16-byte boundaries are copied first.  Wider tiles read them as FP16.
    const bool a_aligned = aligned(A, 16) && lda % 16 == 0;
    TileChoice tile = choose_tile(rows, experts, N, std::max(K, 1), v.num_sms, !a_aligned);
    if (v.i8_tokens) {
        tile.nt = v.i8_tokens;
        tile.ksplit = v.i8_split;
        while (tile.ksplit > 1 && tile.ksplit > cdiv(K, sg::kI8StageK)) tile.ksplit /= 2;
    }
    a.nt = tile.nt;
    const bool direct = a.nt <= 64;
    const bool a_as_stored = direct && a_aligned;
    const int kp = static_cast<int>(cdiv(K, 64) * 64), kb = static_cast<int>(cdiv(K, 16) * 16);
    const size_t a_row = a_as_stored ? 0 : direct ? static_cast<size_t>(kb) : static_cast<size_t>(kp) * 2;

    // The re-layout workspace: B where the TMA cannot read it as stored, then
    // the tokens' rows, as many at a time as fit.
    uint8_t *ws = reinterpret_cast<uint8_t *>(v.d_rl);
    size_t room = v.rl_bytes;
    const bool as_stored = transB && aligned(B, 16) && ldb % 16 == 0 && (experts == 1 || strideB % 16 == 0);
    const size_t b_bytes = as_stored ? 0 : static_cast<size_t>(experts) * N * kb;
    const size_t peak_room = direct ? 0 : sg::kI8Peaks * sizeof(int);
    const size_t b_room = (b_bytes + 1023) / 1024 * 1024 + peak_room;
    bool tc = v.pinned != SGEMM_VARIANT_GENERIC && v.pinned != SGEMM_VARIANT_GENERIC_I8 && K > 0 &&
              ((as_stored && a_as_stored) || ws != nullptr) && (as_stored || v.relayout_mode != SGEMM_RELAYOUT_OFF) &&
              b_room <= room && room - b_room >= a_row * std::min(rows, a.nt);
    if (experts == 1 && !offsets && transB && K > 0 && rows <= sg::kI8FewRows &&
        sg::int8_few_bytes(rows, K) <= sg::kI8FewBytes &&
        (v.pinned == SGEMM_VARIANT_FEW_I8 ||
         (v.pinned != SGEMM_VARIANT_TC_I8 && v.pinned != SGEMM_VARIANT_GENERIC_I8 && v.pinned != SGEMM_VARIANT_GENERIC &&
          (tc ? choose_few(rows, N, K, as_stored, tile.us) : few_beats_generic(N, K))))) {
        const cudaError_t e = sg::launch_int8_few(a, v.num_sms, stream);
        if (e != cudaSuccess) return from_cuda(e);
        sg::record_call(h, SGEMM_VARIANT_FEW_I8, 1, 1, 0);
        return SGEMM_OK;
    }
    const long long ch_tiles = cdiv(N, sg::kI8TileN);
    int per = rows;  // rows of one pass
    if (tc) {
        if (a_row) {
            const long long fit = static_cast<long long>((room - b_room) / a_row);
            if (fit < rows) per = static_cast<int>(fit / a.nt * a.nt);
        }
        const long long tiles = sg::int8_most_tiles(per, experts, a.nt) * ch_tiles;
        tc = tiles < INT_MAX && (static_cast<long long>(per / a.nt) + experts) * ch_tiles < INT_MAX;
        a.ksplit = tile.ksplit;
    }
    CUtensorMap tmB, tmA;
    sg::Int8Copies copies{};
    if (tc) {
        if (!as_stored) {
            copies.B = B;
            copies.ldb = ldb;
            copies.strideB = strideB;
            copies.b_trans = transB;
            copies.b_dst = reinterpret_cast<int8_t *>(ws);
            copies.b_ld = kb;
            a.B = copies.b_dst;
            a.ldb = kb;
            a.strideB = static_cast<long long>(N) * kb;
        }
        copies.lda = lda;
        copies.K = K;
        copies.experts = experts;
        copies.N = N;
        if (a_row) {
            if (!direct) a.peaks = copies.peaks = reinterpret_cast<int *>(ws + b_room - peak_room);
            ws += b_room;
            copies.a_dst = ws;
            copies.a_ld = direct ? kb : kp;
        }
        // a single matrix has any (aligned) matrix stride
        const long long stride = experts > 1 ? a.strideB : a.ldb * static_cast<long long>(N);
        tc = sg::encode_map(&tmB, sg::MapType::kInt8, 3, a.B, K, N, experts, a.ldb, stride, sg::kI8StageK,
                            sg::kI8TileN) &&
             (direct ? sg::encode_map(&tmA, sg::MapType::kInt8, 2, a_as_stored ? static_cast<const void *>(A) : ws, K, per,
                                      1, a_as_stored ? lda : kb, 0, sg::kI8StageK, a.nt)
                     : sg::encode_map(&tmA, sg::MapType::kF16, 2, ws, kp, per, 1, static_cast<long long>(kp) * 2, 0,
                                      64, a.nt / 4));
    }
    if (tc) {
        variant = SGEMM_VARIANT_TC_I8;
        if (copies.b_dst) copied = 2;
        for (int r0 = 0; r0 < rows; r0 += per) {
            a.row0 = r0;
            a.rows = std::min(per, rows - r0);
            cudaError_t e = cudaSuccess;
            if (copies.a_dst || copies.b_dst) {
                copies.A = A + static_cast<long long>(r0) * lda;
                copies.a_rows = a.rows;
                e = sg::launch_int8_copies(&copies, stream);
                a.n_peaks = copies.a_blocks;
                copies.b_dst = nullptr;  // once
                ++launches;
            }
            if (e == cudaSuccess) e = sg::launch_int8_tc(a, tmB, tmA, v.num_sms, v.smem_override, stream);
            if (e != cudaSuccess) return from_cuda(e);
            ++launches;
        }
    } else {
        a.ksplit = 1;
        a.B = B;  // as stored
        a.ldb = ldb;
        a.strideB = strideB;
        const cudaError_t e = sg::launch_int8_generic(a, stream);
        if (e != cudaSuccess) return from_cuda(e);
        ++launches;
    }
    sg::record_call(h, variant, a.ksplit, launches, copied);
    return SGEMM_OK;
}

// Sizes and the slots of a routing call.
int check_slots(int tokens, int choices) {
    if (tokens < 0 || choices < 1) return SGEMM_ERR_INVALID_VALUE;
    if (static_cast<long long>(tokens) * choices > INT_MAX) return SGEMM_ERR_INVALID_VALUE;
    return SGEMM_OK;
}

}  // namespace

extern "C" {

int sgemm_check_args_int8(int transB, int out_type, int M, int N, int K, const int8_t *A, int lda,
                          const float *scaleA, const int8_t *B, int ldb, const float *scaleB, const float *bias,
                          const void *C, int ldc) {
    return check_int8(transB, out_type, 1, M, N, K, nullptr, false, A, lda, scaleA, B, ldb, 0, scaleB, bias, C, ldc);
}

int sgemm_check_args_int8_experts(int transB, int out_type, int experts, int rows, int N, int K, const int *offsets,
                                  const int8_t *A, int lda, const float *scaleA, const int8_t *B, int ldb,
                                  long long strideB, const float *scaleB, const float *bias, const void *C, int ldc) {
    return check_int8(transB, out_type, experts, rows, N, K, offsets, true, A, lda, scaleA, B, ldb, strideB, scaleB,
                      bias, C, ldc);
}

int sgemm_run_int8(sgemm_handle_t h, int transB, int out_type, int M, int N, int K, const int8_t *A, int lda,
                   const float *scaleA, const int8_t *B, int ldb, const float *scaleB, const float *bias, void *C,
                   int ldc, void *stream) {
    int st = enter(h);
    if (st == SGEMM_OK)
        st = check_int8(transB, out_type, 1, M, N, K, nullptr, false, A, lda, scaleA, B, ldb, 0, scaleB, bias, C, ldc);
    if (st != SGEMM_OK) return st;
    if (M == 0 || N == 0) return nothing(h);
    return run_int8(h, transB, out_type, 1, M, N, K, nullptr, A, lda, scaleA, B, ldb, 0, scaleB, bias, C, ldc,
                    static_cast<cudaStream_t>(stream));
}

int sgemm_run_int8_experts(sgemm_handle_t h, int transB, int out_type, int experts, int rows, int N, int K,
                           const int *offsets, const int8_t *A, int lda, const float *scaleA, const int8_t *B,
                           int ldb, long long strideB, const float *scaleB, const float *bias, void *C, int ldc,
                           void *stream) {
    int st = enter(h);
    if (st == SGEMM_OK)
        st = check_int8(transB, out_type, experts, rows, N, K, offsets, true, A, lda, scaleA, B, ldb, strideB,
                        scaleB, bias, C, ldc);
    if (st != SGEMM_OK) return st;
    if (rows == 0 || N == 0) return nothing(h);
    return run_int8(h, transB, out_type, experts, rows, N, K, offsets, A, lda, scaleA, B, ldb, strideB, scaleB, bias,
                    C, ldc, static_cast<cudaStream_t>(stream));
}

int sgemm_quantize_rows(sgemm_handle_t h, int type, int M, int K, const void *X, int ldx, int8_t *Q, int ldq,
                        float *scale, void *stream) {
    int st = enter(h);
    if (st != SGEMM_OK) return st;
    if (M < 0 || check_row(type, K, ldx) != SGEMM_OK || ldq < std::max(1, K)) return SGEMM_ERR_INVALID_VALUE;
    sg::HandleView v;
    sg::view_of(h, &v);
    if (M == 0) return nothing(h);
    if (scale == nullptr || (K > 0 && (X == nullptr || Q == nullptr))) return SGEMM_ERR_NULL;
    if (!aligned(X, size_of(type)) || !aligned(scale, 4)) return SGEMM_ERR_INVALID_VALUE;
    const Range x(X, M, K, ldx, size_of(type)), q(Q, M, K, ldq, 1), s(scale, 1, M, M, 4);
    if (x.meets(q) || x.meets(s) || q.meets(s)) return SGEMM_ERR_ALIAS;
    sg::MoveArgs a{};
    a.X = X;
    a.ldx = ldx;
    a.tokens = M;
    a.choices = 1;
    a.width = K;
    a.Y = Q;
    a.ldy = ldq;
    a.scale = scale;
    return launched(h, sg::launch_quantize(type, a, v.num_sms, static_cast<cudaStream_t>(stream)));
}

int sgemm_expert_sort(sgemm_handle_t h, int tokens, int choices, int experts, const int *ids, int *offsets,
                      int *rows, int *source, void *stream) {
    int st = enter(h);
    if (st == SGEMM_OK) st = check_slots(tokens, choices);
    if (st != SGEMM_OK) return st;
    if (experts < 1 || experts > sg::kMaxExperts) return SGEMM_ERR_INVALID_VALUE;
    const int slots = tokens * choices;
    if (offsets == nullptr || (slots > 0 && (ids == nullptr || rows == nullptr || source == nullptr)))
        return SGEMM_ERR_NULL;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(source, 4))
        return SGEMM_ERR_INVALID_VALUE;
    const Range i(ids, 1, slots, slots, 4), o(offsets, 1, experts + 1, experts + 1, 4), r(rows, 1, slots, slots, 4),
        s(source, 1, slots, slots, 4);
    if (i.meets(o) || i.meets(r) || i.meets(s) || o.meets(r) || o.meets(s) || r.meets(s)) return SGEMM_ERR_ALIAS;
    sg::HandleView v;
    sg::view_of(h, &v);
    if (slots > sg::sort_most_slots(v.ws_floats, experts)) return SGEMM_ERR_INVALID_VALUE;
    int launches = 0;
    const int rc = from_cuda(sg::launch_sort(ids, slots, experts, offsets, rows, source, reinterpret_cast<int *>(v.d_ws),
                                             &launches, static_cast<cudaStream_t>(stream)));
    if (rc == SGEMM_OK) sg::record_call(h, -1, 1, launches, 0);
    return rc;
}

int sgemm_expert_dispatch(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *X, int ldx,
                          const int *rows, void *Y, int ldy, void *stream) {
    int st = enter(h);
    if (st == SGEMM_OK) st = check_slots(tokens, choices);
    if (st == SGEMM_OK) st = check_row(type, width, ldx);
    if (st == SGEMM_OK) st = check_row(type, width, ldy);
    if (st != SGEMM_OK) return st;
    if (tokens == 0 || width == 0) return nothing(h);
    if (X == nullptr || Y == nullptr || rows == nullptr) return SGEMM_ERR_NULL;
    const int size = size_of(type);
    if (!aligned(X, size) || !aligned(Y, size) || !aligned(rows, 4)) return SGEMM_ERR_INVALID_VALUE;
    const int slots = tokens * choices;
    const Range x(X, tokens, width, ldx, size), y(Y, slots, width, ldy, size), r(rows, 1, slots, slots, 4);
    if (y.meets(x) || y.meets(r)) return SGEMM_ERR_ALIAS;
    sg::MoveArgs a{};
    a.X = X;
    a.ldx = ldx;
    a.tokens = tokens;
    a.choices = choices;
    a.width = width;
    a.rows = rows;
    a.Y = Y;
    a.ldy = ldy;
    return launched(h, sg::launch_dispatch(type, a, static_cast<cudaStream_t>(stream)));
}

int sgemm_expert_dispatch_int8(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *X, int ldx,
                               const int *rows, int8_t *Q, int ldq, float *scale, void *stream) {
    int st = enter(h);
    if (st == SGEMM_OK) st = check_slots(tokens, choices);
    if (st == SGEMM_OK) st = check_row(type, width, ldx);
    if (st != SGEMM_OK) return st;
    if (ldq < std::max(1, width)) return SGEMM_ERR_INVALID_VALUE;
    if (tokens == 0) return nothing(h);
    if (rows == nullptr || scale == nullptr || (width > 0 && (X == nullptr || Q == nullptr))) return SGEMM_ERR_NULL;
    const int size = size_of(type), slots = tokens * choices;
    if (!aligned(X, size) || !aligned(scale, 4) || !aligned(rows, 4)) return SGEMM_ERR_INVALID_VALUE;
    const Range x(X, tokens, width, ldx, size), q(Q, slots, width, ldq, 1), r(rows, 1, slots, slots, 4),
        s(scale, 1, slots, slots, 4);
    if (q.meets(x) || q.meets(r) || q.meets(s) || s.meets(x) || s.meets(r)) return SGEMM_ERR_ALIAS;
    sg::HandleView v;
    sg::view_of(h, &v);
    sg::MoveArgs a{};
    a.X = X;
    a.ldx = ldx;
    a.tokens = tokens;
    a.choices = choices;
    a.width = width;
    a.rows = rows;
    a.Y = Q;
    a.ldy = ldq;
    a.scale = scale;
    return launched(h, sg::launch_quantize(type, a, v.num_sms, static_cast<cudaStream_t>(stream)));
}

// out[t] = sum_j w[t][j] * Y[rows[t][j]] (weights NULL only from dispatch_grad).
static int run_gather(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *Y, int ldy,
                      const int *rows, bool weighted, const float *weights, void *out, int ldo, void *stream) {
    int st = enter(h);
    if (st == SGEMM_OK) st = check_slots(tokens, choices);
    if (st == SGEMM_OK) st = check_row(type, width, ldy);
    if (st == SGEMM_OK) st = check_row(type, width, ldo);
    if (st != SGEMM_OK) return st;
    if (tokens == 0 || width == 0) return nothing(h);
    if (Y == nullptr || rows == nullptr || out == nullptr || (weighted && weights == nullptr)) return SGEMM_ERR_NULL;
    const int size = size_of(type), slots = tokens * choices;
    if (!aligned(Y, size) || !aligned(out, size) || !aligned(rows, 4) || !aligned(weights, 4))
        return SGEMM_ERR_INVALID_VALUE;
    const Range y(Y, slots, width, ldy, size), o(out, tokens, width, ldo, size), r(rows, 1, slots, slots, 4),
        w(weights, weights ? 1 : 0, slots, slots, 4);
    if (o.meets(y) || o.meets(r) || o.meets(w)) return SGEMM_ERR_ALIAS;
    sg::MoveArgs a{};
    a.X = out;
    a.ldx = ldo;
    a.tokens = tokens;
    a.choices = choices;
    a.width = width;
    a.rows = rows;
    a.weights = weights;
    a.Y = const_cast<void *>(Y);
    a.ldy = ldy;
    return launched(h, sg::launch_gather(type, a, static_cast<cudaStream_t>(stream)));
}

int sgemm_expert_dispatch_grad(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *dY,
                               int lddy, const int *rows, void *dX, int lddx, void *stream) {
    return run_gather(h, type, tokens, choices, width, dY, lddy, rows, false, nullptr, dX, lddx, stream);
}

int sgemm_expert_combine(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *Y, int ldy,
                         const int *rows, const float *weights, void *out, int ldo, void *stream) {
    return run_gather(h, type, tokens, choices, width, Y, ldy, rows, true, weights, out, ldo, stream);
}

int sgemm_expert_combine_grad(sgemm_handle_t h, int type, int tokens, int choices, int width, const void *dout,
                              int lddo, const void *Y, int ldy, const int *rows, const float *weights, void *dY,
                              int lddy, float *dweights, void *stream) {
    int st = enter(h);
    if (st == SGEMM_OK) st = check_slots(tokens, choices);
    if (st == SGEMM_OK) st = check_row(type, width, lddo);
    if (st == SGEMM_OK) st = check_row(type, width, ldy);
    if (st == SGEMM_OK) st = check_row(type, width, lddy);
    if (st != SGEMM_OK) return st;
    if (tokens == 0) return nothing(h);
    if (rows == nullptr || weights == nullptr || dweights == nullptr ||
        (width > 0 && (dout == nullptr || Y == nullptr || dY == nullptr)))
        return SGEMM_ERR_NULL;
    const int size = size_of(type), slots = tokens * choices;
    if (!aligned(dout, size) || !aligned(Y, size) || !aligned(dY, size) || !aligned(rows, 4) ||
        !aligned(weights, 4) || !aligned(dweights, 4))
        return SGEMM_ERR_INVALID_VALUE;
    const Range g(dout, tokens, width, lddo, size), y(Y, slots, width, ldy, size), d(dY, slots, width, lddy, size),
        r(rows, 1, slots, slots, 4), w(weights, 1, slots, slots, 4), dw(dweights, 1, slots, slots, 4);
    if (d.meets(g) || d.meets(y) || d.meets(r) || d.meets(w) || d.meets(dw) || dw.meets(g) || dw.meets(y) ||
        dw.meets(r) || dw.meets(w))
        return SGEMM_ERR_ALIAS;
    sg::MoveArgs a{};
    a.X = dout;
    a.ldx = lddo;
    a.tokens = tokens;
    a.choices = choices;
    a.width = width;
    a.rows = rows;
    a.weights = weights;
    a.Y = const_cast<void *>(Y);
    a.ldy = ldy;
    a.dY = dY;
    a.lddy = lddy;
    a.scale = dweights;
    return launched(h, sg::launch_combine_grad(type, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
