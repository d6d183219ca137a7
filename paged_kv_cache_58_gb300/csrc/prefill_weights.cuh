// Accumulated attention weights of a prompt chunk: what the CUDA-core and the tensor-core form
// share.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace pkv {

// What request r asks for, checked: n new tokens after c cached ones, of which the last m count,
// `rows` query rows of a kv head, from q row qoff on, into weight row wrow.  rows = 0: nothing to
// do, or out of range, which is reported.
struct Request {
    int n, c, m, rows, qoff, wrow;
};
PKV_DEVINL Request request_of(const PrefillWeightsArgs& a, int r, int group, bool report) {
    Request q;
    q.n = __ldg(a.new_lens + r);
    q.c = __ldg(a.cached_lens + r);
    q.qoff = __ldg(a.q_offsets + r);
    q.wrow = a.row_ids ? __ldg(a.row_ids + r) : r;
    q.m = a.window > 0 ? min(a.window, q.n) : q.n;
    q.rows = 0;
    if (q.n <= 0 || q.wrow < 0) return q;   // no new tokens, or a padding row
    if (q.c < 0 || static_cast<int64_t>(q.c) + q.n > a.max_context || q.n > a.max_new ||
        q.wrow >= a.num_rows || q.qoff < 0 ||
        static_cast<int64_t>(q.qoff) + q.n > a.total_new) {
        if (report) raise_status(a.status, PKV_ERR_OOB);
        return q;
    }
    q.rows = q.m * group;
    return q;
}

}  // namespace pkv
