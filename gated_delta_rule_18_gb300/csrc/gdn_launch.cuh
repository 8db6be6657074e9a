// gdn_launch.cuh -- launch accounting shared by the C entry points: every
// kernel launch goes through launch(), which counts it and, while profiling
// is on, brackets it with a CUDA event pair on its own stream.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <mutex>
#include <vector>

namespace gdn {

enum Kind {
    KPrepL2 = 0, KPrepRms, KTable, KIntra, KState, KFusedF32, KMerge, KFrameGram, KFrameChain,
    KFrameOut, KSegSummary, KSegCombine, KBwdDh, KBwdDq, KBwdDk, KSum, KF32Prep, KF32Serial, KFused,
    KFrameXt, KFrameLam, KFrameTok, KPrepBwd, KMergeBwd, KBwdF32Scan, KBwdF32Reduce, KNorm, KNormBwd,
    KColSum, KConv, KConvBwd, KConvStep, KSsmSum, KSsmChain, KSsmScan, KSsmBwdSum, KSsmBwdChain,
    KSsmBwd, KSsmBwdReduce, KSsmStep, KNumKinds
};
inline const char *kind_name(int kind) {
    static const char *const names[KNumKinds] = {
        "prep_l2", "prep_rms", "chunk_table", "intra_bf16", "state_tc", "fused_f32", "merge", "frame_gram",
        "frame_chain", "frame_out", "seg_summary", "seg_combine", "bwd_dh", "bwd_dq", "bwd_dk", "dir_sum",
        "f32_prep", "f32_serial", "fused_tc", "frame_xt", "frame_lam", "frame_tokgrad", "prep_bwd",
        "merge_bwd", "bwd_f32_scan", "bwd_f32_reduce", "rmsnorm", "rmsnorm_bwd", "col_sum", "conv",
        "conv_bwd", "conv_step", "ssm_sum", "ssm_chain", "ssm_scan", "ssm_bwd_sum", "ssm_bwd_chain",
        "ssm_bwd", "ssm_bwd_reduce", "ssm_step"};
    return names[kind];
}

struct Profiler {
    std::mutex mu;
    std::atomic<bool> on{false};
    std::vector<cudaEvent_t> pool;
    struct Rec {
        int kind;
        cudaEvent_t a, b;
    };
    std::vector<Rec> recs;
};
inline Profiler &prof() {
    static Profiler *p = new Profiler();  // never destroyed: safe at exit
    return *p;
}
inline std::atomic<long long> &launches() {
    static std::atomic<long long> n{0};
    return n;
}

inline cudaEvent_t take_event(Profiler &P) {
    if (!P.pool.empty()) {
        cudaEvent_t e = P.pool.back();
        P.pool.pop_back();
        return e;
    }
    cudaEvent_t e = nullptr;
    if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
    return e;
}

template <class F>
cudaError_t launch(int kind, cudaStream_t st, F &&f) {
    Profiler &P = prof();
    cudaEvent_t a = nullptr, b = nullptr;
    if (P.on.load(std::memory_order_relaxed)) {
        std::lock_guard<std::mutex> g(P.mu);
        a = take_event(P);
        b = take_event(P);
    }
    if (a && b) cudaEventRecord(a, st);
    cudaError_t e = f();
    if (e == cudaSuccess) launches().fetch_add(1);
    if (a && b) {
        cudaEventRecord(b, st);
        std::lock_guard<std::mutex> g(P.mu);
        P.recs.push_back({kind, a, b});
    }
    return e;
}

}  // namespace gdn
