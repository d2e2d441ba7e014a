// Tables of the group norm's launchers by vector width and activation.
#pragma once

#include "groupnorm_fused.cuh"
#include "groupnorm_stream.cuh"

namespace rowops {

template <typename T, int VEC, int ACT>
cudaError_t gn_forward_launch(const void* x, void* y, const void* w, const void* b, float* stats, void* ws, GnArgs a,
                              const GnFused* f, const LaunchCfg& cfg) {
    return f ? gn_forward_fused<T, VEC, ACT>(x, y, w, b, stats, a, *f, cfg)
             : gn_forward_stream<T, VEC, ACT>(x, y, w, b, stats, ws, a, cfg);
}

template <typename T, int VEC, int ACT>
cudaError_t gn_backward_launch(const void* x, const void* dy, const void* w, const void* b, const float* stats,
                               void* dx, float* dw, float* db, void* ws, GnArgs a, const GnFused* f,
                               const LaunchCfg& cfg) {
    return f ? gn_backward_fused<T, VEC, ACT>(x, dy, w, b, stats, dx, dw, db, ws, a, *f, cfg)
             : gn_backward_stream<T, VEC, ACT>(x, dy, w, b, stats, dx, dw, db, ws, a, cfg);
}

template <typename T>
GnForwardLaunch gn_forward_table(int vec, int act) {
    constexpr int V = Elem<T>::kVec;
    static const GnForwardLaunch t[3][4] = {
        {gn_forward_launch<T, 1, 0>, gn_forward_launch<T, 1, 1>, gn_forward_launch<T, 1, 2>, gn_forward_launch<T, 1, 3>},
        {gn_forward_launch<T, 2, 0>, gn_forward_launch<T, 2, 1>, gn_forward_launch<T, 2, 2>, gn_forward_launch<T, 2, 3>},
        {gn_forward_launch<T, V, 0>, gn_forward_launch<T, V, 1>, gn_forward_launch<T, V, 2>, gn_forward_launch<T, V, 3>}};
    return t[vec < 2 ? 0 : (vec == 2 ? 1 : 2)][act];
}

template <typename T>
GnBackwardLaunch gn_backward_table(int vec, int act) {
    constexpr int V = Elem<T>::kVec;
    static const GnBackwardLaunch t[3][4] = {{gn_backward_launch<T, 1, 0>, gn_backward_launch<T, 1, 1>,
                                              gn_backward_launch<T, 1, 2>, gn_backward_launch<T, 1, 3>},
                                             {gn_backward_launch<T, 2, 0>, gn_backward_launch<T, 2, 1>,
                                              gn_backward_launch<T, 2, 2>, gn_backward_launch<T, 2, 3>},
                                             {gn_backward_launch<T, V, 0>, gn_backward_launch<T, V, 1>,
                                              gn_backward_launch<T, V, 2>, gn_backward_launch<T, V, 3>}};
    return t[vec < 2 ? 0 : (vec == 2 ? 1 : 2)][act];
}

}  // namespace rowops
