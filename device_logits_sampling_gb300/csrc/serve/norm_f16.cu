#include "norm_join.cuh"

int arcs::launch_join_f16(const JoinArgs& a, Moves moves, int dev, int sms, cudaStream_t st) {
    return launch_join<ARC_F16>(a, moves, dev, sms, st);
}
