#include "gx_launch.hpp"

GBX_BIG_TABLE(big_fwd_nn_f16, 0, 0, EPI_ACT, false)
