#include "gx_launch.hpp"

GBX_BIG_TABLE(big_slope_nn_bf16, 1, 1, EPI_SLOPE, false)
