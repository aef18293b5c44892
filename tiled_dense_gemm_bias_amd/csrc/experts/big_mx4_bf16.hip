#include "gx_launch.hpp"

GBX_BIG_TABLE(big_mx4_bf16, 2, 1, EPI_ACT, true)
