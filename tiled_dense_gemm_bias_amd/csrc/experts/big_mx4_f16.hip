#include "gx_launch.hpp"

GBX_BIG_TABLE(big_mx4_f16, 2, 0, EPI_ACT, true)
