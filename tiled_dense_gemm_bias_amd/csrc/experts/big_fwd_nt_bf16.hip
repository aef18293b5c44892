#include "gx_launch.hpp"

GBX_BIG_TABLE(big_fwd_nt_bf16, 1, 1, EPI_ACT, true)
