#include "gm_launch.hpp"

GBM_BIG_TABLE(big_f8_act_bf16, 1, EPI_ACT)
