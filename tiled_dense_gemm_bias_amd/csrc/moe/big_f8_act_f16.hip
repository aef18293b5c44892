#include "gm_launch.hpp"

GBM_BIG_TABLE(big_f8_act_f16, 0, EPI_ACT)
