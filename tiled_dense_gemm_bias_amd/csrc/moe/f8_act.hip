#include "gm_launch.hpp"

GBM_RING_TABLE(f8_act, EPI_ACT)
