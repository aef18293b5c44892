#include "gm_launch.hpp"

GBM_STREAM_TABLE(f8_stream_act, EPI_ACT)
GBM_STREAM_TABLE(f8_stream_slope, EPI_SLOPE)
