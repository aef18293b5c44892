#include "gx_launch.hpp"

GBX_RING_TABLE(part_nt, EPI_PART, true)
GBX_RING_TABLE(part_nn, EPI_PART, false)
