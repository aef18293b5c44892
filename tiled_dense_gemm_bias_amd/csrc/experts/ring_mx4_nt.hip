#include "gx_launch.hpp"

GBX_MX4_TABLE(mx4_nt)
GBX_MX4_PART_TABLE(part_mx4)
